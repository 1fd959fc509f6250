"""Plain 64-bit forms of the feed-forward operators and the error bounds their
kernels are held to (used by the CPU and the GPU tests)."""
from __future__ import annotations

import math

import numpy as np
import torch

ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24                       # half a step of fp32


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def smallest(dtype) -> float:
    """Half the spacing of the type's subnormals: the absolute part of a rounding."""
    return {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}[dtype]


def act(z, name):
    """act(z) and act'(z) in the type of z (float64)."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "relu2":
        return z.clamp(min=0) ** 2, 2 * z.clamp(min=0)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def act_bound(z, dz, name):
    """Bounds of the fp32 errors of act and of act' at z known to within dz.

    act: its slope times dz plus its own arithmetic.  silu / gelu_tanh are z S(t): the exponential is
    off by at most 2 + 2 |t| ulp (its argument times log2 e is rounded), the quotient by 2, t by 4
    roundings: S by (6 + 8 |t|) (1 - S) + 6 ulp relative, the product by one more.  gelu: 1 + erf is off
    by 2 ulp of erf, the rounding of its argument (slope 2 / sqrt pi times |z|) and one rounding, all
    absolute below 6 ulp.  Slopes are bounded by 1.13, second slopes by 1.13 (relu2: 2 |z| and 2)."""
    a = z.abs()
    if name == "none":
        return dz, torch.zeros_like(z)
    if name == "relu":
        return dz, torch.zeros_like(z)
    if name == "relu2":
        return (2 * a + dz) * dz + 2 * U * (a + dz) ** 2, 2 * dz + 2 * U * (a + dz)
    if name == "gelu":
        own = 12 * U * a
        slope = 12 * U + 12 * U * (1 + a * a) * a * torch.exp(-z * z / 2)
    else:
        t = z if name == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        t1 = torch.ones_like(z) if name == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
        s = torch.sigmoid(t)
        rel = 2 * U * ((6 + 8 * t.abs()) * (1 - s) + 6)
        own = a * s * (rel + U)
        slope = s * rel + a * s * t1 * (2 * rel * (1 - s) + rel * s + 8 * U)
    tiny = 2.0 ** -120                        # S below e^-87 is flushed
    return 1.13 * dz + own + tiny, 1.13 * dz + slope + tiny


def pre_activation(acc, alpha, s, bias):
    """z and the bound of its fp32 error (two products, one sum)."""
    z0 = acc * alpha * s[:, None]
    z = z0 if bias is None else z0 + bias
    dz = 3.01 * U * z0.abs() + (0 if bias is None else U * z.abs()) + 2.0 ** -140
    return z, dz


def forward(acc, alpha, s, bias, name, gated, residual, dtype):
    """y in 64 bits and the largest error a kernel may have there."""
    z, dz = pre_activation(acc, alpha, s, bias)
    if gated:
        f, _ = act(z[:, ::2], name)
        df, _ = act_bound(z[:, ::2], dz[:, ::2], name)
        u, du = z[:, 1::2], dz[:, 1::2]
        y = f * u
        e = df * u.abs() + f.abs() * du + df * du
        e = e + U * (y.abs() + e)
    else:
        y, _ = act(z, name)
        e, _ = act_bound(z, dz, name)
    if residual is not None:
        y = y + residual
        e = e + U * (y.abs() + e)
    return y, e + half_step(dtype) * (y.abs() + e) + smallest(dtype)


def dz_bound(acc, alpha, s, bias, name, gated, dy):
    """dz in 64 bits and the bound of its fp32 error."""
    z, ez = pre_activation(acc, alpha, s, bias)
    if not gated:
        _, d = act(z, name)
        _, ed = act_bound(z, ez, name)
        return dy * d, dy.abs() * (ed + 2 * U * (d.abs() + ed))
    f, d = act(z[:, ::2], name)
    ef, ed = act_bound(z[:, ::2], ez[:, ::2], name)
    u, eu = z[:, 1::2], ez[:, 1::2]
    out, err = torch.empty_like(z), torch.empty_like(z)
    out[:, ::2], out[:, 1::2] = dy * u * d, dy * f
    err[:, ::2] = dy.abs() * ((u.abs() + eu) * (d.abs() + ed) * (1 + 3 * U) - u.abs() * d.abs())
    err[:, 1::2] = dy.abs() * ((f.abs() + ef) * (1 + 2 * U) - f.abs())
    return out, err + 2.0 ** -140


def gradients(T, acc, alpha, s, bias, name, gated, dy, dtype):
    """(dx, dalpha, dbias) in 64 bits and their bounds.

    dx: e = dz alpha (one more rounding), off by half a step of the fixed point: the token's largest
    |e| / 32639 (bf16), at most 2^-21 of it (fp16: it is 2^21 steps or more) or 2^-29 (fp32); the
    integer sums are exact, joining and scaling the digits takes at most 9 roundings, and the result is
    rounded once.  Column sums: M terms in chains of at most M / 16 + 17 additions, each term off by its
    own bound and 3 roundings."""
    dz, edz = dz_bound(acc, alpha, s, bias, name, gated, dy)
    e, ee = dz * alpha, edz * alpha.abs()
    ee = ee + U * (e.abs() + ee)
    big = (e.abs() + ee).amax(1, keepdim=True)
    step = big / 32639 if dtype is torch.bfloat16 else big * 2.0 ** (-21 if dtype is torch.float16 else -29)
    ee = ee + 0.51 * step + 2 * U * e.abs() * (dtype is torch.bfloat16) + 2.0 ** -114
    A = T.abs()
    dx = e @ T
    edx = ee @ A
    edx = edx + 10 * U * ((e.abs() + ee) @ A)
    edx = edx + half_step(dtype) * (dx.abs() + edx) + smallest(dtype)
    n = dy.shape[0] / 16 + 20
    q = acc.abs() * s[:, None]
    da, eda = (dz * acc * s[:, None]).sum(0), ((edz + n * U * (dz.abs() + edz)) * q).sum(0)
    db, edb = dz.sum(0), (edz + n * U * (dz.abs() + edz)).sum(0)
    return (dx, da, db), (edx, eda + 2.0 ** -140, edb + 2.0 ** -140)


def assert_within(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: got {float(got[at])}, "
                             f"want {float(want[at])}, bound {float(bound[at]):.3g}")


def transposed_words(T: np.ndarray) -> np.ndarray:
    """The transposed layout of T int8 [R][K], word by word from its description."""
    R, K = T.shape
    rt, kt = -(-R // 128), -(-K // 128)
    P = np.zeros((kt * 128, rt * 128), dtype=np.uint32)
    P[:K, :R] = np.where(T.T == 1, 1, np.where(T.T == -1, 2, 0))
    out = np.zeros((kt, rt, 2, 128, 4), dtype=np.uint32)
    for q in range(2):
        for i in range(4):
            for c in range(4):
                for e in range(4):
                    col = P.reshape(kt, 128, rt, 128)[:, :, :, 64 * q + 16 * i + 4 * c + e]
                    out[:, :, q, :, i] |= col.transpose(0, 2, 1) << np.uint32(2 * (c & 1) + 16 * (c >> 1) + 4 * e)
    return out.reshape(-1)
