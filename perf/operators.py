"""Operators of a feed-forward layer over packed 3:4 ternary weights, and their gradients.

linear        y = act(((acc * alpha) * s) + bias) + residual, acc = q(x) . T^T
gated         h = act(g) * u, (g, u) the two projections of x, rows 2n and 2n + 1 of one weight
linear_grad   dx, dalpha, dbias of `linear` (the gradient of the residual is dy itself)
gated_grad    dx, dalpha, dbias of `gated`

q(x), s is the per-token absmax / 127 int8 quantiser of the library (IEEE fp32
division, ties to even); gradients pass through it as through the identity:
with z = acc * alpha * s + bias and dz the gradient of z,
  dx[m][k] = sum_n dz[m][n] alpha[n] T[n][k],  dalpha[n] = sum_m dz[m][n] acc[m][n] s[m],
  dbias[n] = sum_m dz[m][n].
Tensors of a call (x, y, residual, dy, dx) are float32, bfloat16 or float16;
alpha, bias and their gradients are float32, acc is int32.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")


# ---------------------------------------------------------------------- cases
def _case(name, op, M, K, N, dtype, act, bias=False, residual=False, save=False):
    return {"name": name, "op": op, "M": M, "K": K, "N": N, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "save": save}


def listed():
    return [
        # one new token of a feed-forward block while a model answers
        _case("gated_token", "gated", 1, 4096, 14336, "bf16", "silu"),
        # a ragged handful of sequences, small model, biases, sums kept for a backward pass
        _case("gated_ragged_f16", "gated", 7, 2080, 5001, "f16", "gelu_tanh", bias=True, save=True),
        # a prompt
        _case("gated_prompt", "gated", 2048, 4096, 14336, "bf16", "silu"),
        # the same token leaves the block: down projection onto the residual stream
        _case("linear_token", "linear", 1, 14336, 4096, "bf16", "none", residual=True),
        # a batch of answers, one token each
        _case("linear_batch", "linear", 16, 4096, 4096, "f32", "gelu", bias=True, residual=True),
        # training step of odd size that keeps its sums
        _case("linear_ragged_f16", "linear", 333, 1056, 1999, "f16", "relu2", bias=True, save=True),
        # the prompt's down projection
        _case("linear_prompt", "linear", 2048, 14336, 4096, "bf16", "none", residual=True),
        # backward passes: one short sequence in full precision, ragged half precision, long ones
        _case("linear_grad_f32", "linear_grad", 129, 4096, 4096, "f32", "silu", bias=True),
        _case("linear_grad_long", "linear_grad", 2048, 14336, 4096, "bf16", "none"),
        _case("gated_grad_small", "gated_grad", 5, 1024, 2816, "bf16", "silu"),
        _case("gated_grad_ragged", "gated_grad", 300, 2080, 5001, "f16", "gelu", bias=True),
        _case("gated_grad_long", "gated_grad", 2048, 4096, 14336, "bf16", "silu"),
    ]


def draw(rng):
    """Sizes over the whole range, spread over their logarithms; at most the work of the largest listed case."""
    op = rng.choice(("linear", "gated", "linear_grad", "gated_grad"))
    two = 2 if op.startswith("gated") else 1
    lg = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    K = 32 * lg(8, 448)
    N = lg(64, 14336)
    M = max(1, min(lg(1, 4096), 2048 * 4096 * 2 * 14336 // (two * N * K)))
    grad = op.endswith("grad")
    act = rng.choice(ACTS[1:] if two == 2 else ACTS)
    return {"op": op, "M": M, "K": K, "N": N, "dtype": rng.choice(("f32", "bf16", "f16")), "act": act,
            "bias": rng.random() < 0.5, "residual": op == "linear" and rng.random() < 0.5,
            "save": not grad and rng.random() < 0.25}


# --------------------------------------------------------------------- inputs
def _ternarise(W):
    """W [R][K] -> T int8 [R][K] (the smallest |w| of each group of 4 is 0, lowest index on ties), codes int32
    [R][K/4] (zero position | signs of the kept three << 2), alpha [R] (mean kept |w|)."""
    R, K = W.shape
    g = W.view(R, K // 4, 4)
    z = g.abs().argmin(2, keepdim=True)
    T = torch.where(g < 0, -1, 1).to(torch.int8).scatter_(2, z, 0)
    kept = torch.arange(3, device=W.device).view(1, 1, 3)
    kept = kept + (kept >= z).to(kept.dtype)
    neg = (g < 0).gather(2, kept).to(torch.int32)
    codes = z[..., 0].to(torch.int32) | neg[..., 0] << 2 | neg[..., 1] << 3 | neg[..., 2] << 4
    alpha = (g.abs() * T.abs()).sum((1, 2), dtype=torch.float64) / (0.75 * K)
    return T.view(R, K), codes, alpha.float()


def _native(codes):
    """The layout of sherry_repack: per (128 rows, 128 k) five planes of 32-bit words, plane j rotated by 8 j rows."""
    R, G = codes.shape
    tiles, chunks = -(-R // 128), -(-G // 32)
    c = torch.zeros(tiles * 128, chunks * 32, dtype=torch.int64, device=codes.device)
    c[:R, :G] = codes
    c = c.view(tiles, 128, chunks, 32)
    planes = []
    for j in range(5):
        w = torch.zeros(tiles, 128, chunks, dtype=torch.int64, device=codes.device)
        for k in range(32):
            at = 5 * k - 32 * j
            if -5 < at < 32:
                w |= (c[..., k] << at if at >= 0 else c[..., k] >> -at) & 0xFFFFFFFF
        planes.append(torch.roll(w, 8 * j, 1))
    w = torch.stack(planes, 1).permute(0, 3, 1, 2)           # [tile][chunk][plane][position]
    return _bytes(w)


def _transposed(T):
    """The layout of sherry_repack_t: T^T at 2 bits a weight (0, 1 for +1, 2 for -1), per (128 k, 128 rows) block
    [piece 2][k 128][word 4]; word i of piece q covers rows 64 q + 16 i .. + 15 of the block, the weight of row
    4 c + e among them at bit 2 (c & 1) + 16 (c >> 1) + 4 e."""
    R, K = T.shape
    rt, kt = -(-R // 128), -(-K // 128)
    v = torch.zeros(kt * 128, rt * 128, dtype=torch.int64, device=T.device)
    v[:K, :R] = (T.t() == 1).long() + 2 * (T.t() == -1).long()
    v = v.view(kt, 128, rt, 2, 4, 4, 4)                      # [k tile][k][row tile][piece][word][cell][element]
    c = torch.arange(4, device=T.device).view(4, 1)
    e = torch.arange(4, device=T.device).view(1, 4)
    w = (v << (2 * (c & 1) + 16 * (c >> 1) + 4 * e)).sum((5, 6))
    return _bytes(w.permute(0, 2, 3, 1, 4))                  # [k tile][row tile][piece][k][word]


def _bytes(w):
    """64-bit integers holding 32-bit words -> their little-endian bytes."""
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous()
    return w.view(-1).view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, M, K, N, dt = case["op"], case["M"], case["K"], case["N"], DT[case["dtype"]]
    gated, grad = op.startswith("gated"), op.endswith("grad")
    R = 2 * N if gated else N

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    T, codes, alpha = _ternarise(normal(R, K, std=0.02))
    s = {"op": op, "N": N, "K": K, "act": case["act"], "T": T, "alpha": alpha, "save": case["save"],
         "bias": normal(R, std=0.1) if case["bias"] else None}
    x = normal(M, K).to(dt)
    if grad:
        q, scale = _quantise(x)
        s |= {"acc": (q @ T.float().t()).to(torch.int32), "scale": scale, "w_t": _transposed(T),
              "dy": normal(M, N, std=0.01).to(dt)}
    else:
        s |= {"x": x, "w": _native(codes), "residual": normal(M, N).to(dt) if case["residual"] else None}
    return s


# ---------------------------------------------------------------- plain forms
def _quantise(x):
    x = x.float()
    a = x.abs().amax(1)
    s = a / torch.full_like(a, 127.0)                        # tensor by tensor: an IEEE division
    q = (x / torch.where(a == 0, 1.0, s)[:, None]).round().clamp(-127, 127)
    return q, s


def _act(z, act):
    if act == "none":
        return z
    if act in ("relu", "relu2"):
        r = torch.where(z > 0, z, 0.0)
        return r * r if act == "relu2" else r
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    t = (2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)
    return 0.5 * z * (1 + torch.tanh(t))


def _slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return torch.where(z > 0, 2 * z, 0.0)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain(s):
    T, alpha, bias, act = s["T"].float(), s["alpha"], s["bias"], s["act"]
    gated = s["op"].startswith("gated")
    if "dy" in s:
        acc, scale = s["acc"].float(), s["scale"]
    else:
        q, scale = _quantise(s["x"])
        acc = q @ T.t()                                      # whole numbers below 2^24: exact
    z = acc * alpha * scale[:, None]
    if bias is not None:
        z = z + bias
    if "dy" not in s:
        y = _act(z[:, 0::2], act) * z[:, 1::2] if gated else _act(z, act)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        y = y.to(s["x"].dtype)
        return [y, acc.to(torch.int32), scale] if s["save"] else [y]
    dy = s["dy"].float()
    if gated:
        up = dy * _act(z[:, 0::2], act)
        dz = torch.stack((dy * z[:, 1::2] * _slope(z[:, 0::2], act), up), 2).view_as(z)
    else:
        dz = dy * _slope(z, act)
    dx = ((dz * alpha) @ T).to(s["dy"].dtype)
    return [dx, (dz * acc * scale[:, None]).sum(0), dz.sum(0)]


def _own(s):
    import sparse_bit_matmul_b200 as sbm

    op, N, K, alpha, bias, act = s["op"], s["N"], s["K"], s["alpha"], s["bias"], s["act"]
    if op.endswith("grad"):
        call = sbm.gated_backward if op == "gated_grad" else sbm.linear_backward
        return list(call(s["dy"], s["w_t"], alpha, K, s["acc"], s["scale"], bias=bias, act=act))
    x = s["x"]
    kept = {}
    if s["save"]:
        kept = {"acc": torch.empty(x.shape[0], alpha.numel(), dtype=torch.int32, device=x.device),
                "out_s": torch.empty(x.shape[0], dtype=torch.float32, device=x.device)}
    if op == "gated":
        y = sbm.gated(x, s["w"], alpha, N, bias=bias, act=act, **kept)
    else:
        y = sbm.linear_epilogue(x, s["w"], alpha, N, bias=bias, act=act, residual=s["residual"], **kept)
    return [y, kept["acc"], kept["out_s"]] if s["save"] else [y]


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------- work
def work(case):
    op, M, K, N = case["op"], case["M"], case["K"], case["N"]
    e = 4 if case["dtype"] == "f32" else 2
    R = 2 * N if op.startswith("gated") else N
    shared = R * K * 5 / 32 + 4 * R * (2 if case["bias"] else 1)     # 1.25 bit a weight, alpha, bias
    if op.endswith("grad"):
        # the sums are needed for the slopes and for dalpha
        moved = shared + e * M * (N + K) + 4 * M * R + 4 * M + 8 * R
    else:
        moved = shared + e * M * (K + N * (2 if case["residual"] else 1)) + (4 * M * R + 4 * M if case["save"] else 0)
    return {"bytes": moved, "flops": 2.0 * M * R * K}


# ---------------------------------------------------------------------- exact
def exact(case, seed):
    """The definition in 64 bits: the quantiser's own fp32 rounding of the scale and of x / s is part of the operator
    (a quotient of two fp32 numbers rounded from 64 bits is the IEEE fp32 quotient), all else is unrounded."""
    s = prepare(case, seed)
    if "dy" not in s:
        x = s["x"].double()
        scale = (x.abs().max(1).values / 127).float().double()
        ratio = x / scale.clamp(min=1e-300).unsqueeze(1)
        q = torch.round(ratio.float()).double()
        q[scale == 0] = 0
        q = torch.minimum(torch.maximum(q, q.new_tensor(-127)), q.new_tensor(127))
        acc = torch.einsum("mk,nk->mn", q, s["T"].double())
    else:
        acc, scale = s["acc"].double(), s["scale"].double()
    a, act = s["alpha"].double(), s["act"]
    pre = torch.einsum("mn,n,m->mn", acc, a, scale)
    if s["bias"] is not None:
        pre += s["bias"].double()

    def f(v):
        """act(v) and its derivative."""
        if act == "none":
            return v, torch.ones_like(v)
        if act == "relu":
            return v.clamp(min=0), (v > 0).double()
        if act == "relu2":
            return v.clamp(min=0) ** 2, 2 * v.clamp(min=0)
        if act == "silu":
            p = torch.sigmoid(v)
            return v * p, p + v * p * (1 - p)
        if act == "gelu":
            p = torch.special.ndtr(v)
            return v * p, p + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        r = math.sqrt(8 / math.pi)                           # (1 + tanh(t)) / 2 = sigmoid(2 t)
        p = torch.sigmoid(r * v * (1 + 0.044715 * v * v))
        return v * p, p + v * p * (1 - p) * r * (1 + 0.134145 * v * v)

    gated = s["op"].startswith("gated")
    if "dy" not in s:
        y = f(pre[:, ::2])[0] * pre[:, 1::2] if gated else f(pre)[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return [y, None, scale] if s["save"] else [y]
    dy = s["dy"].double()
    if gated:
        v, d = f(pre[:, ::2])
        dpre = torch.empty_like(pre)
        dpre[:, ::2] = dy * pre[:, 1::2] * d
        dpre[:, 1::2] = dy * v
    else:
        dpre = dy * f(pre)[1]
    dx = torch.einsum("mn,nk->mk", dpre * a, s["T"].double())
    return [dx, torch.einsum("mn,mn,m->n", dpre, acc, scale), dpre.sum(0)]
