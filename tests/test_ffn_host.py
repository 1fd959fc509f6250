"""Feed-forward operators without a GPU: the plain forms' gradients against
differences, the layout's size, and the calls that are refused before
anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import ffn_testlib as F
import sparse_bit_matmul_b200 as sbm

FAKE = ctypes.c_void_p(1 << 20)
OFF4 = ctypes.c_void_p((1 << 20) + 4)
OFF1 = ctypes.c_void_p((1 << 20) + 1)
INVALID, SHAPE = sbm.ERR_INVALID_ARG, sbm.ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", F.ACTS)
def test_plain_gradients_against_differences(name, gated):
    g = torch.Generator().manual_seed(3)
    M, K, N = 3, 8, 4
    R = 2 * N if gated else N
    T = torch.randint(-1, 2, (R, K), generator=g).double()
    alpha = torch.rand(R, generator=g, dtype=torch.float64) + 0.5
    bias = torch.randn(R, generator=g, dtype=torch.float64)
    s = torch.rand(M, generator=g, dtype=torch.float64) + 0.1
    x = torch.randn(M, K, generator=g, dtype=torch.float64)        # dequantised activations q * s
    dy = torch.randn(M, N, generator=g, dtype=torch.float64)

    def value(x, alpha, bias):
        z = (x @ T.t()) * alpha + bias
        y = F.act(z[:, ::2], name)[0] * z[:, 1::2] if gated else F.act(z, name)[0]
        return (y * dy).sum()

    acc = (x / s[:, None]) @ T.t()
    (dx, da, db), _ = F.gradients(T, acc, alpha, s, bias, name, gated, dy, torch.float32)
    h = 1e-6
    for got, which in ((dx, 0), (da, 1), (db, 2)):
        args = [x, alpha, bias]
        for i in range(got.numel()):
            d = torch.zeros_like(args[which]).view(-1)
            d[i] = h
            d = d.view_as(args[which])
            plus = [a + d if k == which else a for k, a in enumerate(args)]
            minus = [a - d if k == which else a for k, a in enumerate(args)]
            want = (value(*plus) - value(*minus)) / (2 * h)
            assert abs(float(got.view(-1)[i] - want)) < 1e-6 * (1 + abs(float(want)))


def test_sizes(lib):
    assert sbm.transposed_bytes(4096, 4096) == 32 * 32 * 4096
    assert sbm.transposed_bytes(1, 32) == 4096
    assert sbm.transposed_bytes(129, 160) == 2 * 2 * 4096
    assert sbm.transposed_bytes(128, 33) == 0 and sbm.transposed_bytes(0, 32) == 0
    L = sbm.load()
    assert [L.sherry_grad_digits(d) for d in (0, 1, 2, 3, -1)] == [4, 2, 4, 0, 0]
    assert L.sherry_grad_work_bytes(1, 3, 17) >= 2 * 3 * 32 + 12
    for bad in ((3, 1, 1), (0, 0, 1), (0, 1, 0), (0, 1, 1 << 24), (0, 1 << 30, 1)):
        assert L.sherry_grad_work_bytes(*bad) == 0
    assert L.sherry_grad_work_bytes(0, 70000, 100000) > 2 ** 32     # no 32-bit wrap


def _linear(L, **kw):
    a = dict(x=FAKE, dt=1, w=FAKE, alpha=FAKE, bias=None, act=0, res=None, y=FAKE, acc=None, q=None, s=None, M=1, N=4,
             K=32)
    a.update(kw)
    return L.sherry_linear_epilogue(a["x"], a["dt"], a["w"], a["alpha"], a["bias"], a["act"], a["res"], a["y"],
                                    a["acc"], a["q"], a["s"], a["M"], a["N"], a["K"], None)


def _gated(L, **kw):
    a = dict(x=FAKE, dt=1, w=FAKE, alpha=FAKE, bias=None, act=0, h=FAKE, acc=None, q=None, s=None, M=1, N=4, K=32)
    a.update(kw)
    return L.sherry_gated(a["x"], a["dt"], a["w"], a["alpha"], a["bias"], a["act"], a["h"], a["acc"], a["q"], a["s"],
                          a["M"], a["N"], a["K"], None)


@pytest.mark.parametrize("call,out", [(_linear, "y"), (_gated, "h")])
def test_forward_refusals(call, out, lib):
    L = sbm.load()
    for kw in (dict(x=None), dict(w=None), dict(alpha=None), {out: None}, dict(dt=3), dict(dt=-1), dict(act=6),
               dict(act=-1), dict(M=0), dict(N=0), dict(K=0), dict(M=-1), dict(x=OFF4), dict(w=OFF4),
               dict(q=OFF4, s=FAKE), dict(q=FAKE), {out: OFF1}):
        assert call(L, **kw) == INVALID, kw
    for kw in (dict(K=33), dict(K=(1 << 24) + 32), dict(N=1 << 31), dict(M=1 << 31)):
        assert call(L, **kw) == SHAPE, kw
    if call is _linear:
        assert call(L, res=OFF1) == INVALID
    else:
        assert call(L, N=(1 << 30) + 1) == SHAPE


def _grad(L, fn, **kw):
    a = dict(dy=FAKE, dt=1, acc=FAKE, s=FAKE, wt=FAKE, alpha=FAKE, bias=None, act=3, dx=FAKE, da=FAKE, db=FAKE, work=FAKE,
             M=1, N=4, K=32)
    a.update(kw)
    return getattr(L, fn)(a["dy"], a["dt"], a["acc"], a["s"], a["wt"], a["alpha"], a["bias"], a["act"], a["dx"], a["da"],
                          a["db"], a["work"], a["M"], a["N"], a["K"], None)


@pytest.mark.parametrize("fn", ["sherry_linear_grad", "sherry_gated_grad"])
def test_gradient_refusals(fn, lib):
    L = sbm.load()
    for kw in (dict(dy=None), dict(alpha=None), dict(dx=None, da=None, db=None), dict(wt=None), dict(work=None),
               dict(acc=None), dict(s=None), dict(acc=None, act=0), dict(dt=3), dict(act=6), dict(M=0), dict(N=0),
               dict(K=0), dict(dy=OFF1), dict(dx=OFF1), dict(wt=OFF4), dict(work=OFF4), dict(acc=OFF4)):
        assert _grad(L, fn, **kw) == INVALID, kw
    for kw in (dict(K=33), dict(N=1 << 24), dict(M=1 << 30), dict(N=1 << 62)):
        assert _grad(L, fn, **kw) == SHAPE, kw
    if fn == "sherry_gated_grad":
        assert _grad(L, fn, acc=None, act=0, da=None) == INVALID
        assert _grad(L, fn, N=1 << 23) == SHAPE


def test_repack_and_quantiser_refusals(lib):
    L = sbm.load()
    assert L.sherry_repack_gated(FAKE, None, 4, 32, FAKE, None) == INVALID
    assert L.sherry_repack_gated(None, FAKE, 4, 32, FAKE, None) == INVALID
    assert L.sherry_repack_gated(FAKE, FAKE, 4, 32, OFF4, None) == INVALID
    assert L.sherry_repack_gated(FAKE, FAKE, 0, 32, FAKE, None) == INVALID
    assert L.sherry_repack_gated(FAKE, FAKE, 4, 40, FAKE, None) == SHAPE
    assert L.sherry_repack_gated(FAKE, FAKE, 1 << 62, 32, FAKE, None) == SHAPE
    assert L.sherry_repack_t(None, 4, 32, FAKE, None) == INVALID
    assert L.sherry_repack_t(FAKE, 4, 40, FAKE, None) == SHAPE
    assert L.sherry_repack_gated_t(FAKE, None, 4, 32, FAKE, None) == INVALID
    assert L.sherry_repack_gated_t(FAKE, FAKE, 1 << 62, 32, FAKE, None) == SHAPE
    assert L.sherry_quant_act_dt(FAKE, 3, 1, 32, FAKE, FAKE, None) == INVALID
    assert L.sherry_quant_act_dt(None, 1, 1, 32, FAKE, FAKE, None) == INVALID
    assert L.sherry_quant_act_dt(OFF4, 1, 1, 32, FAKE, FAKE, None) == INVALID
    assert L.sherry_quant_act_dt(FAKE, 2, 1, 33, FAKE, FAKE, None) == SHAPE


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(1, 32)
    w = torch.zeros(2560, dtype=torch.uint8)
    a = torch.zeros(4)
    with pytest.raises(ValueError):
        sbm.linear_epilogue(x, w, a, 4)
    with pytest.raises(ValueError):
        sbm.gated(x, w, torch.zeros(8), 4)
    with pytest.raises(ValueError):
        sbm.linear_backward(torch.zeros(1, 4), w, a, 32)


def test_block_shapes_must_chain(lib):
    W = np.ones((64, 32), dtype=np.float32)
    with pytest.raises(ValueError):
        sbm.GatedFFN.from_weights(W, W, np.ones((32, 32), dtype=np.float32))
    with pytest.raises(ValueError):
        sbm.GatedFFN.from_weights(W, W, np.ones((32, 64), dtype=np.float32), act="tanh")


def test_overlapping_buffers_are_refused(lib):
    L = sbm.load()
    at = lambda k: ctypes.c_void_p((1 << 20) + k)  # noqa: E731
    # bf16, M = 2, K = 32, N = 4: x 128 bytes, y and residual 16, acc 32
    far = at(1 << 16)
    kw = dict(M=2, N=4, K=32, x=at(0), y=far)
    for bad in (dict(kw, y=at(0)), dict(kw, y=at(126)), dict(kw, acc=at(64)), dict(kw, acc=far),
                dict(kw, res=at((1 << 16) + 2)), dict(kw, q=at(16), s=at(1 << 17)), dict(kw, res=at(1 << 18), acc=at(1 << 18)),
                dict(kw, w=far), dict(kw, w=at((1 << 16) - 2544)), dict(kw, bias=far), dict(kw, alpha=at((1 << 16) + 8)),
                dict(kw, s=far), dict(kw, q=at(1 << 17), s=at((1 << 17) + 60)), dict(kw, q=at(1 << 17), s=at(124))):
        assert _linear(L, **bad) == INVALID, bad
    kw = dict(M=2, N=4, K=32, dy=at(0), dx=far, acc=at(1 << 17), da=at(1 << 18), db=at(1 << 19), alpha=at(1 << 21),
              work=at(1 << 22), wt=at(1 << 23), s=at(1 << 24))
    for bad in (dict(kw, dx=at(0)), dict(kw, dx=at((1 << 17) + 16)), dict(kw, da=at(1 << 21)), dict(kw, db=at((1 << 18) + 8)),
                dict(kw, bias=at(1 << 18)), dict(kw, bias=at((1 << 19) - 4)), dict(kw, work=at(0)), dict(kw, work=far),
                dict(kw, wt=at((1 << 16) - 16)), dict(kw, da=at((1 << 24) + 4)), dict(kw, db=at(12)), dict(kw, da=at(1 << 22)),
                dict(kw, dx=at((1 << 21) - 120))):
        assert _grad(L, "sherry_linear_grad", **bad) == INVALID, bad
    assert L.sherry_quant_act_dt(at(0), 1, 2, 32, at(64), far, None) == INVALID
    assert L.sherry_quant_act_dt(at(0), 0, 2, 32, at(192), far, None) == INVALID
    assert L.sherry_quant_act_dt(at(0), 1, 2, 32, far, at((1 << 16) + 60), None) == INVALID
    assert L.sherry_repack_t(at(4090), 4, 32, at(0), None) == INVALID
    assert L.sherry_repack_gated(far, at(2544), 4, 32, at(0), None) == INVALID


def test_feed_forward_sources_never_allocate_or_synchronise():
    """The asynchronous entry points of ffn_cuda.cu and grad_cuda.cu call nothing that allocates, frees,
    clears or waits."""
    import os
    import re
    src = os.path.join(os.path.dirname(sbm.SO_PATH), "csrc")
    for name in ("ffn_cuda.cu", "grad_cuda.cu", "host_common.h", "tile_plan.h"):
        text = open(os.path.join(src, name)).read()
        assert not re.search(r"cuda(Malloc|Free|Memset|Memcpy|DeviceSynchronize|StreamSynchronize|EventSynchronize)", text), name
