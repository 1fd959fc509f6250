"""Feed-forward operators on the GPU against their plain 64-bit forms, within
the bounds of ffn_testlib; int32 sums and scales bit-exact against the oracle."""
import numpy as np
import pytest

import ffn_testlib as F
import oracle
import sparse_bit_matmul_b200 as sbm
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sbm.load()
    assert sbm.last_device_status(reset=True) >= 0
    yield
    torch.cuda.synchronize()
    assert sbm.last_device_status() == 0


_weights = {}


def weight(R, K, gated, seed=0):
    """Native layout, transposed layout, alpha [R] and T [R][K] (float64) of a seeded weight."""
    key = (R, K, gated, seed)
    if key not in _weights:
        if gated:
            parts = [synth.weights(21 + seed, 2 * R + b, R // 2, K) for b in range(2)]
            packed = [sbm.pack(W) for W in parts]
            dev = [torch.from_numpy(c).cuda() for c, _ in packed]
            native = sbm.repack_gated(dev[0], dev[1], R // 2, K)
            w_t = sbm.repack_gated_t(dev[0], dev[1], R // 2, K)
            alpha = np.stack([a for _, a in packed], 1).reshape(-1)
            T = np.stack([oracle.quantise(W)[0] for W in parts], 1).reshape(R, K)
        else:
            W = synth.weights(22 + seed, R, R, K)
            codes, alpha = sbm.pack(W)
            dev = torch.from_numpy(codes).cuda()
            native, w_t = sbm.repack(dev, R, K), sbm.repack_t(dev, R, K)
            T = oracle.quantise(W)[0]
        _weights[key] = native, w_t, torch.from_numpy(np.ascontiguousarray(alpha)).cuda(), \
            torch.from_numpy(np.ascontiguousarray(T)).cuda().double()
    return _weights[key]


def rand(*shape, seed=0, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def exact_sums(x, T):
    """int32 sums and scales by the oracle's quantiser and a 64-bit product."""
    q, s = oracle.quant_act(np.ascontiguousarray(x.float().cpu().numpy()))
    return torch.from_numpy(q).cuda().double() @ T.t(), torch.from_numpy(s).cuda(), torch.from_numpy(q).cuda()


def run_forward(gated, M, K, N, dt, act, bias, residual, x=None):
    R = 2 * N if gated else N
    native, _, alpha, T = weight(R, K, gated)
    dtype = F.DTYPES[dt]
    x = rand(M, K, seed=M, dtype=dtype) if x is None else x
    b = rand(R, seed=1, std=0.3) if bias else None
    r = rand(M, N, seed=2, dtype=dtype) if residual else None
    acc = torch.full((M, R), -7, dtype=torch.int32, device="cuda")
    s = torch.full((M,), -7.0, device="cuda")
    q = torch.full((M, K), -7, dtype=torch.int8, device="cuda")
    if gated:
        y = sbm.gated(x, native, alpha, N, bias=b, act=act, acc=acc, out_q=q, out_s=s)
        plain = sbm.gated(x, native, alpha, N, bias=b, act=act)
    else:
        y = sbm.linear_epilogue(x, native, alpha, N, bias=b, act=act, residual=r, acc=acc, out_q=q, out_s=s)
        plain = sbm.linear_epilogue(x, native, alpha, N, bias=b, act=act, residual=r)
    acc_o, s_o, q_o = exact_sums(x, T)
    assert torch.equal(q, q_o) and torch.equal(s, s_o)
    assert torch.equal(acc.double(), acc_o)
    want, bound = F.forward(acc_o, alpha.double(), s_o.double(), None if b is None else b.double(), act, gated,
                            None if r is None else r.double(), dtype)
    F.assert_within(y, want, bound, f"{'gated' if gated else 'linear'} {M}x{K}x{N} {dt} {act}")
    assert torch.equal(y, plain)              # with and without the kept sums: the same bits
    return y


# token counts of every path: fused decode, decode, each token tile, split and whole tiles
SHAPES = [(1, 32, 1), (1, 256, 128), (1, 4096, 1999), (2, 96, 5), (2, 1056, 130), (3, 160, 7), (16, 4096, 256),
          (17, 288, 129), (33, 1056, 130), (64, 512, 64), (65, 96, 1), (127, 4096, 300), (200, 2080, 1001),
          (1600, 160, 72), (1537, 288, 1003),
          # long batches of few chunks: two epilogue groups
          (2100, 64, 2504), (2100, 160, 2501)]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_epilogue(M, K, N, dt):
    run_forward(False, M, K, N, dt, "silu", True, True)
    run_forward(False, M, K, N, dt, "none", False, False)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_gated(M, K, N, dt):
    run_forward(True, M, K, N, dt, "silu", False, False)
    run_forward(True, M, K, N, dt, "gelu", True, False)


@pytest.mark.parametrize("act", F.ACTS)
@pytest.mark.parametrize("M", [1, 2, 5, 130])
def test_every_activation(M, act):
    for dt in F.DTYPES:
        run_forward(False, M, 288, 200, dt, act, True, False)
        run_forward(False, M, 288, 200, dt, act, False, True)
        run_forward(True, M, 288, 100, dt, act, True, False)


def test_plain_linear_equals_sherry_linear():
    """No bias, no activation, no residual, fp32: the same bits as the linear layer."""
    for M in (1, 2, 9, 100, 1600):
        native, _, alpha, _ = weight(300, 1056, False)
        x = rand(M, 1056, seed=M)
        assert torch.equal(sbm.linear_epilogue(x, native, alpha, 300), sbm.linear(x, native, alpha, 300))


@pytest.mark.parametrize("M", [1, 2, 40, 1600])
def test_residual_in_place_and_odd_alignment(M):
    native, _, alpha, _ = weight(136, 288, False)
    x = rand(M, 288, seed=3, dtype=torch.bfloat16)
    r = rand(M, 136, seed=4, dtype=torch.bfloat16)
    want = sbm.linear_epilogue(x, native, alpha, 136, residual=r, act="relu")
    y = r.clone()
    assert sbm.linear_epilogue(x, native, alpha, 136, residual=y, act="relu", out=y) is y
    assert torch.equal(y, want)
    # outputs and residual at element alignment only, with a guard around the output
    buf = torch.full((M * 136 + 3,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:1 + M * 136].view(M, 136)
    rb = torch.empty(M * 136 + 1, dtype=torch.bfloat16, device="cuda")
    rv = rb[1:].view(M, 136).copy_(r)
    sbm.linear_epilogue(x, native, alpha, 136, residual=rv, act="relu", out=out)
    assert torch.equal(out, want) and buf[0] == 9 and (buf[1 + M * 136:] == 9).all()


@pytest.mark.parametrize("M", [1, 2, 20, 130])
def test_zero_tokens_and_zero_scales(M):
    """All-zero tokens (scale 0) and an all-zero weight row (alpha 0)."""
    native, _, alpha, T = weight(256, 160, True)
    alpha = alpha.clone()
    alpha[4] = 0
    x = rand(M, 160, seed=5, dtype=torch.bfloat16)
    x[M // 2] = 0
    y = sbm.gated(x, native, alpha, 128)
    assert not y[M // 2].any() and not y[:, 2].any() and torch.isfinite(y).all()


def test_empty_batch():
    native, w_t, alpha, _ = weight(256, 160, True)
    x = torch.empty(0, 160, device="cuda")
    assert sbm.gated(x, native, alpha, 128).shape == (0, 128)
    dx, da, db = sbm.gated_backward(torch.empty(0, 128, device="cuda"), w_t, alpha, 160,
                                    torch.empty(0, 256, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda"))
    assert dx.shape == (0, 160) and not da.any() and not db.any() and da.shape == (256,)


def test_binding_refusals():
    native, w_t, alpha, _ = weight(128, 160, False)
    x = rand(4, 160)
    ok = dict(w_native=native, alpha=alpha, N=128)
    for bad in (dict(ok, N=127), dict(ok, N=300), dict(ok, alpha=alpha.double()), dict(ok, alpha=alpha.cpu()),
                dict(ok, bias=alpha[:64]), dict(ok, act="tanh"), dict(ok, residual=rand(4, 128, dtype=torch.bfloat16)),
                dict(ok, residual=rand(128, 4).t()), dict(ok, out=rand(3, 128)),
                dict(ok, acc=torch.empty(4, 128, device="cuda")), dict(ok, w_native=native[:-1])):
        with pytest.raises(ValueError):
            sbm.linear_epilogue(x, **bad)
    for bad in (x.double(), x[:, ::2], x[0], x.t(), rand(4, 168)[:, :160], rand(4, 100)):
        with pytest.raises(ValueError):
            sbm.linear_epilogue(bad, native, alpha, 128)
    with pytest.raises(sbm.SherryError):       # activations must start on 16 bytes
        sbm.linear_epilogue(rand(161)[1:].view(1, 160), native, alpha, 128)
    dy = rand(4, 128)
    with pytest.raises(ValueError):
        sbm.linear_backward(dy, w_t, alpha, 160)                       # no sums
    with pytest.raises(ValueError):
        sbm.linear_backward(dy, native, alpha, 160, want_scales=False)  # not the transposed layout
    with pytest.raises(ValueError):
        sbm.linear_backward(dy, w_t, alpha, 160, want_dx=False, want_scales=False)


def test_one_token_of_a_very_long_row():
    """K beyond what the decode kernel holds: quantiser and tensor cores."""
    run_forward(False, 1, 700000, 8, "bf16", "none", True, True)
    run_forward(True, 1, 700000, 4, "f32", "silu", False, False)


def test_scales_written_just_before():
    """alpha, bias and residual written by the kernel launched just before the call."""
    for M in (1, 2, 40):
        native, _, alpha, _ = weight(256, 288, True)
        x = rand(M, 288, seed=M, dtype=torch.bfloat16)
        a, b = torch.zeros_like(alpha), torch.zeros_like(alpha)
        want = sbm.gated(x, native, alpha * 3, 128, bias=alpha)
        torch.cuda.synchronize()
        for _ in range(20):
            a.copy_(alpha).mul_(3)
            b.copy_(alpha)
            y = sbm.gated(x, native, a, 128, bias=b)
            a.zero_()
            assert torch.equal(y, want)


def test_offsets_past_32_bits():
    """More than 2^31 outputs, sums and digits: the last tokens and rows are right."""
    M, K, N = 65537, 32, 33000
    native, w_t, alpha, T = weight(N, K, False)
    x = rand(M, K, seed=1, dtype=torch.bfloat16)
    s = torch.empty(M, device="cuda")
    acc = torch.empty(M, N, dtype=torch.int32, device="cuda")
    y = sbm.linear_epilogue(x, native, alpha, N, act="relu", acc=acc, out_s=s)
    assert y.numel() > 2 ** 31
    for at in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        acc_o, s_o, _ = exact_sums(x[at], T)
        assert torch.equal(acc[at].double(), acc_o) and torch.equal(s[at], s_o)
        want, bound = F.forward(acc_o, alpha.double(), s_o.double(), None, "relu", False, None, torch.bfloat16)
        F.assert_within(y[at], want, bound, "y")
    y.normal_(std=0.1, generator=torch.Generator(device="cuda").manual_seed(3))
    dx, da, db = sbm.linear_backward(y, w_t, alpha, K, acc, s, act="relu")
    for at in (slice(0, 3), slice(M - 3, M)):
        want, bound = F.gradients(T, acc[at].double(), alpha.double(), s[at].double(), None, "relu", False, y[at].double(),
                                  torch.bfloat16)
        F.assert_within(dx[at], want[0], bound[0], "dx")
    cols = torch.tensor([0, 1, N - 2, N - 1], device="cuda")
    want, bound = F.gradients(T[cols], acc[:, cols].double(), alpha[cols].double(), s.double(), None, "relu", False,
                              y[:, cols].double(), torch.bfloat16)
    F.assert_within(da[cols], want[1], bound[1], "dalpha")
    F.assert_within(db[cols], want[2], bound[2], "dbias")


def test_calls_allocate_nothing():
    """After the workspace is set aside, first calls of the C entry points leave the device's free memory
    as it was (buffers are the caller's)."""
    sbm.reserve_split()
    L = sbm.load()
    st = torch.cuda.current_stream().cuda_stream
    native, w_t, alpha, _ = weight(512, 1056, True)
    M, K, N = 90, 1056, 256
    x = rand(M, K, dtype=torch.bfloat16)
    h, dx = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    acc, q = torch.empty(M, 512, dtype=torch.int32, device="cuda"), torch.empty(M, K, dtype=torch.int8, device="cuda")
    s, da, db = torch.empty(M, device="cuda"), torch.empty(512, device="cuda"), torch.empty(512, device="cuda")
    work = torch.empty(L.sherry_grad_work_bytes(1, M, 512), dtype=torch.uint8, device="cuda")

    def both():
        assert L.sherry_gated(x.data_ptr(), 1, native.data_ptr(), alpha.data_ptr(), None, 3, h.data_ptr(), acc.data_ptr(),
                              q.data_ptr(), s.data_ptr(), M, N, K, st) == sbm.OK
        assert L.sherry_gated_grad(h.data_ptr(), 1, acc.data_ptr(), s.data_ptr(), w_t.data_ptr(), alpha.data_ptr(), None, 3,
                                   dx.data_ptr(), da.data_ptr(), db.data_ptr(), work.data_ptr(), M, N, K, st) == sbm.OK
        torch.cuda.synchronize()

    both()                                     # loads the kernels
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        both()
    assert torch.cuda.mem_get_info()[0] == free


# ------------------------------------------------------------------ layouts
@pytest.mark.parametrize("N,K", [(1, 32), (5, 96), (64, 128), (130, 160), (257, 1056)])
def test_layouts(N, K):
    Wg, Wu = synth.weights(31, 1, N, K), synth.weights(31, 2, N, K)
    (cg, _), (cu, _) = sbm.pack(Wg), sbm.pack(Wu)
    both = np.ascontiguousarray(np.stack([cg, cu], 1).reshape(2 * N, -1))
    dg, du, db = (torch.from_numpy(c).cuda() for c in (cg, cu, both))
    assert torch.equal(sbm.repack_gated(dg, du, N, K), sbm.repack(db, 2 * N, K))
    want = F.transposed_words(oracle.quantise(Wg)[0])
    assert np.array_equal(sbm.repack_t(dg, N, K).cpu().numpy().view(np.uint32), want)
    want = F.transposed_words(sbm.unpack(both, K))
    assert np.array_equal(sbm.repack_gated_t(dg, du, N, K).cpu().numpy().view(np.uint32), want)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 4096), (5, 16384), (2, 20000 // 32 * 32), (2, 32768 + 32), (1, 65568),
                                 # narrow blocks: many tokens
                                 (600, 32), (700, 1056), (601, 4128), (593, 14336), (600, 32800)])
def test_quantiser_of_any_type(M, K, dt):
    x = rand(M, K, seed=K, dtype=F.DTYPES[dt])
    x[M // 2] = 0
    if M > 3:
        x[0] *= 1e-7 if dt == "f16" else 1e-39            # subnormal
        x[1, ::2] = 0
        x[2, K // 3] = -65504.0
    q = torch.empty(M, K, dtype=torch.int8, device="cuda")
    s = torch.empty(M, device="cuda")
    L = sbm.load()
    rc = L.sherry_quant_act_dt(x.data_ptr(), {"f32": 0, "bf16": 1, "f16": 2}[dt], M, K, q.data_ptr(), s.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
    assert rc == sbm.OK
    q_o, s_o = oracle.quant_act(np.ascontiguousarray(x.float().cpu().numpy()))
    assert np.array_equal(q.cpu().numpy(), q_o) and np.array_equal(s.cpu().numpy(), s_o)


# ---------------------------------------------------------------- gradients
def run_backward(gated, M, K, N, dt, act, bias, dy=None):
    R = 2 * N if gated else N
    _, w_t, alpha, T = weight(R, K, gated)
    dtype = F.DTYPES[dt]
    acc, s, _ = exact_sums(rand(M, K, seed=M + 9), T)
    acc = acc.to(torch.int32)
    b = rand(R, seed=8, std=0.3) if bias else None
    dy = rand(M, N, seed=M + 10, std=0.1, dtype=dtype) if dy is None else dy
    fn = sbm.gated_backward if gated else sbm.linear_backward
    got = fn(dy, w_t, alpha, K, acc, s, bias=b, act=act)
    want, bound = F.gradients(T, acc.double(), alpha.double(), s.double(), None if b is None else b.double(), act, gated,
                              dy.double(), dtype)
    for name, g, w, e in zip(("dx", "dalpha", "dbias"), got, want, bound):
        F.assert_within(g, w, e, f"{name} {M}x{K}x{N} {dt} {act}")
    again = fn(dy, w_t, alpha, K, acc, s, bias=b, act=act)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    only = fn(dy, w_t, alpha, K, acc, s, bias=b, act=act, want_scales=False)
    assert torch.equal(only[0], got[0]) and only[1] is None
    only = fn(dy, w_t, alpha, K, acc, s, bias=b, act=act, want_dx=False)
    assert only[0] is None and torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])
    return got


GRAD_SHAPES = [(1, 32, 1), (1, 4096, 300), (2, 96, 5), (7, 160, 130), (9, 1056, 131), (17, 288, 64), (40, 4096, 257),
               (100, 512, 1001), (390, 2080, 129), (800, 160, 72), (600, 96, 2049),
               # few rows and many tokens: wide column blocks, two epilogue groups
               (1500, 4096, 100), (2049, 4064, 91)]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N", GRAD_SHAPES)
def test_linear_gradients(M, K, N, dt):
    run_backward(False, M, K, N, dt, "silu", True)
    run_backward(False, M, K, N, dt, "none", False)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N", GRAD_SHAPES)
def test_gated_gradients(M, K, N, dt):
    run_backward(True, M, K, N, dt, "silu", False)
    run_backward(True, M, K, N, dt, "gelu_tanh", True)


@pytest.mark.parametrize("act", F.ACTS)
def test_every_slope(act):
    for dt in F.DTYPES:
        run_backward(False, 6, 288, 200, dt, act, True)
        run_backward(True, 6, 288, 100, dt, act, True)


def test_gradient_of_more_rows_than_shared_memory_holds():
    run_backward(False, 3, 32, 52001, "bf16", "relu", False)
    run_backward(True, 2, 64, 26004, "f32", "silu", True)
    run_backward(False, 1, 32, 420003, "bf16", "silu", True)


def test_more_tokens_than_one_grid_dimension():
    run_forward(True, 70001, 32, 3, "bf16", "silu", False, False)
    run_backward(True, 70001, 32, 3, "bf16", "silu", False)
    run_backward(False, 131073, 32, 7, "f16", "gelu", True)


@pytest.mark.parametrize("M", [4, 5, 6, 10, 11, 79, 81, 400, 401])
def test_fp16_tokens_around_groups_of_five(M):
    """fp16 digit rows hold five tokens to 16; the output may end inside a group, at element alignment."""
    for K, R in ((160, 136), (256, 5000), (32, 20000)):
        dy = rand(M, R, seed=M, dtype=torch.float16)
        dx = run_backward(False, M, K, R, "f16", "none", False, dy=dy)[0]
        _, w_t, alpha, _ = weight(R, K, False)
        buf = torch.full((M * K + 3,), 9.0, dtype=torch.float16, device="cuda")
        out = buf[1:1 + M * K].view(M, K)
        sbm.linear_backward(dy, w_t, alpha, K, want_scales=False, out=out)
        assert torch.equal(out, dx) and buf[0] == 9 and (buf[1 + M * K:] == 9).all()
        # whatever the buffer of the digits held before
        work = torch.full((sbm.load().sherry_grad_work_bytes(2, M, R),), 0x7f, dtype=torch.uint8, device="cuda")
        rc = sbm.load().sherry_linear_grad(dy.data_ptr(), 2, None, None, w_t.data_ptr(), alpha.data_ptr(), None, 0,
                                           out.data_ptr(), None, None, work.data_ptr(), M, R, K,
                                           torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(out, dx)


def test_linear_gradient_without_sums():
    """act none and no dalpha: dx needs neither sums nor scales."""
    _, w_t, alpha, T = weight(130, 160, False)
    dy = rand(5, 130, dtype=torch.bfloat16)
    dx, da, db = sbm.linear_backward(dy, w_t, alpha, 160, want_scales=False)
    full = sbm.linear_backward(dy, w_t, alpha, 160, torch.ones(5, 130, dtype=torch.int32, device="cuda"),
                               torch.ones(5, device="cuda"))
    assert da is None and db is None and torch.equal(dx, full[0])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_gradient_extremes(dt):
    """Zero tokens give zero rows; a NaN or an Inf only its own row, as NaN; tiny and huge tokens keep
    their precision beside each other."""
    dtype = F.DTYPES[dt]
    _, w_t, alpha, T = weight(256, 160, False)
    M = 8
    dy = rand(M, 256, seed=40).double()
    top = 1e4 if dt == "f16" else 1e30
    low = 1e-3 if dt == "f16" else 1e-30
    dy[1] = 0
    dy[2] *= top / 8
    dy[3] *= low
    dy[6, 1:] *= 2.0 ** -6
    dy = dy.to(dtype)
    acc = torch.zeros(M, 256, dtype=torch.int32, device="cuda")
    s = torch.ones(M, device="cuda")
    clean = sbm.linear_backward(dy, w_t, alpha, 160, acc, s)
    want, bound = F.gradients(T, acc.double(), alpha.double(), s.double(), None, "none", False, dy.double(), dtype)
    F.assert_within(clean[0], want[0], bound[0], "dx")
    assert not clean[0][1].any()
    dy[4, 7] = float("nan")
    dy[5, 200] = float("inf")
    dx = sbm.linear_backward(dy, w_t, alpha, 160, want_scales=False)[0]
    assert dx[4].isnan().all() and dx[5].isnan().all()
    rest = [0, 1, 2, 3, 6, 7]
    assert torch.equal(dx[rest], clean[0][rest])


def test_subnormal_gradients():
    """Tokens below 2^-100 (and fp32 subnormals) stay finite and small."""
    _, w_t, alpha, _ = weight(256, 160, False)
    one = torch.ones_like(alpha)
    dy = torch.zeros(3, 256, device="cuda")
    dy[0, 3], dy[1, 5], dy[2, 9] = 1e-38, 1e-42, 3e38
    for dtype in (torch.float32, torch.bfloat16):
        dx = sbm.linear_backward(dy.to(dtype), w_t, one, 160, want_scales=False)[0]
        assert torch.isfinite(dx).all()
        assert dx[0].abs().max() <= 2e-38 and dx[1].abs().max() <= 2e-38 and dx[2].abs().max() > 2.9e38


# ------------------------------------------------------- streams and graphs
def test_other_stream_and_captured_graph():
    """Forward and backward on a side stream and replayed from a graph: the bits of eager calls."""
    gn, gt, ga, _ = weight(512, 288, True)
    dn, dt_, da, _ = weight(288, 256, False)
    M = 70
    x = rand(M, 288, dtype=torch.bfloat16)
    dy = rand(M, 288, seed=1, std=0.1, dtype=torch.bfloat16)

    def step():
        acc, s = torch.empty(M, 512, dtype=torch.int32, device="cuda"), torch.empty(M, device="cuda")
        acc_d, s_d = torch.empty(M, 288, dtype=torch.int32, device="cuda"), torch.empty(M, device="cuda")
        h = sbm.gated(x, gn, ga, 256, acc=acc, out_s=s)
        y = sbm.linear_epilogue(h, dn, da, 288, residual=x, acc=acc_d, out_s=s_d)
        dh, dad, _ = sbm.linear_backward(dy, dt_, da, 256, acc_d, s_d)
        dx, dag, _ = sbm.gated_backward(dh, gt, ga, 288, acc, s)
        return y, dx, dad, dag

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (5, 6):
        x.copy_(rand(M, 288, seed=seed, dtype=torch.bfloat16))
        dy.copy_(rand(M, 288, seed=seed + 20, std=0.1, dtype=torch.bfloat16))
        g.replay()
        again = [t.clone() for t in out]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, step()))


def test_block_is_its_operators():
    """GatedFFN forward and backward: the operators chained, and PackedLinear's own path."""
    K, H, M = 160, 256, 33
    Wg, Wu, Wd = synth.weights(41, 1, H, K), synth.weights(41, 2, H, K), synth.weights(41, 3, K, H)
    block = sbm.GatedFFN.from_weights(Wg, Wu, Wd, trainable=True)
    x = rand(M, K, dtype=torch.bfloat16)
    y, kept = block.forward(x, residual=x, keep=True)
    assert torch.equal(y, block.forward(x, residual=x))
    Tg, Tu = oracle.quantise(Wg)[0], oracle.quantise(Wu)[0]
    T = torch.from_numpy(np.stack([Tg, Tu], 1).reshape(2 * H, K)).cuda().double()
    Td = torch.from_numpy(oracle.quantise(Wd)[0]).cuda().double()
    acc, s, acc_d, s_d = kept
    acc_o, s_o, _ = exact_sums(x, T)
    assert torch.equal(acc.double(), acc_o) and torch.equal(s, s_o)
    h = sbm.gated(x, block.w_native, block.alpha, H)
    want, bound = F.forward(acc_o, block.alpha.double(), s_o.double(), None, "silu", True, None, torch.bfloat16)
    F.assert_within(h, want, bound, "h")
    acc_do, s_do, _ = exact_sums(h, Td)
    assert torch.equal(acc_d.double(), acc_do) and torch.equal(s_d, s_do)
    want, bound = F.forward(acc_do, block.down.alpha.double(), s_do.double(), None, "none", False, x.double(),
                            torch.bfloat16)
    F.assert_within(y, want, bound, "y")
    assert torch.equal(y, block.down.forward(h, residual=x))
    dy = rand(M, K, seed=3, std=0.1, dtype=torch.bfloat16)
    dx, da, dad = block.backward(dy, kept)
    dh, dad2, _ = sbm.linear_backward(dy, block.down.w_t, block.down.alpha, H, acc_d, s_d)
    want, bound = F.gradients(T, acc_o, block.alpha.double(), s_o.double(), None, "silu", True, dh.double(),
                              torch.bfloat16)
    F.assert_within(dx, want[0], bound[0], "dx")
    F.assert_within(da, want[1], bound[1], "dalpha")
    assert torch.equal(dad, dad2)
