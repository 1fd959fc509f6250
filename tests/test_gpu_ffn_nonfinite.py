"""NaN and Inf activations in the feed-forward operators: rows of NaN, and only those rows."""
import ctypes

import pytest

import sparse_bit_matmul_b200 as sbm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _weight(R, K):
    g = torch.Generator(device="cuda").manual_seed(R + K)
    return (torch.randint(0, 256, (sbm.native_bytes(R, K),), generator=g, device="cuda", dtype=torch.uint8),
            torch.rand(R, generator=g, device="cuda"))


# the fused launch of one token (row in registers, row streamed), the decode kernel, tensor cores (cluster,
# whole tiles, quantiser blocks of every width)
@pytest.mark.parametrize("M,K,N", [(1, 288, 136), (1, 65536, 24), (2, 4096, 136), (5, 3104, 72), (40, 288, 136),
                                   (700, 1056, 40)])
@pytest.mark.parametrize("dt", list(TYPES))
def test_nonfinite_tokens_give_rows_of_nan(M, K, N, dt):
    w, alpha = _weight(2 * N, K)
    wl, al = _weight(N, K)
    al[N // 2] = 0
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").to(TYPES[dt])
    res = torch.randn(M, N, generator=g, device="cuda").to(TYPES[dt])
    calls = [lambda x, s, act=act: sbm.linear_epilogue(x, wl, al, N, act=act, residual=res, out_s=s)
             for act in ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")]
    calls += [lambda x, s, act=act: sbm.gated(x, w, alpha, N, act=act, out_s=s) for act in ("relu", "silu", "gelu")]
    for value in (float("nan"), float("inf"), -float("inf")):
        for at in (0, K // 2 + 1, K - 1):
            bad = x.clone()
            row = M // 2
            bad[row, at] = value
            keep = [m for m in range(M) if m != row]
            for call in calls:
                s, s_bad = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
                y, y_bad = call(x, s), call(bad, s_bad)
                assert y_bad[row].isnan().all() and not y.isnan().any(), (value, at)
                assert s_bad[row].isnan() if value != value else s_bad[row].isinf()
                assert torch.equal(y_bad[keep], y[keep]) and torch.equal(s_bad[keep], s[keep])


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("M,K", [(1, 32), (3, 4096), (601, 1056), (2, 65568)])
def test_quantiser_keeps_them_in_the_scale(M, K, dt):
    x = torch.randn(M, K, generator=torch.Generator(device="cuda").manual_seed(K), device="cuda").to(TYPES[dt])
    x[M // 2, K // 3] = float("nan")
    x[M // 2, K // 5] = float("inf")
    if M > 2:
        x[0, K - 1] = -float("inf")
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    rc = sbm.load().sherry_quant_act_dt(x.data_ptr(), list(TYPES).index(dt), M, K, q.data_ptr(), s.data_ptr(),
                                        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == sbm.OK
    want = x.float().abs().amax(1) / torch.full((M,), 127.0, device="cuda")      # torch's maximum keeps NaN
    assert torch.equal(s.isnan(), want.isnan()) and torch.equal(s[~want.isnan()], want[~want.isnan()])
    assert bool(s[M // 2].isnan()) and (M <= 2 or bool(s[0].isinf()))
