"""Precision of the feed-forward gradients within one token: small terms beside
a large one."""
import numpy as np
import pytest

import ffn_testlib as F
import oracle
import sparse_bit_matmul_b200 as sbm
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# steps of the fixed point below a token's largest |dz alpha|
STEPS = {"f32": 2.0 ** 29, "bf16": 2.0 ** 22 - 1, "f16": 2.0 ** 22 - 1}


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    N, K = 4096, 2048
    W = synth.weights(51, 1, N, K)
    codes, alpha = sbm.pack(W)
    w_t = sbm.repack_t(torch.from_numpy(codes).cuda(), N, K)
    return w_t, torch.from_numpy(alpha).cuda(), torch.from_numpy(np.ascontiguousarray(oracle.quantise(W)[0])).cuda().double()


@pytest.mark.parametrize("dt,ratio", [("bf16", 300), ("bf16", 1000), ("bf16", 10000), ("f16", 300), ("f16", 1000),
                                      ("f32", 30), ("f32", 300)])
@pytest.mark.parametrize("M", [1, 6, 41])
def test_small_terms_beside_a_large_one(layer, dt, ratio, M):
    """Columns of dx whose weight is 0 in the large term's row hold the small terms alone.

    Their error in the 2-norm.  With v = w + d the value before the last rounding R: R(v) - w = (R(v) - v) + d,
    and v is at most |d| further from the nearest number of the type than w is, so |error| <= |R(w) - w| +
    2 |d|.  d: fp32 arithmetic (e is rounded once, the digits joined and scaled with at most 9 roundings,
    the fixed point's scale with 2: 12 half steps, all taken as of one sign) and the fixed point, whose
    rounding is uniform in half a step, each term's on its own: step / sqrt(12) times the root of the
    number of terms, a tenth more for the sample (about 500 columns)."""
    w_t, alpha, T = layer
    N, K = T.shape
    dtype = F.DTYPES[dt]
    g = torch.Generator(device="cuda").manual_seed(ratio + M)
    e = torch.randn(M, N, generator=g, device="cuda", dtype=torch.float64)
    at = [(37 * m + 11) % N for m in range(M)]
    for m in range(M):
        e[m, at[m]] = ratio
    dy = (e / alpha.double() * 2.0 ** -10).to(dtype)
    dx = sbm.linear_backward(dy, w_t, alpha, K, want_scales=False)[0].double()
    e = dy.double() * alpha.double()
    want = e @ T
    for m in range(M):
        quiet = T[at[m]] == 0
        w = want[m, quiet]
        err = (dx[m, quiet] - w).norm()
        rounding = (w.to(dtype).double() - w).norm()
        terms = T[:, quiet].abs().sum(0)
        fixed = 1.1 * (e[m].abs().max() / STEPS[dt]) / 12 ** 0.5 * terms.sum().sqrt()
        bound = rounding + 2 * (fixed + 12 * F.U * w.norm())
        assert err <= bound, (m, float(err / w.norm()), float(bound / w.norm()))
        if dt != "f32" and ratio <= 1000:
            assert fixed <= rounding
