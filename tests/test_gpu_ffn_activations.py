"""silu and gelu_tanh of fp32 tensors over their whole range, element by element: with alpha 0 the
pre-activation is the bias."""
import math

import pytest

import ffn_testlib as F
import sparse_bit_matmul_b200 as sbm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = F.U
N, K = 2050, 64


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _points(name):
    """Above the z where S(t) is flushed (t = -87)."""
    lo = -86.0 if name == "silu" else -10.0
    return torch.linspace(lo, 86.0, N, device="cuda")


def _t(z, name):
    """t of act(z) = z S(t), and t'."""
    if name == "silu":
        return z, torch.ones_like(z)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)


def _relative(t, name):
    """Relative error of S: e^-t is off by 2 ulp (4 half steps) and gelu_tanh's t by 4 roundings, both
    scaled by 1 - S; the sum rounds once, the reciprocal is off by 1 ulp."""
    return U * ((4 + (4 * t.abs() if name == "gelu_tanh" else 0)) * torch.sigmoid(-t) + 3) * 1.01


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 2, 20, 150])
def test_activation_of_fp32(name, M):
    z = _points(name)
    x, zero = torch.ones(M, K, device="cuda"), torch.zeros(N, device="cuda")
    w = torch.zeros(sbm.native_bytes(N, K), dtype=torch.uint8, device="cuda")
    y = sbm.linear_epilogue(x, w, zero, N, bias=z, act=name)
    z = z.double()
    t, _ = _t(z, name)
    want = z * torch.sigmoid(t)
    F.assert_within(y, want.expand(M, N), (want.abs() * (_relative(t, name) + U)).expand(M, N), name)
    # gated: the up projection is the bias alone too, 1
    bias = torch.stack([_points(name), torch.ones(N, device="cuda")], 1).reshape(-1)
    w = torch.zeros(sbm.native_bytes(2 * N, K), dtype=torch.uint8, device="cuda")
    assert torch.equal(sbm.gated(x, w, torch.zeros(2 * N, device="cuda"), N, bias=bias, act=name), y)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_slope_of_fp32(name):
    """dbias of one token is dy act'(z) = S + z S (1 - S) t': S off by r, the product z S by U more, 1 - S
    by S r and a rounding, t' by 3 roundings, the products and the sum by one each."""
    z = _points(name)
    zero = torch.zeros(N, device="cuda")
    acc, one = torch.zeros(1, N, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    _, _, db = sbm.linear_backward(torch.ones(1, N, device="cuda"), None, zero, K, acc, one, bias=z, act=name, want_dx=False)
    z = z.double()
    t, t1 = _t(z, name)
    s = torch.sigmoid(t)
    want = s + z * s * torch.sigmoid(-t) * t1
    r = _relative(t, name)
    bound = s * r + z.abs() * s * t1 * (torch.sigmoid(-t) * (r + 6 * U) + s * r + U) + U * want.abs()
    F.assert_within(db, want, 1.01 * bound, name)
