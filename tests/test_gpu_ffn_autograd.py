"""The feed-forward operators and autograd: no silent loss of history, and the operators inside an
autograd function."""
import pytest

import sparse_bit_matmul_b200 as sbm
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _block():
    return sbm.GatedFFN.from_weights(synth.weights(61, 1, 128, 96), synth.weights(61, 2, 128, 96),
                                     synth.weights(61, 3, 96, 128), trainable=True)


@pytest.mark.parametrize("M", [1, 5])
def test_arguments_that_require_gradients_are_refused(M):
    b = _block()
    x, need = torch.randn(M, 96, device="cuda"), dict(device="cuda", requires_grad=True)
    calls = [lambda: sbm.gated(torch.randn(M, 96, **need), b.w_native, b.alpha, 128),
             lambda: sbm.gated(x, b.w_native, b.alpha.clone().requires_grad_(), 128),
             lambda: sbm.gated(x, b.w_native, b.alpha, 128, bias=torch.zeros(256, **need)),
             lambda: sbm.linear_epilogue(x, b.w_native, b.alpha.clone().requires_grad_(), 256),
             lambda: sbm.linear_epilogue(x, b.w_native, b.alpha, 256, residual=torch.zeros(M, 256, **need)),
             lambda: sbm.linear_backward(torch.randn(M, 256, **need), b.w_t, b.alpha, 96, want_scales=False),
             lambda: b.forward(torch.randn(M, 96, **need))]
    for call in calls:
        with pytest.raises(ValueError, match="autograd"):
            call()
        with torch.no_grad():
            call()


def test_block_inside_an_autograd_function():
    """What the refusal names: the block as a function, its gradients those of GatedFFN.backward."""
    b = _block()

    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, alpha):
            y, ctx.kept = b.forward(x, residual=x, keep=True)
            return y

        @staticmethod
        def backward(ctx, dy):
            dx, dalpha, _ = b.backward(dy, ctx.kept)
            return dx + dy, dalpha

    x = torch.randn(7, 96, device="cuda", requires_grad=True)
    alpha = b.alpha.clone().requires_grad_()
    y = Block.apply(x, alpha)
    dy = torch.randn_like(y)
    y.backward(dy)
    with torch.no_grad():
        want, kept = b.forward(x, residual=x, keep=True)
        dx, dalpha, _ = b.backward(dy, kept)
    assert torch.equal(y, want) and torch.equal(x.grad, dx + dy) and torch.equal(alpha.grad, dalpha)


def test_scales_alone_need_no_transposed_gate():
    """backward(want_dx=False) reads the down projection's transposed weight only."""
    b = _block()
    lean = sbm.GatedFFN(b.w_native, b.alpha, b.down, b.F, b.K, b.act)
    x, dy = torch.randn(9, 96, device="cuda"), torch.randn(9, 96, device="cuda")
    _, kept = lean.forward(x, keep=True)
    want = b.backward(dy, kept)
    got = lean.backward(dy, kept, want_dx=False)
    assert got[0] is None and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    with pytest.raises(ValueError, match="trainable"):
        lean.backward(dy, kept)
