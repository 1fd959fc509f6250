"""The feed-forward operators on every launch the library has for them (ffn_cases.py), against their plain
64-bit forms within the bounds of ffn_testlib."""
import pytest

import ffn_testlib as F
import sparse_bit_matmul_b200 as sbm
from ffn_cases import ACTS, COLUMNS, FORWARD, GRADIENT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert sbm.last_device_status(reset=True) >= 0
    yield
    _weight.kept = None
    torch.cuda.synchronize()
    assert sbm.last_device_status() == 0


def _decode(codes, K):
    """T int8 [R][K] of canonical codes, on the device."""
    table = torch.zeros(32, 4, dtype=torch.int8)
    for c in range(32):
        signs = iter((c >> 2 & 1, c >> 3 & 1, c >> 4 & 1))
        for i in range(4):
            if i != c & 3:
                table[c, i] = -1 if next(signs) else 1
    word = torch.zeros(codes.shape[0], K // 32, dtype=torch.int64, device="cuda")
    for b in range(5):
        word |= codes.view(codes.shape[0], K // 32, 5)[:, :, b].long() << 8 * b
    code = torch.stack([word >> 5 * g & 31 for g in range(8)], 2).view(codes.shape[0], K // 4)
    return table.cuda()[code].view(codes.shape[0], K)


def _weight(R, K, gated):
    """Native and transposed layout, alpha, T int8 of a weight of random codes; the last one is kept."""
    key = (R, K, gated)
    if getattr(_weight, "kept", None) is None or _weight.kept[0] != key:
        _weight.kept = None
        g = torch.Generator(device="cuda").manual_seed(R + K)
        codes = torch.randint(0, 256, (R, K // 32 * 5), generator=g, device="cuda", dtype=torch.uint8)
        alpha = (torch.rand(R, generator=g, device="cuda") + 0.5) * (2.0 / K) ** 0.5
        if gated:
            gate, up = codes[::2].contiguous(), codes[1::2].contiguous()
            native, w_t = sbm.repack_gated(gate, up, R // 2, K), sbm.repack_gated_t(gate, up, R // 2, K)
        else:
            native, w_t = sbm.repack(codes, R, K), sbm.repack_t(codes, R, K)
        _weight.kept = key, (native, w_t, alpha, _decode(codes, K))
    return _weight.kept[1]


def _randn(*shape, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _exact_sums(x, T):
    """Sums and scales of the quantiser's rule; products of whole numbers below 2^24 are exact in fp32."""
    assert 127 * T.shape[1] < 2 ** 24
    x = x.float()
    s = x.abs().amax(1) / torch.full((x.shape[0],), 127.0, device="cuda")
    q = (x / s[:, None]).round().clamp(-127, 127)
    return torch.cat([q @ t.float().t() for t in T.split(8192)], 1).double(), s


def _name(case):
    path, kind, dt, act, *_, M, N, K = case
    return f"{kind}-{path.replace('/', '.')}-{dt}-{M}x{K}x{N}"


@pytest.mark.parametrize("case", sorted(FORWARD, key=lambda c: (c[1], c[8], c[9])), ids=_name)
def test_forward(case):
    _, kind, dt, act, bias, residual, keep, M, N, K = case
    gated, dtype = kind == "gated", F.DTYPES[dt]
    R = 2 * N if gated else N
    native, _, alpha, T = _weight(R, K, gated)
    x = _randn(M, K, seed=M, dtype=dtype)
    b = _randn(R, seed=1, std=0.3) if bias else None
    r = _randn(M, N, seed=2, dtype=dtype) if residual else None
    kept = {}
    if keep:
        kept = {"acc": torch.full((M, R), -7, dtype=torch.int32, device="cuda"), "out_s": torch.full((M,), -7.0, device="cuda")}
    buf = torch.full((M * N + 16,), 9.0, dtype=dtype, device="cuda")
    out = buf[:M * N].view(M, N)
    call = (lambda **k: sbm.gated(x, native, alpha, N, bias=b, act=act, **k)) if gated else \
        (lambda **k: sbm.linear_epilogue(x, native, alpha, N, bias=b, act=act, residual=k.pop("residual", r), **k))
    y = call(out=out, **kept)
    assert y is out and (buf[M * N:] == 9).all()
    acc, s = _exact_sums(x, T)
    if keep:
        assert torch.equal(kept["acc"].double(), acc) and torch.equal(kept["out_s"], s)
    want, bound = F.forward(acc, alpha.double(), s.double(), None if b is None else b.double(), act, gated,
                            None if r is None else r.double(), dtype)
    F.assert_within(y, want, bound, _name(case))
    first = y.clone()
    assert torch.equal(call(**kept), first)
    if residual:
        z = r.clone()
        assert call(out=z, residual=z, **kept) is z and torch.equal(z, first)


def _gradients(gated, dt, act, M, N, K, bias=True, unaligned=False, scales=True):
    dtype = F.DTYPES[dt]
    R = 2 * N if gated else N
    _, w_t, alpha, T = _weight(R, K, gated)
    acc, s = _exact_sums(_randn(M, K, seed=M), T)
    acc = acc.to(torch.int32)
    b = _randn(R, seed=1, std=0.3) if bias else None
    dy = _randn(M, N, seed=3, std=0.1, dtype=dtype)
    if unaligned:                                     # rows of 16 bytes from an odd element on
        dy = torch.empty(M * N + 1, dtype=dtype, device="cuda")[1:].view(M, N).copy_(dy)
    fn = sbm.gated_backward if gated else sbm.linear_backward
    buf = torch.full((M * K + 16,), 9.0, dtype=dtype, device="cuda")
    got = fn(dy, w_t, alpha, K, acc, s, bias=b, act=act, out=buf[:M * K].view(M, K))
    assert (buf[M * K:] == 9).all()
    want, bound = F.gradients(T.double(), acc.double(), alpha.double(), s.double(), None if b is None else b.double(), act,
                              gated, dy.double(), dtype)
    for name, g, w, e in zip(("dx", "dalpha", "dbias"), got, want, bound):
        F.assert_within(g, w, e, f"{name} {M}x{K}x{N} {dt} {act}")
    again = fn(dy, w_t, alpha, K, acc, s, bias=b, act=act)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    only = fn(dy, w_t, alpha, K, acc, s, bias=b, act=act, want_scales=False)
    assert torch.equal(only[0], got[0])
    only = fn(dy, w_t, alpha, K, acc, s, bias=b, act=act, want_dx=False)
    assert torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])


@pytest.mark.parametrize("case", sorted(GRADIENT, key=lambda c: (c[1], c[8], c[9])), ids=_name)
def test_gradient(case):
    _, kind, dt, act, bias, _, _, M, N, K = case
    _gradients(kind == "gated_grad", dt, act, M, N, K, bias)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", COLUMNS)
def test_column_sums_of_many_tokens(M, N, K, gated, dt):
    n = N // 2 if gated else N
    acts = ACTS[1:] if gated else ACTS
    for i in range(2):
        act = acts[(M + 3 * i + len(dt)) % len(acts)]
        _gradients(gated, dt, act, M, n, K, bias=i == 0)
    _gradients(gated, dt, acts[M % len(acts)], M, n - 1, K)       # rows of no 16-byte multiple
    if N % 8 == 0:
        _gradients(gated, dt, "silu", M, n, K, unaligned=True)


@pytest.mark.parametrize("act", ACTS)
def test_column_sums_of_every_activation(act):
    for dt in F.DTYPES:
        _gradients(False, dt, act, 1025, 2432, 32)
        _gradients(True, dt, act, 1025, 1217, 32)
