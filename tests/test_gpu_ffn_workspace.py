"""Workspace of the feed-forward operators on the GPU: calls without enough of it."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A process of its own, with nothing reserved: shapes whose launch splits tiles
# through the workspace are refused and leave every output as it was.
UNRESERVED = r"""
import torch
import sparse_bit_matmul_b200 as sbm

L = sbm.load()
st = torch.cuda.current_stream().cuda_stream
seven = lambda *shape, dtype=torch.float32: torch.full(shape, 7, dtype=dtype, device="cuda")
refused = 0
bf16 = torch.bfloat16
for M, N, K in ((3, 128, 10240), (17, 768, 30688), (65, 3200, 20480)):
    w, alpha = torch.zeros(sbm.native_bytes(N, K), dtype=torch.uint8, device="cuda"), torch.ones(N, device="cuda")
    x, y = torch.ones(M, K, device="cuda", dtype=bf16), seven(M, N, dtype=bf16)
    q, s, acc = seven(M, K, dtype=torch.int8), seven(M), seven(M, N, dtype=torch.int32)
    rc = L.sherry_linear_epilogue(x.data_ptr(), 1, w.data_ptr(), alpha.data_ptr(), None, 0, None, y.data_ptr(), acc.data_ptr(),
                                  q.data_ptr(), s.data_ptr(), M, N, K, st)
    outs = [y, q, s, acc]
    torch.cuda.synchronize()
    if rc == sbm.ERR_WORKSPACE:
        refused += 1
        assert all(bool((t == 7).all()) for t in outs), ("linear", M)
    else:
        assert rc == sbm.OK
for M, R, C in ((3, 10240, 128), (16, 20480, 512), (31, 10240, 2176)):
    w_t, alpha = torch.zeros(sbm.transposed_bytes(R, C), dtype=torch.uint8, device="cuda"), torch.ones(R, device="cuda")
    dy, acc, s = torch.ones(M, R, device="cuda", dtype=bf16), seven(M, R, dtype=torch.int32), torch.ones(M, device="cuda")
    dx, da, db = seven(M, C, dtype=bf16), seven(R), seven(R)
    work = seven(L.sherry_grad_work_bytes(1, M, R), dtype=torch.uint8)
    rc = L.sherry_linear_grad(dy.data_ptr(), 1, acc.data_ptr(), s.data_ptr(), w_t.data_ptr(), alpha.data_ptr(), None, 0,
                              dx.data_ptr(), da.data_ptr(), db.data_ptr(), work.data_ptr(), M, R, C, st)
    torch.cuda.synchronize()
    if rc == sbm.ERR_WORKSPACE:
        refused += 1
        assert all(bool((t == 7).all()) for t in (dx, da, db, work)), ("gradient", M)
    else:
        assert rc == sbm.OK
assert refused >= 4, refused
print("ok", refused)
"""


def test_refused_for_want_of_workspace_leaves_outputs_alone():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    res = subprocess.run([sys.executable, "-c", UNRESERVED], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert res.stdout.startswith("ok")


# (gated, M, K, N): launches that split tiles of 16, 32, 64, 128 and 192 tokens through the workspace
SPLIT_FORWARD = [(False, 3, 10240, 128), (True, 17, 51200, 256), (False, 33, 20480, 2432), (False, 65, 20480, 3200),
                 (True, 1537, 30688, 256), (False, 1537, 14336, 2176)]
# (M, K, R) of gradients
SPLIT_GRADIENT = [(3, 128, 10240), (16, 512, 20480), (31, 2176, 10240), (33, 3200, 20480), (1000, 256, 30688)]


def _bytes(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8)


def _forward_call(sbm, gated, M, K, N, seed):
    """A call on seeded inputs (any bytes are codes), as a closure that returns its outputs."""
    R = 2 * N if gated else N
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    w, alpha = _bytes(sbm.native_bytes(R, K), seed), torch.rand(R, generator=g, device="cuda")
    res = None if gated else torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)

    def call():
        acc, s = torch.empty(M, R, dtype=torch.int32, device="cuda"), torch.empty(M, device="cuda")
        y = sbm.gated(x, w, alpha, N, acc=acc, out_s=s) if gated else \
            sbm.linear_epilogue(x, w, alpha, N, residual=res, acc=acc, out_s=s)
        return y, acc, s
    return call


def _gradient_call(sbm, M, K, R, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w_t = _bytes(sbm.transposed_bytes(R, K), seed)               # a field of 3 is read as 0
    alpha = torch.rand(R, generator=g, device="cuda")
    dy = torch.randn(M, R, generator=g, device="cuda").to(torch.float16)
    return lambda: (sbm.linear_backward(dy, w_t, alpha, K, want_scales=False)[0],)


@pytest.mark.parametrize("which", ["forward", "gradient"])
def test_calls_on_streams_without_order(which):
    """Calls that split tiles, on two streams with no event between them, replayed from two graphs on two
    streams, and beside eager calls: the bits of one call at a time."""
    import sparse_bit_matmul_b200 as sbm
    shapes = SPLIT_FORWARD if which == "forward" else SPLIT_GRADIENT
    make = _forward_call if which == "forward" else _gradient_call
    for shape in shapes:
        calls = [make(sbm, *shape, seed) for seed in (1, 2)]
        want = [[t.clone() for t in c()] for c in calls]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        graphs, outs = [], []
        for c in calls:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(c())
            graphs.append(g)
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(8):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[i].append(calls[i]())
        torch.cuda.synchronize()
        for i in range(2):
            for r in got[i]:
                assert all(torch.equal(a, b) for a, b in zip(r, want[i])), (which, shape)
        for _ in range(4):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    graphs[i].replay()
            eager = calls[0]()                            # on a third stream
            torch.cuda.synchronize()
            for r, w in ((outs[0], want[0]), (outs[1], want[1]), (eager, want[0])):
                assert all(torch.equal(a, b) for a, b in zip(r, w)), (which, shape)


def test_the_callers_workspace_and_the_reserved_one():
    """The same bits through a workspace of any contents and through the reserved one; nothing is written
    behind the caller's; too few bytes are refused with the outputs left alone."""
    import sparse_bit_matmul_b200 as sbm
    L = sbm.load()
    sbm.reserve_split()
    st = torch.cuda.current_stream().cuda_stream
    for M, K, N in ((3, 10240, 128), (33, 20480, 2432), (65, 20480, 3200)):
        w, alpha = _bytes(sbm.native_bytes(N, K), M), torch.rand(N, device="cuda")
        x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
        y, q, s = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16), torch.zeros(M, K, dtype=torch.int8, device="cuda"), \
            torch.zeros(M, device="cuda")
        need = L.sherry_linear_split_bytes(1, 0, 0, 0, M, N, K)
        assert need > 0 and need % 16 == 0
        args = [x.data_ptr(), 1, w.data_ptr(), alpha.data_ptr(), None, 0, None, y.data_ptr(), None, q.data_ptr(), s.data_ptr()]
        split = _bytes(need + 64, 5)
        guard = split[need:].clone()
        assert L.sherry_linear_epilogue_ws(*args, split.data_ptr(), need - 16, M, N, K, st) == sbm.ERR_WORKSPACE
        torch.cuda.synchronize()
        assert not y.any() and not q.any() and not s.any()
        got = []
        for _ in range(3):
            assert L.sherry_linear_epilogue_ws(*args, split.data_ptr(), need, M, N, K, st) == sbm.OK
            got.append(y.clone())
            split[:need] = _bytes(need, 6)
            assert L.sherry_linear_epilogue(*args, M, N, K, st) == sbm.OK
            got.append(y.clone())
        want = sbm.linear_epilogue(x, w, alpha, N)
        assert all(torch.equal(t, want) for t in got) and torch.equal(split[need:], guard)
    for M, K, R in ((3, 128, 10240), (31, 2176, 10240)):
        w_t, alpha = _bytes(sbm.transposed_bytes(R, K), M), torch.rand(R, device="cuda")
        dy, dx = torch.randn(M, R, device="cuda").to(torch.float16), torch.zeros(M, K, device="cuda", dtype=torch.float16)
        work = _bytes(L.sherry_grad_work_bytes(2, M, R), 7)
        need = L.sherry_grad_split_bytes(2, M, R, K)
        assert need > 0 and need % 16 == 0
        args = [dy.data_ptr(), 2, None, None, w_t.data_ptr(), alpha.data_ptr(), None, 0, dx.data_ptr(), None, None,
                work.data_ptr()]
        split = _bytes(need + 64, 8)
        guard = split[need:].clone()
        assert L.sherry_linear_grad_ws(*args, split.data_ptr(), need - 16, M, R, K, st) == sbm.ERR_WORKSPACE
        torch.cuda.synchronize()
        assert not dx.any()
        want = sbm.linear_backward(dy, w_t, alpha, K, want_scales=False)[0]
        for _ in range(2):
            assert L.sherry_linear_grad_ws(*args, split.data_ptr(), need, M, R, K, st) == sbm.OK
            assert torch.equal(dx, want)
            split[:need] = _bytes(need, 9)
            assert L.sherry_linear_grad(*args, M, R, K, st) == sbm.OK
            assert torch.equal(dx, want)
        assert torch.equal(split[need:], guard)
