"""Buffers of the feed-forward calls: what is refused before anything is launched."""
import ctypes

import sparse_bit_matmul_b200 as sbm

INVALID = sbm.ERR_INVALID_ARG


def at(k):
    return ctypes.c_void_p((1 << 20) + k)


def test_bad_workspaces_are_refused(lib):
    L = sbm.load()
    far = 1 << 24
    fwd = [at(0), 1, at(far), at(2 * far), None, 0]
    shape = [2, 4, 32, None]
    for split, size in ((at(3 * far + 8), 64), (at(4 * far), 64), (at(0), 64), (at(112), 64), (at(2 * far - 48), 64)):
        assert L.sherry_linear_epilogue_ws(*fwd, None, at(4 * far), None, None, None, split, size, *shape) == INVALID
        assert L.sherry_gated_ws(*fwd, at(4 * far), None, None, None, split, size, *shape) == INVALID
    grad = [at(0), 1, at(far), at(2 * far), at(3 * far), at(4 * far), None, 3, at(5 * far), at(6 * far), at(7 * far), at(8 * far)]
    for split, size in ((at(9 * far + 8), 64), (at(0), 64), (at(far), 64), (at(5 * far + 16), 64), (at(6 * far), 16),
                        (at(8 * far + 32), 16)):
        assert L.sherry_linear_grad_ws(*grad, split, size, *shape) == INVALID
        assert L.sherry_gated_grad_ws(*grad, split, size, *shape) == INVALID


def test_size_queries_of_bad_arguments(lib):
    L = sbm.load()
    for bad in ((3, 0, 0, 0, 8, 8, 32), (0, 6, 0, 0, 8, 8, 32), (0, 0, 0, 0, 0, 8, 32), (0, 0, 0, 0, 8, 0, 32),
                (0, 0, 0, 0, 8, 8, 33)):
        assert L.sherry_linear_split_bytes(*bad) == 0
        assert L.sherry_gated_split_bytes(*bad[:2], *bad[3:]) == 0
    assert L.sherry_gated_split_bytes(0, 0, 0, 8, 1 << 62, 32) == 0
    for bad in ((3, 8, 8, 32), (0, 0, 8, 32), (0, 8, 1 << 24, 32), (0, 8, 8, 33), (0, 1 << 30, 8, 32)):
        assert L.sherry_grad_split_bytes(*bad) == 0


def test_arrays_off_their_elements_are_refused(lib):
    """fp32 and int32 arguments at addresses that are no multiple of 4."""
    L = sbm.load()
    far = 1 << 24
    for off in (1, 2, 3):
        for i in (3, 4, 8, 10):                       # alpha, bias, acc, x_scale
            a = [at(0), 1, at(far), at(2 * far), at(3 * far), 0, None, at(4 * far), at(5 * far), at(6 * far), at(7 * far)]
            a[i] = at((20 + i) * far + off)
            assert L.sherry_linear_epilogue(*a, 2, 4, 32, None) == INVALID, (i, off)
            del a[6]
            assert L.sherry_gated(*a, 2, 4, 32, None) == INVALID, (i, off)
        for i in (3, 5, 6, 9, 10):                    # x_scale, alpha, bias, dalpha, dbias
            a = [at(0), 1, at(far), at(2 * far), at(3 * far), at(4 * far), at(5 * far), 3, at(6 * far), at(7 * far),
                 at(8 * far), at(9 * far)]
            a[i] = at((20 + i) * far + off)
            assert L.sherry_linear_grad(*a, 2, 4, 32, None) == INVALID, (i, off)
            assert L.sherry_gated_grad(*a, 2, 4, 32, None) == INVALID, (i, off)
        assert L.sherry_quant_act_dt(at(0), 1, 2, 32, at(far), at(2 * far + off), None) == INVALID
