"""Python binding of libsherry_b200 (include/sherry.h): the Sherry 3:4 ternary
matmul on B200.

Only argument marshalling lives here: every step of the path runs in the C /
CUDA library.  Host functions take numpy arrays; device functions take torch
CUDA tensors (torch supplies device memory and the current stream).  There
is no fallback: if the library is missing or a call fails, an exception is
raised.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
SO_PATH = os.path.join(HERE, "libsherry_b200.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_SHAPE, ERR_NONFINITE, ERR_CUDA, ERR_DEVICE, ERR_WORKSPACE = range(7)

# every entry point declared in include/sherry.h
ABI_SYMBOLS = (
    "sherry_status_string", "sherry_version", "sherry_packed_bytes", "sherry_native_bytes",
    "sherry_pack", "sherry_unpack", "sherry_repack", "sherry_quant_act", "sherry_gemm",
    "sherry_gemm_acc", "sherry_gemm_tc", "sherry_gemm_gemv", "sherry_gemm_simt", "sherry_gemm_noalloc",
    "sherry_gemm_decode", "sherry_linear", "sherry_linear_ex", "sherry_last_device_status",
    "sherry_workspace_bytes", "sherry_reserve", "sherry_selftest_wait",
    "sherry_w4a8_packed_bytes", "sherry_w4a8_native_bytes", "sherry_w4a8_pack", "sherry_w4a8_unpack",
    "sherry_w4a8_repack", "sherry_w4a8_gemm", "sherry_w4a8_gemm_acc", "sherry_w4a8_gemm_tc",
    "sherry_w4a8_gemm_gemv",
    "sherry_quant_act_dt", "sherry_repack_gated", "sherry_linear_epilogue", "sherry_gated",
    "sherry_transposed_bytes", "sherry_repack_t", "sherry_repack_gated_t", "sherry_grad_work_bytes",
    "sherry_grad_digits", "sherry_linear_grad", "sherry_gated_grad",
    "sherry_linear_split_bytes", "sherry_linear_epilogue_ws", "sherry_gated_split_bytes", "sherry_gated_ws",
    "sherry_grad_split_bytes", "sherry_linear_grad_ws", "sherry_gated_grad_ws",
)

_lib = None


class SherryError(RuntimeError):
    def __init__(self, what: str, status: int):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def load() -> ctypes.CDLL:
    """Load the in-tree library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(SO_PATH):
        raise ImportError(f"{SO_PATH} is missing: run `python -m sparse_bit_matmul_b200.build`")
    L = ctypes.CDLL(SO_PATH)
    i64, vp, c_int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    L.sherry_status_string.argtypes = [c_int]
    L.sherry_status_string.restype = ctypes.c_char_p
    L.sherry_version.restype = c_int
    L.sherry_packed_bytes.argtypes = [i64, i64]
    L.sherry_packed_bytes.restype = ctypes.c_size_t
    L.sherry_native_bytes.argtypes = [i64, i64]
    L.sherry_native_bytes.restype = ctypes.c_size_t
    L.sherry_pack.argtypes = [vp, i64, i64, vp, vp]
    L.sherry_unpack.argtypes = [vp, i64, i64, vp]
    L.sherry_repack.argtypes = [vp, i64, i64, vp, vp]
    L.sherry_quant_act.argtypes = [vp, i64, i64, vp, vp, vp]
    L.sherry_gemm.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_gemm_acc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_gemm_simt.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_gemm_tc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_gemm_gemv.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_gemm_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_gemm_decode.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_linear.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_linear_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_last_device_status.argtypes = [c_int]
    L.sherry_workspace_bytes.argtypes = [i64, i64]
    L.sherry_workspace_bytes.restype = ctypes.c_size_t
    L.sherry_reserve.argtypes = [i64, i64]
    L.sherry_selftest_wait.argtypes = [ctypes.c_uint64, vp]
    L.sherry_w4a8_packed_bytes.argtypes = [i64, i64]
    L.sherry_w4a8_packed_bytes.restype = ctypes.c_size_t
    L.sherry_w4a8_native_bytes.argtypes = [i64, i64]
    L.sherry_w4a8_native_bytes.restype = ctypes.c_size_t
    L.sherry_w4a8_pack.argtypes = [vp, i64, i64, vp, vp]
    L.sherry_w4a8_unpack.argtypes = [vp, i64, i64, vp]
    L.sherry_w4a8_repack.argtypes = [vp, i64, i64, vp, vp]
    L.sherry_w4a8_gemm.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_w4a8_gemm_acc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_w4a8_gemm_tc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_w4a8_gemm_gemv.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_quant_act_dt.argtypes = [vp, c_int, i64, i64, vp, vp, vp]
    L.sherry_repack_gated.argtypes = [vp, vp, i64, i64, vp, vp]
    L.sherry_linear_epilogue.argtypes = [vp, c_int, vp, vp, vp, c_int, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_gated.argtypes = [vp, c_int, vp, vp, vp, c_int, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_transposed_bytes.argtypes = [i64, i64]
    L.sherry_transposed_bytes.restype = ctypes.c_size_t
    L.sherry_repack_t.argtypes = [vp, i64, i64, vp, vp]
    L.sherry_repack_gated_t.argtypes = [vp, vp, i64, i64, vp, vp]
    L.sherry_grad_work_bytes.argtypes = [c_int, i64, i64]
    L.sherry_grad_work_bytes.restype = ctypes.c_size_t
    L.sherry_grad_digits.argtypes = [c_int]
    grad = [vp, c_int, vp, vp, vp, vp, vp, c_int, vp, vp, vp, vp, i64, i64, i64, vp]
    L.sherry_linear_grad.argtypes = grad
    L.sherry_gated_grad.argtypes = grad
    split = [vp, ctypes.c_size_t, i64, i64, i64, vp]           # in place of M, N, K, stream
    for name in ("sherry_linear_epilogue", "sherry_gated", "sherry_linear_grad", "sherry_gated_grad"):
        getattr(L, name + "_ws").argtypes = getattr(L, name).argtypes[:-4] + split
    L.sherry_linear_split_bytes.argtypes = [c_int, c_int, c_int, c_int, i64, i64, i64]
    L.sherry_gated_split_bytes.argtypes = [c_int, c_int, c_int, i64, i64, i64]
    L.sherry_grad_split_bytes.argtypes = [c_int, i64, i64, i64]
    for name in ("linear", "gated", "grad"):
        getattr(L, f"sherry_{name}_split_bytes").restype = ctypes.c_size_t
    for name in ABI_SYMBOLS:
        getattr(L, name).restype = getattr(L, name).restype or c_int
    _lib = L
    return L


def status_string(status: int) -> str:
    return load().sherry_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != OK:
        raise SherryError(what, rc)


def _np_ptr(a: np.ndarray):
    assert a.flags["C_CONTIGUOUS"]
    return a.ctypes.data


def _dptr(t):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "device arguments must be contiguous CUDA tensors"
    return t.data_ptr()


def _stream(t):
    import torch
    return torch.cuda.current_stream(t.device).cuda_stream


# ----------------------------------------------------------------- host side
def packed_bytes(N: int, K: int) -> int:
    return int(load().sherry_packed_bytes(N, K))


def native_bytes(N: int, K: int) -> int:
    return int(load().sherry_native_bytes(N, K))


def pack(W: np.ndarray):
    """fp32 W [N][K] -> (canonical codes uint8 [N][5K/32], alpha fp32 [N])."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    codes = np.empty((N, K // 32 * 5), dtype=np.uint8)
    alpha = np.empty(N, dtype=np.float32)
    _check(load().sherry_pack(_np_ptr(W), N, K, _np_ptr(codes), _np_ptr(alpha)), "sherry_pack")
    return codes, alpha


def unpack(codes: np.ndarray, K: int) -> np.ndarray:
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    N = codes.shape[0]
    T = np.empty((N, K), dtype=np.int8)
    _check(load().sherry_unpack(_np_ptr(codes), N, K, _np_ptr(T)), "sherry_unpack")
    return T


# --------------------------------------------------------------- device side
_reserved = {}          # device index -> (max_M, max_K) reserved through this binding


def workspace_bytes(max_M: int, max_K: int) -> int:
    """Device bytes sherry_reserve(max_M, max_K) sets aside on the current device."""
    return int(load().sherry_workspace_bytes(max_M, max_K))


def reserve(max_M: int, max_K: int, device=None):
    """sherry_reserve on `device` (default: the current CUDA device): host-
    synchronous; sets aside the workspace of every later call with
    M <= max_M and K <= max_K.  Call it before capturing CUDA graphs."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    m0, k0 = _reserved.get(idx, (0, 0))
    m1, k1 = max(m0, int(max_M)), max(k0, int(max_K))
    if (m1, k1) != (m0, k0):
        with torch.cuda.device(idx):
            _check(load().sherry_reserve(m1, k1), "sherry_reserve")
        _reserved[idx] = (m1, k1)


def _ensure_workspace(t, M: int, K: int):
    # the asynchronous entry points never allocate: the binding reserves (host,
    # synchronous) the first time a call needs more than was set aside
    m0, k0 = _reserved.get(t.device.index, (0, 0))
    if M > m0 or K > k0:
        reserve(M, K, t.device)


def repack(codes_dev, N: int, K: int, out=None):
    """Canonical codes on the device -> kernel-native layout (uint8 tensor)."""
    import torch
    if out is None:
        out = torch.empty(native_bytes(N, K), dtype=torch.uint8, device=codes_dev.device)
    _check(load().sherry_repack(_dptr(codes_dev), N, K, _dptr(out), _stream(codes_dev)), "sherry_repack")
    return out


def quant_act(x, out_q=None, out_s=None):
    """fp32 x [M][K] -> (int8 [M][K], fp32 scale [M])."""
    import torch
    M, K = x.shape
    q = out_q if out_q is not None else torch.empty((M, K), dtype=torch.int8, device=x.device)
    s = out_s if out_s is not None else torch.empty(M, dtype=torch.float32, device=x.device)
    _check(load().sherry_quant_act(_dptr(x), M, K, _dptr(q), _dptr(s), _stream(x)), "sherry_quant_act")
    return q, s


GEMV_MAX_M = 4      # SHERRY_GEMV_MAX_M
DECODE_MAX_M = 8    # SHERRY_DECODE_MAX_M
GEMM_DECODE_AUTO_MAX_M = 2   # SHERRY_GEMM_DECODE_AUTO_MAX_M
LINEAR_FUSED_MAX_M = 1   # SHERRY_LINEAR_FUSED_MAX_M


def gemm(x_i8, x_scale, w_native, alpha, N: int, out=None, acc=None, want_y: bool = True,
         kernel: str = "auto"):
    """y fp32 [M][N] (and optionally exact int32 acc) from int8 activations and
    kernel-native codes.  kernel: "auto" (sherry_gemm: the decode kernel
    for M <= 2, tensor cores above), "decode", "tc", "gemv" (the page's
    table lookup), "simt" (comparison kernel) or "noalloc"."""
    import torch
    M, K = x_i8.shape
    y = None
    if want_y:
        y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=x_i8.device)
    L = load()
    if kernel != "noalloc":
        _ensure_workspace(x_i8, M, K)
    args = (_dptr(x_i8), _dptr(x_scale), _dptr(w_native), _dptr(alpha), _dptr(y), _dptr(acc), M, N, K,
            _stream(x_i8))
    if kernel == "auto":
        if acc is None:
            rc = L.sherry_gemm(args[0], args[1], args[2], args[3], args[4], M, N, K, args[-1])
        else:
            rc = L.sherry_gemm_acc(*args)
    elif kernel == "tc":
        rc = L.sherry_gemm_tc(*args)
    elif kernel == "gemv":
        rc = L.sherry_gemm_gemv(*args)
    elif kernel == "simt":
        rc = L.sherry_gemm_simt(*args)
    elif kernel == "noalloc":
        rc = L.sherry_gemm_noalloc(*args)
    elif kernel == "decode":
        rc = L.sherry_gemm_decode(*args)
    else:
        raise ValueError(kernel)
    _check(rc, f"sherry_gemm[{kernel}]")
    return y


def linear(x, w_native, alpha, N: int, out=None, acc=None, out_q=None, out_s=None, want_y: bool = True):
    """y fp32 [M][N] straight from fp32 activations x [M][K] (sherry_linear:
    quantiser + GEMM, one launch for M = 1).  Optional acc int32 [M][N] and
    out_q int8 [M][K] / out_s fp32 [M] receive the exact accumulators and the
    quantised activations."""
    import torch
    M, K = x.shape
    y = None
    if want_y:
        y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=x.device)
    L = load()
    _ensure_workspace(x, M, K)
    if acc is None and out_q is None and out_s is None:
        rc = L.sherry_linear(_dptr(x), _dptr(w_native), _dptr(alpha), _dptr(y), M, N, K, _stream(x))
    else:
        rc = L.sherry_linear_ex(_dptr(x), _dptr(w_native), _dptr(alpha), _dptr(y), _dptr(acc), _dptr(out_q),
                                _dptr(out_s), M, N, K, _stream(x))
    _check(rc, "sherry_linear")
    return y


def last_device_status(reset: bool = False) -> int:
    return int(load().sherry_last_device_status(1 if reset else 0))


DEV_TIMEOUT_SELFTEST = 0x107   # device status code of sherry_selftest_wait


def selftest_wait(limit_ns: int, stream=None):
    """sherry_selftest_wait on the current stream: a bounded wait that runs out."""
    import torch
    st = torch.cuda.current_stream().cuda_stream if stream is None else stream
    _check(load().sherry_selftest_wait(int(limit_ns), st), "sherry_selftest_wait")


# --------------------------------------------------- feed-forward operators
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4, "gelu_tanh": 5}   # sherry_act
_torch = _is_grad_enabled = None
_DTYPES = {}            # torch dtype -> sherry_dtype, filled on first use
_split_reserved = set()  # devices whose split-K workspace covers every call
SPLIT_MAX_M = 1536      # from this many tokens on the split-K workspace no longer grows


def _types():
    """Imports torch on first use: sherry_dtype by torch dtype."""
    global _torch, _is_grad_enabled
    if _torch is None:
        import torch
        load()
        _is_grad_enabled = torch.is_grad_enabled
        _DTYPES.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
        _torch = torch
    return _DTYPES


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _refuse(name: str, t, want: str):
    raise ValueError(f"{name}: want a contiguous CUDA tensor {want}, got {t.dtype} {tuple(t.shape)} on {t.device}, "
                     f"strides {tuple(t.stride())}")


def _ptr(t, name: str, dtype, shape, idx: int):
    """Data pointer of a tensor argument of the given type and shape on device idx."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != idx or not t.is_contiguous():
        _refuse(name, t, f"{dtype} {shape} on cuda:{idx}")
    return t.data_ptr()


def _matrix(t, name: str):
    """Shape, sherry_dtype and device index of the [M][.] tensor a feed-forward call starts from."""
    code = _types().get(t.dtype)
    shape = t.shape
    idx = t.get_device()                                # -1: not on a GPU
    if code is None or len(shape) != 2 or idx < 0 or not t.is_contiguous():
        _refuse(name, t, "[M][.] of float32, bfloat16 or float16")
    return shape[0], shape[1], code, idx


def _no_history(what: str):
    raise ValueError(f"{what} is not recorded by autograd and an argument requires a gradient: call it under "
                     "torch.no_grad(), or in a torch.autograd.Function with the *_backward call as its backward")


def _activation(act) -> int:
    a = ACTIVATIONS.get(act)
    if a is None:
        raise ValueError(f"act: want one of {list(ACTIVATIONS)[1:]}, got {act!r}")
    return a


@functools.lru_cache(maxsize=1024)
def _forward_split_bytes(idx: int, gated: bool, dtype: int, act: int, res: bool, acc: bool, M: int, N: int, K: int) -> int:
    """Split-K workspace of a forward call on device idx (the current one)."""
    if gated:
        return int(load().sherry_gated_split_bytes(dtype, act, acc, M, N, K))
    return int(load().sherry_linear_split_bytes(dtype, act, res, acc, M, N, K))


@functools.lru_cache(maxsize=1024)
def _grad_bytes(idx: int, dtype: int, M: int, R: int, K: int):
    """Work buffer (a multiple of 16) and split-K workspace of a gradient call on device idx."""
    return ((int(load().sherry_grad_work_bytes(dtype, M, R)) + 15) & ~15,
            int(load().sherry_grad_split_bytes(dtype, M, R, K)))


def _stream_of(idx: int):
    return _torch._C._cuda_getCurrentRawStream(idx)


def _on_device(fn):
    """Runs a call with its first argument's device current."""
    @functools.wraps(fn)
    def call(x, *args, **kwargs):
        import torch
        if not x.is_cuda or x.device.index == torch.cuda.current_device():
            return fn(x, *args, **kwargs)
        with torch.cuda.device(x.device):
            return fn(x, *args, **kwargs)
    return call


def reserve_split(device=None):
    """Sets aside, host-synchronously, the split-K workspace (about 15 MB) of the C entry points that take
    none from the caller, for any number of tokens on `device` (default: the current one).  Such calls
    share it (sherry.h); linear_epilogue, gated and the gradients bring their own and need no reserve."""
    _types()
    dev = _torch.device("cuda" if device is None else device) if not isinstance(device, int) else \
        _torch.device("cuda", device)
    idx = dev.index if dev.index is not None else _torch.cuda.current_device()
    if idx in _split_reserved:
        return
    if _torch.cuda.is_current_stream_capturing():
        raise RuntimeError("the workspace is not set aside yet: call reserve_split() before capturing a graph")
    with _torch.cuda.device(idx):
        _check(load().sherry_reserve(SPLIT_MAX_M, 1), "sherry_reserve")
    _split_reserved.add(idx)


@_on_device
def repack_gated(gate_dev, up_dev, N: int, K: int, out=None):
    """Canonical codes of a gate and an up projection [N][5K/32] on the device -> the native layout of the
    2N-row weight whose rows 2n, 2n + 1 are row n of each."""
    import torch
    if out is None:
        out = torch.empty(native_bytes(2 * N, K), dtype=torch.uint8, device=gate_dev.device)
    _check(load().sherry_repack_gated(_dptr(gate_dev), _dptr(up_dev), N, K, _dptr(out), _stream(gate_dev)),
           "sherry_repack_gated")
    return out


def transposed_bytes(R: int, K: int) -> int:
    return int(load().sherry_transposed_bytes(R, K))


@_on_device
def repack_t(codes_dev, N: int, K: int, out=None):
    """Canonical codes on the device -> the transposed layout the gradients read."""
    import torch
    if out is None:
        out = torch.empty(transposed_bytes(N, K), dtype=torch.uint8, device=codes_dev.device)
    _check(load().sherry_repack_t(_dptr(codes_dev), N, K, _dptr(out), _stream(codes_dev)), "sherry_repack_t")
    return out


@_on_device
def repack_gated_t(gate_dev, up_dev, N: int, K: int, out=None):
    """repack_t of the interleaved 2N-row weight of repack_gated."""
    import torch
    if out is None:
        out = torch.empty(transposed_bytes(2 * N, K), dtype=torch.uint8, device=gate_dev.device)
    _check(load().sherry_repack_gated_t(_dptr(gate_dev), _dptr(up_dev), N, K, _dptr(out), _stream(gate_dev)),
           "sherry_repack_gated_t")
    return out


def _forward(gated, x, w_native, alpha, N, bias, act, residual, out, acc, out_q, out_s):
    M, K, dt, idx = _matrix(x, "x")
    if _is_grad_enabled() and (
            x.requires_grad or alpha is not None and alpha.requires_grad or bias is not None and bias.requires_grad or
            residual is not None and residual.requires_grad or out is not None and out.requires_grad):
        _no_history("gated" if gated else "linear_epilogue")
    if idx != _torch._C._cuda_getDevice():
        with _torch.cuda.device(idx):
            return _forward(gated, x, w_native, alpha, N, bias, act, residual, out, acc, out_q, out_s)
    a = _activation(act)
    if N <= 0 or K <= 0 or K % 32:
        raise ValueError(f"want N > 0 and K a positive multiple of 32, got N={N}, K={K}")
    R = 2 * N if gated else N
    if w_native is None or alpha is None:
        raise ValueError("w_native and alpha are needed")
    f32 = _torch.float32
    wp = _ptr(w_native, "w_native", _torch.uint8, (-(-R // 128) * -(-K // 128) * 2560,), idx)
    ap = _ptr(alpha, "alpha", f32, (R,), idx)
    bp = None if bias is None else _ptr(bias, "bias", f32, (R,), idx)
    rp = None if residual is None else _ptr(residual, "residual", x.dtype, (M, N), idx)
    cp = None if acc is None else _ptr(acc, "acc", _torch.int32, (M, R), idx)
    qp = None if out_q is None else _ptr(out_q, "out_q", _torch.int8, (M, K), idx)
    sp = None if out_s is None else _ptr(out_s, "out_s", f32, (M,), idx)
    if out is None:
        out = x.new_empty(M, N)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", x.dtype, (M, N), idx)
    if M == 0:
        return out
    # the call's own buffer for the int8 activations, their scales and the split-K sums: nothing is shared
    # with other streams or graphs (one token of up to 65536 needs none)
    kp, split = None, 0
    if M > 1 or K > 65536:
        split = _forward_split_bytes(idx, gated, dt, a, rp is not None, cp is not None, M, N, K)
        # K % 32 == 0: the scales are aligned
        at = (M * K + 4 * M + 15) & ~15 if qp is None or sp is None else 0
        if at or split:
            own = w_native.new_empty(at + split)
            kp = own.data_ptr()
            if qp is None:
                qp = kp
            if sp is None:
                sp = kp + M * K
            kp = kp + at if split else None
    elif qp is not None and sp is None:
        own = w_native.new_empty(4)
        sp = own.data_ptr()
    if gated:
        rc = _lib.sherry_gated_ws(x.data_ptr(), dt, wp, ap, bp, a, op, cp, qp, sp, kp, split, M, N, K, _stream_of(idx))
    else:
        rc = _lib.sherry_linear_epilogue_ws(x.data_ptr(), dt, wp, ap, bp, a, rp, op, cp, qp, sp, kp, split, M, N, K,
                                            _stream_of(idx))
    if rc != OK:
        _check(rc, "sherry_gated" if gated else "sherry_linear_epilogue")
    return out


def linear_epilogue(x, w_native, alpha, N: int, bias=None, act: str = "none", residual=None, out=None, acc=None,
                    out_q=None, out_s=None):
    """y [M][N] = act(linear(x) + bias) + residual in one contraction (sherry_linear_epilogue).

    x, residual and y are float32, bfloat16 or float16 (one type per call); bias fp32 [N]; act a key of
    ACTIVATIONS.  out may be residual itself.  acc int32 [M][N], out_q int8 [M][K] and out_s fp32 [M]
    receive the exact sums, the quantised activations and their scales (linear_backward needs acc and
    out_s).  Not recorded by autograd: with gradients enabled, arguments that require one are refused."""
    return _forward(False, x, w_native, alpha, N, bias, act, residual, out, acc, out_q, out_s)


def gated(x, w_native, alpha, N: int, bias=None, act: str = "silu", out=None, acc=None, out_q=None, out_s=None):
    """h [M][N] = act(gate(x)) * up(x) in one contraction (sherry_gated).

    w_native from repack_gated; alpha, bias fp32 [2N] and acc int32 [M][2N] interleave gate and up
    (entries 2n, 2n + 1).  Other arguments, and autograd, as linear_epilogue."""
    return _forward(True, x, w_native, alpha, N, bias, act, None, out, acc, out_q, out_s)


def _backward(gated, dy, w_t, alpha, K, acc, x_scale, bias, act, out, want_dx, want_scales):
    M, N, dt, idx = _matrix(dy, "dy")
    if _is_grad_enabled() and (
            dy.requires_grad or alpha is not None and alpha.requires_grad or bias is not None and bias.requires_grad or
            out is not None and out.requires_grad):
        _no_history("gated_backward" if gated else "linear_backward")
    if idx != _torch._C._cuda_getDevice():
        with _torch.cuda.device(idx):
            return _backward(gated, dy, w_t, alpha, K, acc, x_scale, bias, act, out, want_dx, want_scales)
    a = _activation(act)
    if N <= 0 or K <= 0 or K % 32:
        raise ValueError(f"want N > 0 and K a positive multiple of 32, got N={N}, K={K}")
    if not (want_dx or want_scales):
        raise ValueError("nothing to compute: want_dx and want_scales are both False")
    if acc is None and (gated or a != 0 or want_scales):
        raise ValueError("acc: needed for this gradient")
    if acc is not None and x_scale is None:
        raise ValueError("x_scale: needed with acc")
    if alpha is None or (w_t is None and want_dx):
        raise ValueError("alpha, and for dx w_t, are needed")
    R = 2 * N if gated else N
    f32 = _torch.float32
    ap = _ptr(alpha, "alpha", f32, (R,), idx)
    bp = None if bias is None else _ptr(bias, "bias", f32, (R,), idx)
    cp = None if acc is None else _ptr(acc, "acc", _torch.int32, (M, R), idx)
    sp = None if x_scale is None else _ptr(x_scale, "x_scale", f32, (M,), idx)
    dx = dalpha = dbias = wp = xp = kp = dap = dbp = lp = None
    split = 0
    if want_dx:
        wp = _ptr(w_t, "w_t", _torch.uint8, (-(-R // 128) * -(-K // 128) * 4096,), idx)
        dx = dy.new_empty(M, K) if out is None else out
        xp = dx.data_ptr() if out is None else _ptr(out, "out", dy.dtype, (M, K), idx)
    if want_scales:
        make = _torch.empty_like if M else _torch.zeros_like
        dalpha, dbias = make(alpha), make(alpha)
        dap, dbp = dalpha.data_ptr(), dbias.data_ptr()
    if M == 0:
        return dx, dalpha, dbias
    if want_dx:
        digits, split = _grad_bytes(idx, dt, M, R, K)
        work = w_t.new_empty(digits + split)            # nothing is shared with other streams or graphs
        kp = work.data_ptr()
        if split:
            lp = kp + digits
    fn = _lib.sherry_gated_grad_ws if gated else _lib.sherry_linear_grad_ws
    rc = fn(dy.data_ptr(), dt, cp, sp, wp, ap, bp, a, xp, dap, dbp, kp, lp, split, M, N, K, _stream_of(idx))
    if rc != OK:
        _check(rc, "sherry_gated_grad" if gated else "sherry_linear_grad")
    return dx, dalpha, dbias


def linear_backward(dy, w_t, alpha, K: int, acc=None, x_scale=None, bias=None, act: str = "none", out=None,
                    want_dx: bool = True, want_scales: bool = True):
    """Gradients of linear_epilogue: (dx [M][K] of dy's type, dalpha fp32 [N], dbias fp32 [N]).

    dy [M][N]; w_t from repack_t; acc and x_scale as the forward call gave them (acc and out_s), bias and
    act as it took them.  want_dx / want_scales False leave out dx / dalpha and dbias (None in their
    place); with act "none" and want_scales False acc and x_scale are not needed.  The gradient of the
    residual is dy itself."""
    return _backward(False, dy, w_t, alpha, K, acc, x_scale, bias, act, out, want_dx, want_scales)


def gated_backward(dh, w_t, alpha, K: int, acc, x_scale, bias=None, act: str = "silu", out=None,
                   want_dx: bool = True, want_scales: bool = True):
    """Gradients of gated: (dx [M][K], dalpha fp32 [2N], dbias fp32 [2N], interleaved).  w_t from
    repack_gated_t; other arguments as linear_backward."""
    return _backward(True, dh, w_t, alpha, K, acc, x_scale, bias, act, out, want_dx, want_scales)


class PackedLinear:
    """Weights of one Sherry linear layer resident on the device.

    ``PackedLinear.from_weights(W)`` packs on the host (sherry_pack), copies
    the canonical codes and alpha to the device and repacks them into the
    kernel-native layout.  ``forward(x)`` quantises the activations and runs
    the GEMM (sherry_linear), asynchronously on the current stream; with a
    bias, an activation or a residual, or 16-bit activations, it is
    sherry_linear_epilogue.  ``trainable=True`` also lays out the transposed
    weight that ``backward`` reads.
    """

    def __init__(self, w_native, alpha, N: int, K: int, w_t=None):
        self.w_native, self.alpha, self.N, self.K, self.w_t = w_native, alpha, N, K, w_t

    @classmethod
    def from_weights(cls, W: np.ndarray, device="cuda", trainable: bool = False):
        import torch
        codes, alpha = pack(W)
        return cls.from_codes(codes, alpha, W.shape[1], device, trainable)

    @classmethod
    def from_codes(cls, codes: np.ndarray, alpha: np.ndarray, K: int, device="cuda", trainable: bool = False):
        import torch
        N = codes.shape[0]
        codes_d = torch.from_numpy(codes).to(device)
        w_native = repack(codes_d, N, K)
        return cls(w_native, torch.from_numpy(alpha).to(device), N, K, repack_t(codes_d, N, K) if trainable else None)

    def forward(self, x, out=None, bias=None, act: str = "none", residual=None, acc=None, out_s=None):
        import torch
        if x.dtype is torch.float32 and bias is None and act in (None, "none") and residual is None and out_s is None:
            return linear(x, self.w_native, self.alpha, self.N, out=out, acc=acc)
        return linear_epilogue(x, self.w_native, self.alpha, self.N, bias=bias, act=act, residual=residual, out=out,
                               acc=acc, out_s=out_s)

    def backward(self, dy, acc=None, x_scale=None, bias=None, act: str = "none", want_dx: bool = True,
                 want_scales: bool = True):
        """linear_backward of this layer: (dx, dalpha, dbias)."""
        _need(self.w_t is not None or not want_dx, "backward: the layer was made without trainable=True")
        return linear_backward(dy, self.w_t, self.alpha, self.K, acc, x_scale, bias=bias, act=act, want_dx=want_dx,
                               want_scales=want_scales)


class GatedFFN:
    """A gated feed-forward block over packed weights: y = down(act(gate(x)) * up(x)) + residual.

    ``GatedFFN.from_weights(W_gate, W_up, W_down)`` (fp32 [F][K], [F][K], [K2][F]) packs on the host;
    ``forward(x, residual)`` is two contractions, each with its epilogue.  With ``trainable=True``,
    ``forward(x, residual, keep=True)`` also returns what ``backward(dy, kept)`` needs for the gradients
    of x and of the scales (the packed weights themselves stay as they are).  Autograd does not record
    them: see linear_epilogue.
    """

    def __init__(self, w_native, alpha, down: PackedLinear, F: int, K: int, act: str = "silu", w_t=None):
        self.w_native, self.alpha, self.down, self.F, self.K, self.act, self.w_t = w_native, alpha, down, F, K, act, w_t

    @classmethod
    def from_weights(cls, W_gate: np.ndarray, W_up: np.ndarray, W_down: np.ndarray, act: str = "silu", device="cuda",
                     trainable: bool = False):
        import torch
        _need(W_gate.shape == W_up.shape and W_down.shape[1] == W_gate.shape[0],
              f"GatedFFN: shapes {W_gate.shape}, {W_up.shape}, {W_down.shape} do not chain")
        _activation(act)
        F, K = W_gate.shape
        (cg, ag), (cu, au) = pack(W_gate), pack(W_up)
        cg, cu = torch.from_numpy(cg).to(device), torch.from_numpy(cu).to(device)
        alpha = torch.from_numpy(np.ascontiguousarray(np.stack([ag, au], 1).reshape(-1))).to(device)
        return cls(repack_gated(cg, cu, F, K), alpha, PackedLinear.from_weights(W_down, device, trainable), F, K, act,
                   repack_gated_t(cg, cu, F, K) if trainable else None)

    def forward(self, x, residual=None, keep: bool = False):
        import torch
        if not keep:
            h = gated(x, self.w_native, self.alpha, self.F, act=self.act)
            return linear_epilogue(h, self.down.w_native, self.down.alpha, self.down.N, residual=residual)
        M = x.shape[0]
        acc = torch.empty((M, 2 * self.F), dtype=torch.int32, device=x.device)
        acc_d = torch.empty((M, self.down.N), dtype=torch.int32, device=x.device)
        s, s_d = (torch.empty(M, dtype=torch.float32, device=x.device) for _ in range(2))
        h = gated(x, self.w_native, self.alpha, self.F, act=self.act, acc=acc, out_s=s)
        y = linear_epilogue(h, self.down.w_native, self.down.alpha, self.down.N, residual=residual, acc=acc_d, out_s=s_d)
        return y, (acc, s, acc_d, s_d)

    def backward(self, dy, kept, want_dx: bool = True, want_scales: bool = True):
        """(dx, dalpha fp32 [2F] interleaved, dalpha of the down projection fp32 [K2]); the gradient of the
        residual is dy itself."""
        _need(self.w_t is not None or not want_dx, "backward: the block was made without trainable=True")
        acc, s, acc_d, s_d = kept
        dh, dalpha_d, _ = self.down.backward(dy, acc_d, s_d, want_scales=want_scales)
        dx, dalpha, _ = gated_backward(dh, self.w_t, self.alpha, self.K, acc, s, act=self.act, want_dx=want_dx,
                                       want_scales=want_scales)
        return dx, dalpha, dalpha_d


# ------------------------------------------------ W4A8 FastGEMM (SINT4 x int8)
def w4a8_packed_bytes(N: int, K: int) -> int:
    return int(load().sherry_w4a8_packed_bytes(N, K))


def w4a8_native_bytes(N: int, K: int) -> int:
    return int(load().sherry_w4a8_native_bytes(N, K))


def w4a8_pack(W: np.ndarray):
    """fp32 W [N][K] -> (canonical SINT4 rows uint8 [N][K/2], per-channel scale fp32 [N])."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    w4 = np.empty((N, K // 2), dtype=np.uint8)
    scale = np.empty(N, dtype=np.float32)
    _check(load().sherry_w4a8_pack(_np_ptr(W), N, K, _np_ptr(w4), _np_ptr(scale)), "sherry_w4a8_pack")
    return w4, scale


def w4a8_unpack(w4: np.ndarray, K: int) -> np.ndarray:
    w4 = np.ascontiguousarray(w4, dtype=np.uint8)
    N = w4.shape[0]
    Wq = np.empty((N, K), dtype=np.int8)
    _check(load().sherry_w4a8_unpack(_np_ptr(w4), N, K, _np_ptr(Wq)), "sherry_w4a8_unpack")
    return Wq


def w4a8_repack(w4_dev, N: int, K: int, out=None):
    """Canonical SINT4 rows on the device -> kernel-native layout (uint8 tensor)."""
    import torch
    if out is None:
        out = torch.empty(w4a8_native_bytes(N, K), dtype=torch.uint8, device=w4_dev.device)
    _check(load().sherry_w4a8_repack(_dptr(w4_dev), N, K, _dptr(out), _stream(w4_dev)), "sherry_w4a8_repack")
    return out


W4A8_GEMV_MAX_M = 4   # SHERRY_W4A8_GEMV_MAX_M


def w4a8_gemm(x_i8, x_scale, w4_native, scale, N: int, out=None, acc=None, want_y: bool = True,
              kernel: str = "auto"):
    """y fp32 [M][N] (and optionally the int32 sums after the division by 16)
    from int8 activations and kernel-native SINT4 weights.  kernel: "auto"
    (sherry_w4a8_gemm: the tensor-core kernel for every M), "tc" or "gemv"
    (the CUDA-core comparison kernel, M <= 4)."""
    import torch
    M, K = x_i8.shape
    y = None
    if want_y:
        y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=x_i8.device)
    L = load()
    _ensure_workspace(x_i8, M, K)
    args = (_dptr(x_i8), _dptr(x_scale), _dptr(w4_native), _dptr(scale), _dptr(y), _dptr(acc), M, N, K,
            _stream(x_i8))
    if kernel == "auto":
        if acc is None:
            rc = L.sherry_w4a8_gemm(args[0], args[1], args[2], args[3], args[4], M, N, K, args[-1])
        else:
            rc = L.sherry_w4a8_gemm_acc(*args)
    elif kernel == "tc":
        rc = L.sherry_w4a8_gemm_tc(*args)
    elif kernel == "gemv":
        rc = L.sherry_w4a8_gemm_gemv(*args)
    else:
        raise ValueError(kernel)
    _check(rc, f"sherry_w4a8_gemm[{kernel}]")
    return y


class W4A8Linear:
    """Weights of one W4A8 linear layer resident on the device.

    ``W4A8Linear.from_weights(W)`` quantises and packs on the host
    (sherry_w4a8_pack), copies the SINT4 rows and the channel scales to the
    device and repacks them (sherry_w4a8_repack).  ``forward(x)`` quantises
    the activations (sherry_quant_act) and runs the W4A8 GEMM
    (sherry_w4a8_gemm), asynchronously on the current stream.
    """

    def __init__(self, w_native, scale, N: int, K: int):
        self.w_native, self.scale, self.N, self.K = w_native, scale, N, K

    @classmethod
    def from_weights(cls, W: np.ndarray, device="cuda"):
        import torch
        w4, scale = w4a8_pack(W)
        N, K = W.shape
        w_native = w4a8_repack(torch.from_numpy(w4).to(device), N, K)
        return cls(w_native, torch.from_numpy(scale).to(device), N, K)

    def forward(self, x, out=None):
        q, s = quant_act(x)
        return w4a8_gemm(q, s, self.w_native, self.scale, self.N, out=out)
