"""ctypes binding of ``libsgemm_gb300.so`` — argument marshalling only.

Each function here has the name and argument order of the C entry point in
``include/sgemm.h``. All arithmetic happens in the CUDA kernels; there is no
CPU path. If the shared library has not been built, every call raises
``RuntimeError`` (build it with ``dense_fp32_matrix_strict_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

SGEMM_OK = 0
SGEMM_ERR_INVALID_VALUE = 1
SGEMM_ERR_UNSUPPORTED_DEVICE = 2
SGEMM_ERR_LAUNCH = 3
SGEMM_ERR_DEVICE_TIMEOUT = 4
SGEMM_ERR_CUDA = 5
SGEMM_ERR_DEVICE_CHECK = 6

# Every function include/sgemm.h declares.
EXPORTED_SYMBOLS = (
    "sgemm", "sgemm_check_status", "sgemm_error_string", "sgemm_last_cuda_error",
    "sgemm_plan", "sgemm_set_config", "sgemm_set_wait_timeout_ns", "sgemm_fp32_peak",
    "sgemm_selftest_wait_timeout", "sgemm_config_names", "sgemm_noalloc", "sgemm_3xtf32",
    "sgemm_set_shape_config", "sgemm_clear_shape_configs", "sgemm_ex", "sgemm_plan_ex",
    "sgemm_3xtf32_ex", "sgemm_host", "sgemm_noalloc_check_status", "sgemm_fp32_peak_ex",
    "sgemm_null_launch", "sgemm_tf32_mma_peak", "sgemm_selftest_occupy",
    "sgemm_route", "sgemm_route_backward", "sgemm_grouped", "sgemm_grouped_wgrad", "sgemv_w4",
)

SGEMM_PEAK_FFMA, SGEMM_PEAK_FFMA2, SGEMM_PEAK_OUTER = 0, 1, 2

SGEMM_OP_N, SGEMM_OP_T = 0, 1

# Element types of the expert-layer entry points.
SGEMM_TYPE_F32, SGEMM_TYPE_BF16 = 0, 1
# Largest rows, M, N, K of the grouped products, and N of sgemv_w4.
SGEMM_GROUPED_MAX_DIM = 2 ** 31 - 65536
# Largest K of sgemv_w4.
SGEMV_W4_MAX_K = 524288

_lock = threading.Lock()
_lib = None


class SgemmError(RuntimeError):
    """A non-zero return code from the library."""

    def __init__(self, func: str, code: int):
        self.code = int(code)
        msg = _lib.sgemm_error_string(code).decode() if _lib is not None else str(code)
        cuda = _lib.sgemm_last_cuda_error() if _lib is not None else 0
        extra = f" (CUDA error {cuda})" if cuda and code in (SGEMM_ERR_LAUNCH, SGEMM_ERR_CUDA) else ""
        super().__init__(f"{func} failed: {msg} [code {code}]{extra}")


def library_path() -> str:
    return os.environ.get("SGEMM_LIBRARY") or _build.LIB_PATH


def load():
    """Load the shared library (once). Raises RuntimeError if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        # SGEMM_LIBRARY selects another build of the same library (the
        # debug build, for instance); by default the in-tree release build.
        path = os.environ.get("SGEMM_LIBRARY") or _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: the CUDA library has not been built "
                "(run `python -m dense_fp32_matrix_strict_gb300.build`); there is no CPU path")
        lib = ctypes.CDLL(path)
        i64, f32, vp, ci, f64p = (ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int,
                                  ctypes.POINTER(ctypes.c_double))
        lib.sgemm.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
        lib.sgemm.restype = ci
        lib.sgemm_check_status.argtypes = [vp, ctypes.POINTER(ci)]
        lib.sgemm_check_status.restype = ci
        lib.sgemm_error_string.argtypes = [ci]
        lib.sgemm_error_string.restype = ctypes.c_char_p
        lib.sgemm_last_cuda_error.argtypes = []
        lib.sgemm_last_cuda_error.restype = ci
        lib.sgemm_plan.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64,
                                   ctypes.c_char_p, ci, ctypes.POINTER(ci)]
        lib.sgemm_plan.restype = ci
        lib.sgemm_set_config.argtypes = [ctypes.c_char_p]
        lib.sgemm_set_config.restype = ci
        lib.sgemm_config_names.argtypes = [ctypes.c_char_p, ci]
        lib.sgemm_config_names.restype = ci
        lib.sgemm_set_shape_config.argtypes = [i64, i64, i64, ctypes.c_char_p]
        lib.sgemm_set_shape_config.restype = ci
        lib.sgemm_clear_shape_configs.argtypes = []
        lib.sgemm_clear_shape_configs.restype = ci
        lib.sgemm_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
        lib.sgemm_set_wait_timeout_ns.restype = ci
        lib.sgemm_fp32_peak.argtypes = [ctypes.c_double, f64p, f64p, f64p, vp]
        lib.sgemm_fp32_peak.restype = ci
        lib.sgemm_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
        lib.sgemm_selftest_wait_timeout.restype = ci
        lib.sgemm_selftest_occupy.argtypes = [ci, ctypes.c_uint64, vp]
        lib.sgemm_selftest_occupy.restype = ci
        lib.sgemm_noalloc.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
        lib.sgemm_noalloc.restype = ci
        lib.sgemm_noalloc_check_status.argtypes = [vp, ctypes.POINTER(ci)]
        lib.sgemm_noalloc_check_status.restype = ci
        lib.sgemm_fp32_peak_ex.argtypes = [ci, ctypes.c_double, f64p, f64p, f64p, vp]
        lib.sgemm_fp32_peak_ex.restype = ci
        lib.sgemm_null_launch.argtypes = [vp]
        lib.sgemm_tf32_mma_peak.argtypes = [ci, ctypes.c_double, f64p, f64p, f64p, vp]
        lib.sgemm_tf32_mma_peak.restype = ci
        lib.sgemm_null_launch.restype = ci
        lib.sgemm_3xtf32.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
        lib.sgemm_3xtf32.restype = ci
        lib.sgemm_ex.argtypes = [ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
        lib.sgemm_ex.restype = ci
        lib.sgemm_3xtf32_ex.argtypes = [ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp,
                                        i64, vp]
        lib.sgemm_3xtf32_ex.restype = ci
        lib.sgemm_plan_ex.argtypes = [ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64,
                                      ctypes.c_char_p, ci, ctypes.POINTER(ci)]
        lib.sgemm_plan_ex.restype = ci
        lib.sgemm_host.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
        lib.sgemm_host.restype = ci
        lib.sgemm_route.argtypes = [ci, i64, i64, i64, ci, vp, i64, vp, vp, vp, vp, vp, vp]
        lib.sgemm_route.restype = ci
        lib.sgemm_route_backward.argtypes = [ci, i64, i64, i64, ci, vp, i64, vp, vp, vp, i64, vp]
        lib.sgemm_route_backward.restype = ci
        lib.sgemm_grouped.argtypes = [ci, ci, i64, i64, i64, i64, f32, vp, i64, vp, i64, i64, vp,
                                      f32, vp, i64, vp]
        lib.sgemm_grouped.restype = ci
        lib.sgemm_grouped_wgrad.argtypes = [ci, i64, i64, i64, i64, f32, vp, i64, vp, i64, vp, f32,
                                            ci, vp, i64, i64, vp]
        lib.sgemm_grouped_wgrad.restype = ci
        lib.sgemv_w4.argtypes = [ci, i64, i64, i64, i64, i64, vp, i64, vp, i64, i64, vp, vp, i64,
                                 vp, vp, i64, vp]
        lib.sgemv_w4.restype = ci
        _lib = lib
        return lib


def _check(func: str, rc: int) -> int:
    if rc != SGEMM_OK:
        raise SgemmError(func, rc)
    return rc


# ---- raw entry points (same names and argument order as the C ABI) --------

def sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """C = alpha*A*B + beta*C on device pointers (ints); returns the raw code."""
    return load().sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """sgemm without any device allocation (fixed scratch inside the library);
    device pointers as ints; returns the raw code."""
    return load().sgemm_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_noalloc_check_status(stream=0):
    """Returns (code, bits) of the scratch status word sgemm_noalloc writes."""
    bits = ctypes.c_int(0)
    rc = load().sgemm_noalloc_check_status(stream, ctypes.byref(bits))
    return rc, bits.value


def sgemm_3xtf32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """The tcgen05 3xTF32 path (device pointers as ints); returns the raw code."""
    return load().sgemm_3xtf32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_ex(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """C = alpha*op(A)*op(B) + beta*C (op: SGEMM_OP_N / SGEMM_OP_T); raw code."""
    return load().sgemm_ex(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_3xtf32_ex(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().sgemm_3xtf32_ex(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_plan_ex(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc):
    """Returns (code, kernel name, grid)."""
    buf = ctypes.create_string_buffer(128)
    grid = ctypes.c_int(0)
    rc = load().sgemm_plan_ex(opa, opb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, buf, 128,
                              ctypes.byref(grid))
    return rc, buf.value.decode(), grid.value


def sgemm_host(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """C = alpha*A*B + beta*C with HOST pointers (ints); returns the raw code."""
    return load().sgemm_host(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_check_status(stream=0):
    """Returns (code, bits)."""
    bits = ctypes.c_int(0)
    rc = load().sgemm_check_status(stream, ctypes.byref(bits))
    return rc, bits.value


def sgemm_error_string(code: int) -> str:
    return load().sgemm_error_string(code).decode()


def sgemm_last_cuda_error() -> int:
    return load().sgemm_last_cuda_error()


def sgemm_plan(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc):
    """Returns (code, kernel name, grid)."""
    buf = ctypes.create_string_buffer(128)
    grid = ctypes.c_int(0)
    rc = load().sgemm_plan(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, buf, 128,
                           ctypes.byref(grid))
    return rc, buf.value.decode(), grid.value


def sgemm_set_config(name: str) -> int:
    return load().sgemm_set_config(name.encode())


def sgemm_set_shape_config(M: int, N: int, K: int, name) -> int:
    """Per-shape configuration rule; name None or "auto" removes it."""
    return load().sgemm_set_shape_config(M, N, K, None if name is None else name.encode())


def sgemm_clear_shape_configs() -> int:
    return load().sgemm_clear_shape_configs()


def sgemm_config_names():
    """Returns (code, [family names])."""
    buf = ctypes.create_string_buffer(4096)
    rc = load().sgemm_config_names(buf, 4096)
    names = buf.value.decode().split(",") if rc == SGEMM_OK and buf.value else []
    return rc, names


def sgemm_set_wait_timeout_ns(ns: int) -> int:
    return load().sgemm_set_wait_timeout_ns(int(ns))


def sgemm_fp32_peak(target_ms: float = 200.0, stream=0):
    """Returns (code, gflops, ms, flops)."""
    g, m, f = ctypes.c_double(0), ctypes.c_double(0), ctypes.c_double(0)
    rc = load().sgemm_fp32_peak(float(target_ms), ctypes.byref(g), ctypes.byref(m),
                                ctypes.byref(f), stream)
    return rc, g.value, m.value, f.value


def sgemm_fp32_peak_ex(form: int, target_ms: float = 200.0, stream=0):
    """Returns (code, gflops, ms, flops) of the chosen instruction form."""
    g, m, f = ctypes.c_double(0), ctypes.c_double(0), ctypes.c_double(0)
    rc = load().sgemm_fp32_peak_ex(int(form), float(target_ms), ctypes.byref(g),
                                   ctypes.byref(m), ctypes.byref(f), stream)
    return rc, g.value, m.value, f.value


def sgemm_tf32_mma_peak(n: int = 128, target_ms: float = 100.0, stream=0):
    """Returns (code, tflops, ms, flops) of the TF32 tcgen05 MMA ceiling."""
    t, m, f = ctypes.c_double(0), ctypes.c_double(0), ctypes.c_double(0)
    rc = load().sgemm_tf32_mma_peak(int(n), float(target_ms), ctypes.byref(t), ctypes.byref(m),
                                    ctypes.byref(f), stream)
    return rc, t.value, m.value, f.value


def sgemm_null_launch(stream=0) -> int:
    """One empty kernel on `stream` (the launch-latency floor); raw code."""
    return load().sgemm_null_launch(stream)


def sgemm_selftest_wait_timeout(timeout_ns: int, stream=0) -> int:
    return load().sgemm_selftest_wait_timeout(int(timeout_ns), stream)


def sgemm_selftest_occupy(ctas: int, ns: int, stream=0) -> int:
    """`ctas` CTAs holding one SM each for `ns` ns on `stream`; raw code."""
    return load().sgemm_selftest_occupy(int(ctas), int(ns), stream)


def sgemm_route(type, T, E, top, renorm, logits, ldl, weights, experts, offsets, order, place,
                stream=0) -> int:
    """Top-k routing of T tokens on device pointers (ints); returns the raw code."""
    return load().sgemm_route(type, T, E, top, renorm, logits, ldl, weights, experts, offsets,
                              order, place, stream)


def sgemm_route_backward(type, T, E, top, renorm, logits, ldl, experts, dweights, dlogits, ldd,
                         stream=0) -> int:
    """Gradient of the logits (device pointers as ints); returns the raw code."""
    return load().sgemm_route_backward(type, T, E, top, renorm, logits, ldl, experts, dweights,
                                       dlogits, ldd, stream)


def sgemm_grouped(opw, type, groups, rows, N, K, alpha, X, ldx, W, ldw, stride_w, offsets, beta, Y,
                  ldy, stream=0) -> int:
    """Products grouped by expert (device pointers as ints); returns the raw code."""
    return load().sgemm_grouped(opw, type, groups, rows, N, K, alpha, X, ldx, W, ldw, stride_w,
                                offsets, beta, Y, ldy, stream)


def sgemm_grouped_wgrad(type, groups, rows, M, N, alpha, P, ldp, Q, ldq, offsets, beta, out_type, D,
                        ldd, stride_d, stream=0) -> int:
    """Weight gradients grouped by expert (device pointers as ints); raw code."""
    return load().sgemm_grouped_wgrad(type, groups, rows, M, N, alpha, P, ldp, Q, ldq, offsets,
                                      beta, out_type, D, ldd, stride_d, stream)


def sgemv_w4(type, pairs, repeat, N, K, group, X, ldx, Q, ldq, stride_q, scales, zeros, num_experts,
             experts, Y, ldy, stream=0) -> int:
    """Products of a few tokens with 4-bit weights (device pointers as ints); raw code."""
    return load().sgemv_w4(type, pairs, repeat, N, K, group, X, ldx, Q, ldq, stride_q, scales,
                           zeros, num_experts, experts, Y, ldy, stream)


# ---- torch tensor convenience (marshalling only) --------------------------

def _ld(t, rows, cols, name):
    import torch
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(t.shape)}")
    if rows == 0 or cols == 0:
        return max(cols, 1)
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with contiguous columns")
    return max(t.stride(0) if rows > 1 else cols, cols, 1)


def _stream_handle(stream, device):
    import torch
    if stream is None:
        idx = device.index if hasattr(device, "index") else device
        if idx is None:
            idx = torch.cuda.current_device()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return int(raw(idx))
        stream = torch.cuda.current_stream(idx)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


class _on_device:
    """Make `device` current for the duration of a call (no-op if it is)."""

    def __init__(self, device):
        import torch
        self.idx = device.index if device.index is not None else torch.cuda.current_device()
        self.prev = None

    def __enter__(self):
        import torch
        cur = torch.cuda.current_device()
        if cur != self.idx:
            self.prev = cur
            torch.cuda.set_device(self.idx)
        return self

    def __exit__(self, *exc):
        if self.prev is not None:
            import torch
            torch.cuda.set_device(self.prev)
        return False


def _shapes(A, B, transa, transb):
    """(M, N, K, lda, ldb) of op(A) op(B) from the stored tensors."""
    M, K = (A.shape[1], A.shape[0]) if transa else (A.shape[0], A.shape[1])
    K2, N = (B.shape[1], B.shape[0]) if transb else (B.shape[0], B.shape[1])
    if K2 != K:
        raise ValueError(f"inner dimensions differ: op(A) is {(M, K)}, op(B) is {(K2, N)}")
    lda = _ld(A, A.shape[0], A.shape[1], "A")
    ldb = _ld(B, B.shape[0], B.shape[1], "B")
    return M, N, K, lda, ldb


def _op(flag: bool) -> int:
    return SGEMM_OP_T if flag else SGEMM_OP_N


def sgemm_tensors(alpha, A, B, beta, C, stream=None, transa=False, transb=False) -> None:
    """C = alpha * op(A) @ op(B) + beta * C in place on row-major float32 CUDA tensors.

    op(X) is X, or X.T when trans* is set (the tensor is then the stored,
    untransposed matrix: A of shape (K, M), B of shape (N, K)). Rows may be
    strided (leading dimension = stride(0)). Launches on ``stream``
    (default: torch's current stream on C's device). Raises SgemmError on a
    non-zero return code.
    """
    M, N, K, lda, ldb = _shapes(A, B, transa, transb)
    ldc = _ld(C, M, N, "C")
    if not (A.device == B.device == C.device):
        raise ValueError("A, B and C must be on the same device")
    with _on_device(C.device):
        h = _stream_handle(stream, C.device)
        if transa or transb:
            rc = load().sgemm_ex(_op(transa), _op(transb), M, N, K, float(alpha), A.data_ptr(),
                                 lda, B.data_ptr(), ldb, float(beta), C.data_ptr(), ldc, h)
        else:
            rc = load().sgemm(M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb,
                              float(beta), C.data_ptr(), ldc, h)
    if rc != SGEMM_OK:
        raise SgemmError("sgemm_ex" if (transa or transb) else "sgemm", rc)


def sgemm_3xtf32_tensors(alpha, A, B, beta, C, stream=None, transa=False, transb=False) -> None:
    """sgemm_tensors through the tcgen05 3xTF32 entry points."""
    M, N, K, lda, ldb = _shapes(A, B, transa, transb)
    ldc = _ld(C, M, N, "C")
    with _on_device(C.device):
        h = _stream_handle(stream, C.device)
        if transa or transb:
            rc = load().sgemm_3xtf32_ex(_op(transa), _op(transb), M, N, K, float(alpha),
                                        A.data_ptr(), lda, B.data_ptr(), ldb, float(beta),
                                        C.data_ptr(), ldc, h)
        else:
            rc = load().sgemm_3xtf32(M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb,
                                     float(beta), C.data_ptr(), ldc, h)
    if rc != SGEMM_OK:
        raise SgemmError("sgemm_3xtf32", rc)


def _host_ld(t, rows, cols, name):
    import torch
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.is_cuda:
        raise TypeError(f"{name} must be a host (CPU) tensor")
    if t.dim() != 2 or tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(t.shape)}")
    if rows == 0 or cols == 0:
        return max(cols, 1)
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with contiguous columns")
    return max(t.stride(0) if rows > 1 else cols, cols, 1)


def sgemm_host_tensors(alpha, A, B, beta, C, stream=None, device=None) -> None:
    """sgemm_host on row-major float32 CPU tensors (pin them for overlap).

    Enqueued on ``stream`` (default: torch's current stream on ``device``);
    C is complete once that stream is synchronised.
    """
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    lda = _host_ld(A, M, K, "A")
    ldb = _host_ld(B, K, N, "B")
    ldc = _host_ld(C, M, N, "C")
    dev = (torch.device("cuda", torch.cuda.current_device()) if device is None
           else torch.device(device))
    with _on_device(dev):
        rc = load().sgemm_host(M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb,
                               float(beta), C.data_ptr(), ldc, _stream_handle(stream, dev))
    if rc != SGEMM_OK:
        raise SgemmError("sgemm_host", rc)


# The expert-layer calls are short (a few microseconds on the device), so their
# wrappers ask each tensor for as little as they can.

_types = None           # {dtype: SGEMM_TYPE_*}
_i32 = _u8 = _f32 = None
_get_device = _raw_stream = None


def _bind_torch():
    """torch's dtypes and current-device functions, on the first call."""
    global _types, _i32, _u8, _f32, _get_device, _raw_stream
    import torch
    _i32, _u8, _f32 = torch.int32, torch.uint8, torch.float32
    _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                   or (lambda i: torch.cuda.current_stream(i).cuda_stream))
    _types = {torch.float32: SGEMM_TYPE_F32, torch.bfloat16: SGEMM_TYPE_BF16}
    return _types


def _type_of(t, name):
    typ = (_types or _bind_torch()).get(t.dtype)
    if typ is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return typ


def _index_of(t, name):
    """Device index of a CUDA tensor."""
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return dev


def _placed(t, name, dtype, dev):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} must be on the same device as the other tensors")


def _typed_ld(t, rows, cols, name, dtype, dev):
    """Row stride of a rows x cols tensor of `dtype` with contiguous columns."""
    _placed(t, name, dtype, dev)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(t.shape)}")
    if rows < 2 or cols == 0:
        ld, st = max(cols, 1), t.stride(1)
    else:
        ld, st = t.stride()
    if st != 1 and cols > 1 and rows:
        raise ValueError(f"{name} must be row-major with contiguous columns")
    return ld


def _stacked_ld(t, shape, name, dtype, dev):
    """(row stride, matrix stride) of a stack of row-major matrices."""
    _placed(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    groups, rows, cols = shape
    if groups == 0 or rows == 0 or cols == 0:
        return max(cols, 1), 0
    stride, ld, st = t.stride()
    if cols > 1 and st != 1:
        raise ValueError(f"{name} must be row-major with contiguous columns")
    if rows < 2:
        ld = max(cols, 1)
    return ld, stride if groups > 1 else rows * ld


def _flat(t, shape, name, dtype, dev):
    """Pointer of a contiguous tensor of this shape and type."""
    _placed(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _call(func, name, dev, stream, *args):
    """func(*args, stream) with `dev` current; SgemmError on a non-zero code."""
    if stream is None:
        handle = _raw_stream(dev)
    else:
        handle = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    if _get_device() == dev:
        rc = func(*args, handle)
    else:
        import torch
        with torch.cuda.device(dev):
            rc = func(*args, handle)
    if rc != SGEMM_OK:
        raise SgemmError(name, rc)


def sgemm_route_tensors(logits, weights, experts, offsets, order, place, renorm=True,
                        stream=None) -> None:
    """sgemm_route on CUDA tensors: logits (T, E) float32 or bfloat16; outputs
    weights (T, top) float32, experts and place (T, top), offsets (E + 1,) and
    order (T * top,), all int32. Enqueued on ``stream`` (default: torch's
    current stream)."""
    typ = _type_of(logits, "logits")
    if logits.dim() != 2 or weights.dim() != 2:
        raise ValueError("logits and weights must have two dimensions")
    T, E = logits.shape
    top = weights.shape[1]
    dev = _index_of(logits, "logits")
    ldl = _typed_ld(logits, T, E, "logits", logits.dtype, dev)
    w = _flat(weights, (T, top), "weights", _f32, dev)
    e = _flat(experts, (T, top), "experts", _i32, dev)
    f = _flat(offsets, (E + 1,), "offsets", _i32, dev)
    o = _flat(order, (T * top,), "order", _i32, dev)
    pl = _flat(place, (T, top), "place", _i32, dev)
    _call(load().sgemm_route, "sgemm_route", dev, stream, typ, T, E, top, 1 if renorm else 0,
          logits.data_ptr(), ldl, w, e, f, o, pl)


def sgemm_route_backward_tensors(logits, experts, dweights, dlogits, renorm=True,
                                 stream=None) -> None:
    """sgemm_route_backward on CUDA tensors: dlogits (T, E) of logits' type from
    dweights (T, top) float32 and the experts (T, top) int32 of the forward call."""
    typ = _type_of(logits, "logits")
    if logits.dim() != 2 or experts.dim() != 2:
        raise ValueError("logits and experts must have two dimensions")
    T, E = logits.shape
    top = experts.shape[1]
    dev = _index_of(logits, "logits")
    dtype = logits.dtype
    ldl = _typed_ld(logits, T, E, "logits", dtype, dev)
    ldd = _typed_ld(dlogits, T, E, "dlogits", dtype, dev)
    e = _flat(experts, (T, top), "experts", _i32, dev)
    dw = _flat(dweights, (T, top), "dweights", _f32, dev)
    _call(load().sgemm_route_backward, "sgemm_route_backward", dev, stream, typ, T, E, top,
          1 if renorm else 0, logits.data_ptr(), ldl, e, dw, dlogits.data_ptr(), ldd)


def sgemm_grouped_tensors(alpha, X, W, offsets, beta, Y, stream=None, transw=False) -> None:
    """Y[r] = alpha * X[r] @ op(W[g]) + beta * Y[r] for the rows offsets[g] <= r < offsets[g+1].

    X (rows, K) and Y (rows, N), float32 or bfloat16; W (groups, K, N), or
    (groups, N, K) with transw; offsets (groups + 1,) int32 on the device.
    Rows and matrices may be strided, columns are contiguous. Enqueued on
    ``stream`` (default: torch's current stream).
    """
    typ = _type_of(X, "X")
    if X.dim() != 2 or W.dim() != 3:
        raise ValueError("X must have two and W three dimensions")
    rows, K = X.shape
    shape = W.shape
    groups, K2, N = shape
    if transw:
        K2, N = N, K2
    if K2 != K:
        raise ValueError(f"inner dimensions differ: X is {(rows, K)}, op(W) is {(groups, K2, N)}")
    dtype = X.dtype
    dev = _index_of(X, "X")
    ldx = _typed_ld(X, rows, K, "X", dtype, dev)
    ldw, stride_w = _stacked_ld(W, shape, "W", dtype, dev)
    ldy = _typed_ld(Y, rows, N, "Y", dtype, dev)
    off = _flat(offsets, (groups + 1,), "offsets", _i32, dev)
    _call(load().sgemm_grouped, "sgemm_grouped", dev, stream, 1 if transw else 0, typ, groups, rows, N,
          K, alpha, X.data_ptr(), ldx, W.data_ptr(), ldw, stride_w, off, beta, Y.data_ptr(), ldy)


def sgemm_grouped_wgrad_tensors(alpha, P, Q, offsets, beta, D, stream=None) -> None:
    """D[g] = alpha * P[rows of g].T @ Q[rows of g] + beta * D[g].

    P (rows, M) and Q (rows, N), float32 or bfloat16; D (groups, M, N) float32
    or of P's type; offsets (groups + 1,) int32 on the device.
    """
    typ = _type_of(P, "P")
    out = _type_of(D, "D")
    if P.dim() != 2 or Q.dim() != 2 or D.dim() != 3:
        raise ValueError("P and Q must have two and D three dimensions")
    rows, M = P.shape
    N = Q.shape[1]
    groups = D.shape[0]
    dtype = P.dtype
    dev = _index_of(P, "P")
    ldp = _typed_ld(P, rows, M, "P", dtype, dev)
    ldq = _typed_ld(Q, rows, N, "Q", dtype, dev)
    ldd, stride_d = _stacked_ld(D, (groups, M, N), "D", D.dtype, dev)
    off = _flat(offsets, (groups + 1,), "offsets", _i32, dev)
    _call(load().sgemm_grouped_wgrad, "sgemm_grouped_wgrad", dev, stream, typ, groups, rows, M, N,
          alpha, P.data_ptr(), ldp, Q.data_ptr(), ldq, off, beta, out, D.data_ptr(), ldd, stride_d)


def sgemv_w4_tensors(X, Q, scales, Y, group, zeros=None, experts=None, stream=None) -> None:
    """Y[p] = X[p // repeat] @ dequantised(Q).T for a few tokens, weights in 4 bits.

    X (tokens, K) and Y (pairs, N), float32 or bfloat16, pairs = repeat *
    tokens; Q (N, ceil(K / 2)) uint8, the lower half of a byte first; scales
    (N, ceil(K / group)) of X's type and zeros the same shape in uint8, any
    value (None: 8).
    With experts (pairs,) int32 on the device, Q, scales and zeros have a
    leading dimension of experts and row p uses those of experts[p] (negative:
    a row of zeros).
    """
    typ = _type_of(X, "X")
    if X.dim() != 2 or Y.dim() != 2:
        raise ValueError("X and Y must have two dimensions")
    tokens, K = X.shape
    pairs, N = Y.shape
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    if pairs and (tokens == 0 or pairs % tokens):
        raise ValueError(f"Y has {pairs} rows, not a multiple of X's {tokens}")
    repeat = pairs // tokens if tokens and pairs else 1
    nbytes, ngroups = (K + 1) // 2, -(-K // group)
    dtype = X.dtype
    dev = _index_of(X, "X")
    ldx = _typed_ld(X, tokens, K, "X", dtype, dev)
    ldy = _typed_ld(Y, pairs, N, "Y", dtype, dev)
    if experts is None:
        count, ids, stride_q = 1, 0, 0
        ldq = _typed_ld(Q, N, nbytes, "Q", _u8, dev)
        meta = (N, ngroups)
    else:
        if Q.dim() != 3:
            raise ValueError("with experts Q must have three dimensions")
        count = Q.shape[0]
        ldq, stride_q = _stacked_ld(Q, (count, N, nbytes), "Q", _u8, dev)
        ids = _flat(experts, (pairs,), "experts", _i32, dev)
        meta = (count, N, ngroups)
    s = _flat(scales, meta, "scales", dtype, dev)
    z = 0 if zeros is None else _flat(zeros, meta, "zeros", _u8, dev)
    _call(load().sgemv_w4, "sgemv_w4", dev, stream, typ, pairs, repeat, N, K, group, X.data_ptr(), ldx,
          Q.data_ptr(), ldq, stride_q, s, z, count, ids, Y.data_ptr(), ldy)


def plan_tensors(alpha, A, B, beta, C, transa=False, transb=False):
    """Kernel name and grid sgemm_tensors would use for these tensors."""
    M, N, K, lda, ldb = _shapes(A, B, transa, transb)
    with _on_device(C.device):
        rc, name, grid = sgemm_plan_ex(_op(transa), _op(transb), M, N, K, float(alpha),
                                       A.data_ptr(), lda, B.data_ptr(), ldb, float(beta),
                                       C.data_ptr(), _ld(C, M, N, "C"))
    _check("sgemm_plan_ex", rc)
    return name, grid


def check_status(stream=None, device=None) -> int:
    """Synchronise and read/clear the device status word; raise on a time-out."""
    import torch
    dev = device if device is not None else torch.cuda.current_device()
    with torch.cuda.device(dev):
        rc, bits = sgemm_check_status(_stream_handle(stream, dev))
    _check("sgemm_check_status", rc)
    return bits


def fp32_peak(target_ms: float = 200.0, stream=None, device=None, form: int = SGEMM_PEAK_FFMA):
    """Measured FP32 ceiling in one instruction form (SGEMM_PEAK_FFMA,
    SGEMM_PEAK_FFMA2, or SGEMM_PEAK_OUTER: the GEMM's register outer product
    without its loads): dict(gflops, ms, flops)."""
    import torch
    dev = device if device is not None else torch.cuda.current_device()
    with torch.cuda.device(dev):
        rc, g, m, f = sgemm_fp32_peak_ex(form, target_ms, _stream_handle(stream, dev))
    _check("sgemm_fp32_peak_ex", rc)
    return {"gflops": g, "ms": m, "flops": f}
