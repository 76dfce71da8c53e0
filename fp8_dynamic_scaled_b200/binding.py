"""ctypes binding of libfp8.so -- argument marshalling only.

Every function here has the name of the C entry point it calls (include/fp8.h)
and does nothing but check tensor types, turn torch tensors into device
pointers and raise on a non-zero status.  All arithmetic runs in the CUDA
kernels of libfp8.so; there is no CPU or PyTorch fallback, and importing this
module fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m fp8_dynamic_scaled_b200.build` "
                      "(the FP8 path has no fallback)")

_lib = ctypes.CDLL(LIB_PATH)

# enums (include/fp8.h)
FP8_E4M3, FP8_E5M2 = 0, 1
FP8_SCALE_TENSOR, FP8_SCALE_ROW, FP8_SCALE_BLOCK_1x128 = 0, 1, 2
FP8_SCALE_BLOCK_128x128, FP8_SCALE_MX32, FP8_SCALE_DELAYED = 3, 4, 5
FP8_OK, FP8_ERR_INVALID_ARG, FP8_ERR_ALIGNMENT, FP8_ERR_UNSUPPORTED_DEVICE = 0, 1, 2, 3
FP8_ERR_NONFINITE, FP8_ERR_TIMEOUT, FP8_ERR_CUDA, FP8_ERR_WORKSPACE = 4, 5, 6, 7

EXPORTED = ("fp8_abi_version", "fp8_status_string", "fp8_device_check", "fp8_workspace_size",
            "fp8_quantize", "fp8_scaled_gemm", "fp8_linear_forward", "fp8_linear_forward_noalloc",
            "fp8_amax", "fp8_quantize_with_amax", "fp8_scaled_gemm_ex", "fp8_linear_forward_ex",
            "fp8_weight_only_linear", "fp8_scaled_gemm_act", "fp8_linear_forward_act", "fp8_rmsnorm_quantize",
            "fp8_kv_append", "fp8_kv_attention", "fp8_kv_attention_workspace_size",
            "fp8_testing_set_wait_limit_ns", "fp8_testing_encode_f32_range")
FP8_WEIGHT_ONLY_MAX_TOKENS = 64
FP8_NOALLOC_SCRATCH_BYTES = 4194304
FP8_RMSNORM_MAX_COLS = 32768
FP8_ACT_NONE, FP8_ACT_RELU, FP8_ACT_GELU, FP8_ACT_GELU_TANH, FP8_ACT_SILU = 0, 1, 2, 3, 4


class fp8_history_t(ctypes.Structure):
    _fields_ = [("ring_dev", ctypes.c_void_p), ("len", ctypes.c_int32), ("step", ctypes.c_int64),
                ("pending_dev", ctypes.c_void_p), ("ticket_dev", ctypes.c_void_p)]


class fp8_epilogue_t(ctypes.Structure):
    _fields_ = [("bias_dev", ctypes.c_void_p), ("amax_dev", ctypes.c_void_p), ("yq_dev", ctypes.c_void_p),
                ("yq_scale_dev", ctypes.c_void_p), ("yq_fmt", ctypes.c_int32), ("ldq", ctypes.c_int64)]


class fp8_epilogue_act_t(ctypes.Structure):
    _fields_ = [("base", fp8_epilogue_t), ("activation", ctypes.c_int32), ("residual_dev", ctypes.c_void_p),
                ("ldres", ctypes.c_int64)]


class fp8_kv_cache_t(ctypes.Structure):
    _fields_ = [("k_dev", ctypes.c_void_p), ("v_dev", ctypes.c_void_p), ("k_scale_dev", ctypes.c_void_p),
                ("v_scale_dev", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("fmt", ctypes.c_int32),
                ("page_table_dev", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("kv_lens_dev", ctypes.c_void_p), ("batch", ctypes.c_int32)]


_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_lib.fp8_abi_version.restype, _lib.fp8_abi_version.argtypes = _I32, []
_lib.fp8_status_string.restype, _lib.fp8_status_string.argtypes = ctypes.c_char_p, [_I32]
_lib.fp8_device_check.restype, _lib.fp8_device_check.argtypes = _I32, []
_lib.fp8_workspace_size.restype = _SZ
_lib.fp8_workspace_size.argtypes = [_I32, _I64, _I64, _I64, _I32]
_lib.fp8_quantize.restype = _I32
_lib.fp8_quantize.argtypes = [_P, _I64, _I64, _I64, _I32, _I32, _P, _P, ctypes.POINTER(fp8_history_t), _P, _P,
                              _P, _SZ, _P]
_lib.fp8_scaled_gemm.restype = _I32
_lib.fp8_scaled_gemm.argtypes = [_P, _P, _I32, _I32, _P, _P, _I32, _I32, _I64, _I64, _I64, _P, _I64, _P, _P,
                                 _SZ, _P]
_lib.fp8_linear_forward.restype = _I32
_lib.fp8_linear_forward.argtypes = [_P, _I64, _I64, _I64, _I32, _I32, ctypes.POINTER(fp8_history_t), _P, _P,
                                    _I32, _I32, _I64, _P, _I64, _P, _P, _SZ, _P]
_lib.fp8_amax.restype = _I32
_lib.fp8_amax.argtypes = [_P, _I64, _I64, _I64, _P, _P, _P, _SZ, _P]
_lib.fp8_quantize_with_amax.restype = _I32
_lib.fp8_quantize_with_amax.argtypes = [_P, _I64, _I64, _I64, _I32, _P, _P, _P, _P, _P, _P]
_lib.fp8_scaled_gemm_ex.restype = _I32
_lib.fp8_scaled_gemm_ex.argtypes = [_P, _P, _I32, _I32, _P, _P, _I32, _I32, _I64, _I64, _I64, _P, _I64,
                                    ctypes.POINTER(fp8_epilogue_t), _P, _P, _SZ, _P]
_lib.fp8_linear_forward_ex.restype = _I32
_lib.fp8_linear_forward_ex.argtypes = [_P, _I64, _I64, _I64, _I32, _I32, ctypes.POINTER(fp8_history_t), _P, _P,
                                       _I32, _I32, _I64, _P, _I64, ctypes.POINTER(fp8_epilogue_t), _P, _P, _SZ,
                                       _P]
_lib.fp8_scaled_gemm_act.restype = _I32
_lib.fp8_scaled_gemm_act.argtypes = [_P, _P, _I32, _I32, _P, _P, _I32, _I32, _I64, _I64, _I64, _P, _I64,
                                     ctypes.POINTER(fp8_epilogue_act_t), _P, _P, _SZ, _P]
_lib.fp8_linear_forward_act.restype = _I32
_lib.fp8_linear_forward_act.argtypes = [_P, _I64, _I64, _I64, _I32, _I32, ctypes.POINTER(fp8_history_t), _P, _P,
                                        _I32, _I32, _I64, _P, _I64, ctypes.POINTER(fp8_epilogue_act_t), _P, _P, _SZ,
                                        _P]
_lib.fp8_rmsnorm_quantize.restype = _I32
_lib.fp8_rmsnorm_quantize.argtypes = [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, ctypes.c_float, _I32, _I32, _P, _P,
                                      _P, _P, _P, _P]
_lib.fp8_kv_append.restype = _I32
_lib.fp8_kv_append.argtypes = [ctypes.POINTER(fp8_kv_cache_t), _P, _I64, _P, _I64, _I64, _P, _I32, _P, _P]
_lib.fp8_kv_attention_workspace_size.restype = _SZ
_lib.fp8_kv_attention_workspace_size.argtypes = [_I32, _I32, _I32, _I32, _I32, _I64]
_lib.fp8_kv_attention.restype = _I32
_lib.fp8_kv_attention.argtypes = [ctypes.POINTER(fp8_kv_cache_t), _P, _I64, _I32, _I64, _P, _I32, _I64, ctypes.c_float,
                                  _P, _I64, _P, _P, _SZ, _P]
_lib.fp8_weight_only_linear.restype = _I32
_lib.fp8_weight_only_linear.argtypes = [_P, _I64, _I64, _I64, _P, _P, _I32, _I32, _I64, _P, _I64, _P, _P]
_lib.fp8_testing_set_wait_limit_ns.restype = None
_lib.fp8_testing_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
_lib.fp8_testing_encode_f32_range.restype = _I32
_lib.fp8_testing_encode_f32_range.argtypes = [ctypes.c_uint32, _I64, _I32, _P, _P]
_lib.fp8_linear_forward_noalloc.restype = _I32
_lib.fp8_linear_forward_noalloc.argtypes = [_P, _I64, _I64, _I64, _I32, _I32, ctypes.POINTER(fp8_history_t), _P,
                                            _P, _I32, _I32, _I64, _P, _I64, _P, _P]


class FP8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {fp8_status_string(status)} ({status})")
        self.status = status


def _check(rc: int, where: str):
    if rc != FP8_OK:
        raise FP8Error(rc, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        if torch.cuda.is_initialized():       # what current_stream() looks up, without building its object
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on_current_device(*tensors):
    """The library works on the current device; tensors elsewhere are refused here.  Given every tensor of a
    call whose address a kernel gets."""
    device = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -2
    for t in tensors:
        if t is not None and t.get_device() != device:            # -1: a host tensor
            raise ValueError("the tensors must be on the current CUDA device")


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


# ------------------------------------------------------------------ entry points
def fp8_abi_version() -> int:
    return _lib.fp8_abi_version()


def fp8_status_string(status: int) -> str:
    return _lib.fp8_status_string(status).decode()


def fp8_device_check() -> int:
    return _lib.fp8_device_check()


def fp8_testing_set_wait_limit_ns(ns: int) -> None:
    """Testing hook (include/fp8_testing.h): limit of each GEMM pipeline wait; 0 = default."""
    _lib.fp8_testing_set_wait_limit_ns(int(ns))


def fp8_testing_encode_f32_range(first_bits: int, q, fmt: int, *, stream=None) -> None:
    """Testing hook (include/fp8_testing.h): q[i] = encode step of the fp32 value with bit
    pattern first_bits + i, for every byte of the uint8 device tensor q."""
    if q.dtype != torch.uint8 or not q.is_contiguous():
        raise TypeError("q must be a contiguous uint8 tensor")
    _check(_lib.fp8_testing_encode_f32_range(int(first_bits), q.numel(), fmt, _ptr(q), _stream(stream)),
           "fp8_testing_encode_f32_range")


def fp8_workspace_size(which: int, M: int, N: int, K: int, mode: int) -> int:
    return _lib.fp8_workspace_size(which, M, N, K, mode)


class History:
    """Device state of delayed scaling: ring[len], pending, ticket (all zero at step 0)."""

    def __init__(self, length: int = 16, device="cuda"):
        self.ring = torch.zeros(length, dtype=torch.float32, device=device)
        self.pending = torch.zeros(1, dtype=torch.float32, device=device)
        self.ticket = torch.zeros(1, dtype=torch.int32, device=device)
        self.c = fp8_history_t(self.ring.data_ptr(), length, 0, self.pending.data_ptr(), self.ticket.data_ptr())

    @property
    def step(self) -> int:
        return self.c.step


def fp8_quantize(x, fmt, mode, q, scale, *, hist: History | None = None, dequant=None, dev_status=None,
                 workspace=None, stream=None):
    """Quantize bf16 x [rows, cols] (row stride x.stride(0)) into q, scale (and dequant)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or (x.numel() and x.stride(1) != 1):
        raise TypeError("x must be a 2-D bf16 tensor with unit column stride")
    if q.dtype != torch.uint8:
        raise TypeError("q must be uint8")
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    rc = _lib.fp8_quantize(_ptr(x), rows, cols, ld, fmt, mode, _ptr(q), _ptr(scale),
                           ctypes.byref(hist.c) if hist is not None else None, _ptr(dequant), _ptr(dev_status),
                           _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "fp8_quantize")


def fp8_scaled_gemm(a, a_scale, a_mode, fmt_a, b, b_scale, b_mode, fmt_b, y, *, dev_status=None,
                    workspace=None, stream=None):
    """y[M, N] (bf16, row stride y.stride(0)) = scaled a[M, K] . b[N, K]^T."""
    if a.dtype != torch.uint8 or b.dtype != torch.uint8 or y.dtype != torch.bfloat16:
        raise TypeError("a, b must be uint8 codes and y bf16")
    M, K = a.shape
    N = b.shape[0]
    ldy = y.stride(0) if y.shape[0] > 1 else y.shape[1]
    rc = _lib.fp8_scaled_gemm(_ptr(a), _ptr(a_scale), a_mode, fmt_a, _ptr(b), _ptr(b_scale), b_mode, fmt_b,
                              M, N, K, _ptr(y), ldy, _ptr(dev_status), _ptr(workspace), _nbytes(workspace),
                              _stream(stream))
    _check(rc, "fp8_scaled_gemm")


def fp8_linear_forward(x, x_fmt, x_mode, w, w_scale, w_mode, w_fmt, y, workspace, *, hist: History | None = None,
                       dev_status=None, stream=None):
    """y = FP8 linear(x): quantize x with x_mode into the workspace, then the scaled GEMM with w."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.uint8 or y.dtype != torch.bfloat16:
        raise TypeError("x bf16, w uint8 codes, y bf16")
    M, K = x.shape
    N = w.shape[0]
    ldx = x.stride(0) if M > 1 else K
    ldy = y.stride(0) if y.shape[0] > 1 else y.shape[1]
    rc = _lib.fp8_linear_forward(_ptr(x), M, K, ldx, x_fmt, x_mode,
                                 ctypes.byref(hist.c) if hist is not None else None, _ptr(w), _ptr(w_scale),
                                 w_mode, w_fmt, N, _ptr(y), ldy, _ptr(dev_status), _ptr(workspace),
                                 _nbytes(workspace), _stream(stream))
    _check(rc, "fp8_linear_forward")


def fp8_amax(x, amax, *, dev_status=None, workspace=None, stream=None):
    """amax[0] (device fp32) = max |x| over bf16 x [rows, cols]."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or (x.numel() and x.stride(1) != 1):
        raise TypeError("x must be a 2-D bf16 tensor with unit column stride")
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    rc = _lib.fp8_amax(_ptr(x), rows, cols, ld, _ptr(amax), _ptr(dev_status), _ptr(workspace), _nbytes(workspace),
                       _stream(stream))
    _check(rc, "fp8_amax")


def fp8_quantize_with_amax(x, fmt, amax, q, scale, *, dequant=None, dev_status=None, stream=None):
    """Per-tensor cast of bf16 x with the scale of a given device amax: scale[0] = max(amax, 1e-12)/F_max."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or (x.numel() and x.stride(1) != 1):
        raise TypeError("x must be a 2-D bf16 tensor with unit column stride")
    if q.dtype != torch.uint8:
        raise TypeError("q must be uint8")
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    rc = _lib.fp8_quantize_with_amax(_ptr(x), rows, cols, ld, fmt, _ptr(amax), _ptr(q), _ptr(scale), _ptr(dequant),
                                     _ptr(dev_status), _stream(stream))
    _check(rc, "fp8_quantize_with_amax")


def _epilogue(N, bias, amax, yq, yq_scale, yq_fmt):
    if bias is None and amax is None and yq is None:
        return None
    if bias is not None and (bias.dtype != torch.bfloat16 or bias.numel() != N):
        raise TypeError("bias must be bf16 [N]")
    ldq = 0
    if yq is not None:
        if yq.dtype != torch.uint8:
            raise TypeError("yq must be uint8 codes")
        ldq = yq.stride(0) if yq.shape[0] > 1 else yq.shape[1]
    return fp8_epilogue_t(_ptr(bias), _ptr(amax), _ptr(yq), _ptr(yq_scale), yq_fmt, ldq)


def fp8_scaled_gemm_ex(a, a_scale, a_mode, fmt_a, b, b_scale, b_mode, fmt_b, y, *, bias=None, amax=None, yq=None,
                       yq_scale=None, yq_fmt=FP8_E4M3, dev_status=None, workspace=None, stream=None):
    """fp8_scaled_gemm with the epilogue options: bias [N] (bf16), amax (device fp32, max |y| folded in),
    yq [M, N] FP8 codes of y / yq_scale.  y may be None when yq is given."""
    if a.dtype != torch.uint8 or b.dtype != torch.uint8 or (y is not None and y.dtype != torch.bfloat16):
        raise TypeError("a, b must be uint8 codes and y bf16")
    M, K = a.shape
    N = b.shape[0]
    ldy = 0 if y is None else (y.stride(0) if y.shape[0] > 1 else y.shape[1])
    epi = _epilogue(N, bias, amax, yq, yq_scale, yq_fmt)
    rc = _lib.fp8_scaled_gemm_ex(_ptr(a), _ptr(a_scale), a_mode, fmt_a, _ptr(b), _ptr(b_scale), b_mode, fmt_b,
                                 M, N, K, _ptr(y), ldy, ctypes.byref(epi) if epi is not None else None,
                                 _ptr(dev_status), _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "fp8_scaled_gemm_ex")


def fp8_linear_forward_ex(x, x_fmt, x_mode, w, w_scale, w_mode, w_fmt, y, workspace, *, hist: History | None = None,
                          bias=None, amax=None, yq=None, yq_scale=None, yq_fmt=FP8_E4M3, dev_status=None,
                          stream=None):
    """fp8_linear_forward with the epilogue options of fp8_scaled_gemm_ex."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.uint8 or (y is not None and y.dtype != torch.bfloat16):
        raise TypeError("x bf16, w uint8 codes, y bf16")
    M, K = x.shape
    N = w.shape[0]
    ldx = x.stride(0) if M > 1 else K
    ldy = 0 if y is None else (y.stride(0) if y.shape[0] > 1 else y.shape[1])
    epi = _epilogue(N, bias, amax, yq, yq_scale, yq_fmt)
    rc = _lib.fp8_linear_forward_ex(_ptr(x), M, K, ldx, x_fmt, x_mode,
                                    ctypes.byref(hist.c) if hist is not None else None, _ptr(w), _ptr(w_scale),
                                    w_mode, w_fmt, N, _ptr(y), ldy, ctypes.byref(epi) if epi is not None else None,
                                    _ptr(dev_status), _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "fp8_linear_forward_ex")


def _check_gemm_act(M, N, K, w, y, bias, amax, yq, yq_scale):
    """Shapes and types of what the *_act calls take beside their first operand; returns y's row stride."""
    if w.dim() != 2 or w.shape[1] != K or not w.is_contiguous():
        raise TypeError(f"the weight must be dense uint8 codes [N, {K}]")
    ldy = 0
    for name, t in (("y", y), ("yq", yq)):
        if t is not None and (t.shape != (M, N) or (N > 1 and t.stride(1) != 1)):
            raise TypeError(f"{name} must be [{M}, {N}] with unit column stride")
    if y is not None:
        ldy = y.stride(0) if M > 1 else N
    if bias is not None and not bias.is_contiguous():
        raise TypeError("bias must be dense bf16 [N]")
    for name, t in (("amax", amax), ("yq_scale", yq_scale)):
        if t is not None and (t.dtype is not torch.float32 or t.numel() < 1):
            raise TypeError(f"{name} must be a device fp32")
    return ldy


def _check_scale(name, scale, mode, rows, cols):
    """A buffer of the mode's scales for [rows, cols] codes (a mode that does not exist is the library's to refuse)."""
    if scale is not None and FP8_SCALE_TENSOR <= mode <= FP8_SCALE_DELAYED:
        one_byte = mode == FP8_SCALE_MX32                          # uint8 or float8_e8m0fnu
        if (scale.element_size() != 1 if one_byte else scale.dtype is not torch.float32) or not scale.is_contiguous() or \
                scale.numel() < math.prod(scale_shape(mode, rows, cols)):
            raise TypeError(f"{name} must be a dense buffer of the mode's scales")


def _epilogue_act(M, N, bias, activation, residual, amax, yq, yq_scale, yq_fmt):
    epi = fp8_epilogue_act_t()
    base = _epilogue(N, bias, amax, yq, yq_scale, yq_fmt)
    if base is not None:
        epi.base = base
    epi.activation = activation
    if residual is not None:
        stride = residual.stride()
        if residual.dtype is not torch.bfloat16 or residual.shape != (M, N) or (N > 1 and stride[1] != 1):
            raise TypeError("residual must be bf16 [M, N] with unit column stride")
        epi.residual_dev, epi.ldres = residual.data_ptr(), stride[0] if M > 1 else N
    return epi


def fp8_scaled_gemm_act(a, a_scale, a_mode, fmt_a, b, b_scale, b_mode, fmt_b, y, *, bias=None,
                        activation=FP8_ACT_NONE, residual=None, amax=None, yq=None, yq_scale=None, yq_fmt=FP8_E4M3,
                        dev_status=None, workspace=None, stream=None):
    """y = act(scaled a . b^T + bias) + residual, with the options of fp8_scaled_gemm_ex.  residual
    (bf16 [M, N]) may be y itself; y may be None when yq is given."""
    if a.dtype != torch.uint8 or b.dtype != torch.uint8 or (y is not None and y.dtype != torch.bfloat16):
        raise TypeError("a, b must be uint8 codes and y bf16")
    if a.dim() != 2 or not a.is_contiguous():
        raise TypeError("a must be dense uint8 codes [M, K]")
    M, K = a.shape
    N = b.shape[0]
    ldy = _check_gemm_act(M, N, K, b, y, bias, amax, yq, yq_scale)
    epi = _epilogue_act(M, N, bias, activation, residual, amax, yq, yq_scale, yq_fmt)
    _on_current_device(a, a_scale, b, b_scale, y, bias, residual, amax, yq, yq_scale, dev_status)
    if K and N:
        _check_scale("a_scale", a_scale, a_mode, M, K)
        _check_scale("b_scale", b_scale, b_mode, N, K)
    rc = _lib.fp8_scaled_gemm_act(_ptr(a), _ptr(a_scale), a_mode, fmt_a, _ptr(b), _ptr(b_scale), b_mode, fmt_b,
                                  M, N, K, _ptr(y), ldy, ctypes.byref(epi), _ptr(dev_status), _ptr(workspace),
                                  _nbytes(workspace), _stream(stream))
    _check(rc, "fp8_scaled_gemm_act")


def fp8_linear_forward_act(x, x_fmt, x_mode, w, w_scale, w_mode, w_fmt, y, workspace, *, hist: History | None = None,
                           bias=None, activation=FP8_ACT_NONE, residual=None, amax=None, yq=None, yq_scale=None,
                           yq_fmt=FP8_E4M3, dev_status=None, stream=None):
    """fp8_linear_forward with the epilogue of fp8_scaled_gemm_act."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.uint8 or (y is not None and y.dtype != torch.bfloat16):
        raise TypeError("x bf16, w uint8 codes, y bf16")
    if x.dim() != 2:
        raise TypeError("x must be a 2-D bf16 tensor with unit column stride")
    M, K = x.shape
    N = w.shape[0]
    ldx = _rows_of(x, "x", M, K)
    ldy = _check_gemm_act(M, N, K, w, y, bias, amax, yq, yq_scale)
    epi = _epilogue_act(M, N, bias, activation, residual, amax, yq, yq_scale, yq_fmt)
    _on_current_device(x, w, w_scale, y, workspace, bias, residual, amax, yq, yq_scale, dev_status)
    if hist is not None:
        _on_current_device(hist.ring, hist.pending, hist.ticket)
    if K and N:
        _check_scale("w_scale", w_scale, w_mode, N, K)
    rc = _lib.fp8_linear_forward_act(_ptr(x), M, K, ldx, x_fmt, x_mode,
                                     ctypes.byref(hist.c) if hist is not None else None, _ptr(w), _ptr(w_scale),
                                     w_mode, w_fmt, N, _ptr(y), ldy, ctypes.byref(epi), _ptr(dev_status),
                                     _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "fp8_linear_forward_act")


def _rows_of(t, name, rows, cols):
    """Row stride of a bf16 [rows, cols] tensor with unit column stride."""
    stride = t.stride()
    if t.dtype is not torch.bfloat16 or t.shape != (rows, cols) or (rows and cols and stride[1] != 1):
        raise TypeError(f"{name} must be bf16 [{rows}, {cols}] with unit column stride")
    return stride[0] if rows > 1 and cols else cols


def fp8_rmsnorm_quantize(x, weight, eps, fmt, mode, q, scale, *, residual=None, sum_out=None, y=None, amax=None,
                         dev_status=None, stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight; (q, scale) = y quantized (ROW, BLOCK_1x128,
    MX32, or TENSOR with the scale of the device amax).  sum_out (may be x or residual) receives h, y the
    normalised rows, both bf16."""
    if x.dim() != 2:
        raise TypeError("x must be a 2-D bf16 tensor with unit column stride")
    rows, cols = x.shape
    ldx = _rows_of(x, "x", rows, cols)
    ldr = 0 if residual is None else _rows_of(residual, "residual", rows, cols)
    lds = 0 if sum_out is None else _rows_of(sum_out, "sum_out", rows, cols)
    if weight is not None and (weight.dtype != torch.bfloat16 or weight.numel() != cols or not weight.is_contiguous()):
        raise TypeError("weight must be bf16 [cols]")
    if q.dtype is not torch.uint8 or q.shape != (rows, cols) or not q.is_contiguous():
        raise TypeError("q must be dense uint8 [rows, cols]")
    mx = mode == FP8_SCALE_MX32
    need = rows if mode == FP8_SCALE_ROW else rows * (cols // 32) if mx else rows * -(-cols // 128) \
        if mode == FP8_SCALE_BLOCK_1x128 else 1
    if scale.dtype is not (torch.uint8 if mx else torch.float32) or not scale.is_contiguous() or scale.numel() < need:
        raise TypeError("scale must be a dense buffer of the mode's scales")
    if y is not None and (y.dtype is not torch.bfloat16 or y.shape != (rows, cols) or not y.is_contiguous()):
        raise TypeError("y must be dense bf16 [rows, cols]")
    if amax is not None and amax.dtype is not torch.float32:
        raise TypeError("amax must be fp32")
    _on_current_device(x, weight, residual, sum_out, q, scale, y, amax, dev_status)
    rc = _lib.fp8_rmsnorm_quantize(_ptr(x), rows, cols, ldx, _ptr(residual), ldr, _ptr(sum_out), lds, _ptr(weight),
                                   float(eps), fmt, mode, _ptr(amax), _ptr(q), _ptr(scale), _ptr(y), _ptr(dev_status),
                                   _stream(stream))
    _check(rc, "fp8_rmsnorm_quantize")


class KVCache:
    """A paged FP8 KV cache: uint8 codes k, v [num_pages, kv_heads, page_size, head_dim] and fp32 scales
    k_scale, v_scale [num_pages, kv_heads], dense, kept by the caller."""

    def __init__(self, k, v, k_scale, v_scale, fmt=FP8_E4M3):
        for t in (k, v):
            if t.dtype != torch.uint8 or t.dim() != 4 or t.shape != k.shape or not t.is_contiguous():
                raise TypeError("k, v must be dense uint8 codes [num_pages, kv_heads, page_size, head_dim]")
        for t in (k_scale, v_scale):
            if t.dtype != torch.float32 or t.shape != k.shape[:2] or not t.is_contiguous():
                raise TypeError("k_scale, v_scale must be dense fp32 [num_pages, kv_heads]")
        if len({t.get_device() for t in (k, v, k_scale, v_scale)}) != 1:
            raise ValueError("k, v and their scales must be on one device")
        self.k, self.v, self.k_scale, self.v_scale, self.fmt = k, v, k_scale, v_scale, fmt
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.c = fp8_kv_cache_t(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), self.num_pages,
                                self.page_size, self.kv_heads, self.head_dim, fmt, None, 0, 0, None, 0)

    @classmethod
    def empty(cls, num_pages, kv_heads, page_size, head_dim, fmt=FP8_E4M3, device="cuda"):
        """A cache with no tokens yet."""
        shape = (num_pages, kv_heads, page_size, head_dim)
        codes = [torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales, fmt)

    def view(self, page_table, kv_lens):
        """The C descriptor with a batch's page table [batch, max_pages] and lengths [batch] (int32)."""
        shape, stride = page_table.shape, page_table.stride()
        if page_table.dtype is not torch.int32 or len(shape) != 2 or (shape[0] and shape[1] and stride[1] != 1):
            raise TypeError("page_table must be int32 [batch, max_pages] with unit column stride")
        batch, pages = shape
        if kv_lens.dtype is not torch.int32 or kv_lens.shape != (batch,) or not kv_lens.is_contiguous():
            raise TypeError("kv_lens must be int32 [batch]")
        c = fp8_kv_cache_t.from_buffer_copy(self.c)      # the call's own: calls of two threads may overlap
        c.page_table_dev, c.max_pages = page_table.data_ptr(), pages
        c.table_stride = stride[0] if batch > 1 and pages else pages
        c.kv_lens_dev, c.batch = kv_lens.data_ptr(), batch
        return c


def _head_rows(t, name, heads, dim):
    """Token stride of a bf16 [tokens, heads, dim] tensor whose heads are dense within a token."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not torch.bfloat16 or len(shape) != 3 or shape[1] != heads or shape[2] != dim or \
            (shape[0] and (stride[2] != 1 or (heads > 1 and stride[1] != dim))):
        raise TypeError(f"{name} must be bf16 [tokens, {heads}, {dim}], its heads dense within a token")
    return stride[0] if shape[0] > 1 else heads * dim


def _cu_q(cu_q, batch):
    if cu_q is None:
        return None
    if cu_q.dtype is not torch.int32 or cu_q.shape != (batch + 1,) or not cu_q.is_contiguous():
        raise TypeError("cu_q must be int32 [batch + 1]")
    return cu_q.data_ptr()


def fp8_kv_append(k, v, cache: KVCache, page_table, kv_lens, *, cu_q=None, max_q_len=1, dev_status=None, stream=None):
    """Quantize the new tokens' k, v (bf16 [tokens, kv_heads, head_dim]) into their pages: rows
    [cu_q[b], cu_q[b + 1]) are the last tokens of sequence b, whose length with them is kv_lens[b]."""
    ldk = _head_rows(k, "k", cache.kv_heads, cache.head_dim)
    ldv = _head_rows(v, "v", cache.kv_heads, cache.head_dim)
    if k.shape[0] != v.shape[0]:
        raise TypeError("k and v must have as many tokens")
    c = cache.view(page_table, kv_lens)
    cu = _cu_q(cu_q, c.batch)
    _on_current_device(k, v, cache.k, page_table, kv_lens, cu_q, dev_status)    # the cache's tensors share a device
    _check(_lib.fp8_kv_append(ctypes.byref(c), _ptr(k), ldk, _ptr(v), ldv, k.shape[0], cu, max_q_len, _ptr(dev_status),
                              _stream(stream)), "fp8_kv_append")


def fp8_kv_attention_workspace_size(batch: int, q_heads: int, kv_heads: int, head_dim: int, max_q_len: int,
                                    max_kv_len: int) -> int:
    return _lib.fp8_kv_attention_workspace_size(batch, q_heads, kv_heads, head_dim, max_q_len, max_kv_len)


def kv_attention_workspace(q, cache: KVCache, batch: int, max_q_len: int, max_kv_len: int):
    """Workspace of fp8_kv_attention for q [tokens, q_heads, head_dim], or None when it needs none."""
    n = fp8_kv_attention_workspace_size(batch, q.shape[1], cache.kv_heads, cache.head_dim, max_q_len, max_kv_len)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def fp8_kv_attention(q, cache: KVCache, page_table, kv_lens, out, *, max_kv_len, cu_q=None, max_q_len=1,
                     softmax_scale=None, workspace=None, dev_status=None, stream=None):
    """Causal attention of q (bf16 [tokens, q_heads, head_dim]) over the cache into out (the same shape, not q);
    softmax_scale defaults to head_dim ** -0.5."""
    if q.dim() != 3 or out.shape != q.shape:
        raise TypeError("q and out must be bf16 [tokens, q_heads, head_dim]")
    if out.data_ptr() == q.data_ptr() and q.numel():
        raise ValueError("out must not be q: heads of a row are written while others are still read")
    tokens, heads, dim = q.shape
    ldq = _head_rows(q, "q", heads, cache.head_dim)
    ldo = _head_rows(out, "out", heads, cache.head_dim)
    c = cache.view(page_table, kv_lens)
    cu = _cu_q(cu_q, c.batch)
    scale = dim ** -0.5 if softmax_scale is None else float(softmax_scale)
    _on_current_device(q, out, cache.k, page_table, kv_lens, cu_q, workspace, dev_status)
    _check(_lib.fp8_kv_attention(ctypes.byref(c), _ptr(q), ldq, heads, tokens, cu, max_q_len,
                                 max_kv_len, scale, _ptr(out), ldo, _ptr(dev_status), _ptr(workspace),
                                 _nbytes(workspace), _stream(stream)), "fp8_kv_attention")


def fp8_weight_only_linear(x, w, w_scale, w_mode, w_fmt, y, *, dev_status=None, stream=None):
    """y [M, N] bf16 = x [M, K] bf16 times the FP8 weight w [N, K] (codes) with its scale."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.uint8 or y.dtype != torch.bfloat16:
        raise TypeError("x bf16, w uint8 codes, y bf16")
    M, K = x.shape
    N = w.shape[0]
    ldx = x.stride(0) if M > 1 else K
    ldy = y.stride(0) if y.shape[0] > 1 else y.shape[1]
    rc = _lib.fp8_weight_only_linear(_ptr(x), M, K, ldx, _ptr(w), _ptr(w_scale), w_mode, w_fmt, N, _ptr(y), ldy,
                                     _ptr(dev_status), _stream(stream))
    _check(rc, "fp8_weight_only_linear")


def fp8_linear_forward_noalloc(x, x_fmt, x_mode, w, w_scale, w_mode, w_fmt, y, *, hist: History | None = None,
                               dev_status=None, stream=None):
    """fp8_linear_forward without a workspace argument, for callers that cannot allocate:
    the scratch is the library's fixed FP8_NOALLOC_SCRATCH_BYTES device array, shared by
    all calls (order overlapping calls on one stream)."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.uint8 or y.dtype != torch.bfloat16:
        raise TypeError("x bf16, w uint8 codes, y bf16")
    M, K = x.shape
    N = w.shape[0]
    ldx = x.stride(0) if M > 1 else K
    ldy = y.stride(0) if y.shape[0] > 1 else y.shape[1]
    rc = _lib.fp8_linear_forward_noalloc(_ptr(x), M, K, ldx, x_fmt, x_mode,
                                         ctypes.byref(hist.c) if hist is not None else None, _ptr(w),
                                         _ptr(w_scale), w_mode, w_fmt, N, _ptr(y), ldy, _ptr(dev_status),
                                         _stream(stream))
    _check(rc, "fp8_linear_forward_noalloc")


# ------------------------------------------------------------------ allocation helpers
def scale_shape(mode: int, rows: int, cols: int):
    if mode in (FP8_SCALE_TENSOR, FP8_SCALE_DELAYED):
        return (1,)
    if mode == FP8_SCALE_ROW:
        return (rows,)
    if mode == FP8_SCALE_BLOCK_1x128:
        return (rows, -(-cols // 128))
    if mode == FP8_SCALE_BLOCK_128x128:
        return (-(-rows // 128), -(-cols // 128))
    if mode == FP8_SCALE_MX32:
        return (rows, cols // 32)
    raise ValueError(mode)


def empty_quant_outputs(rows: int, cols: int, mode: int, device="cuda", dequant: bool = False):
    """Output buffers of fp8_quantize for a [rows, cols] input: (q, scale, dequant or None)."""
    q = torch.empty((rows, cols), dtype=torch.uint8, device=device)
    sdt = torch.uint8 if mode == FP8_SCALE_MX32 else torch.float32
    s = torch.empty(scale_shape(mode, rows, cols), dtype=sdt, device=device)
    d = torch.empty((rows, cols), dtype=torch.bfloat16, device=device) if dequant else None
    return q, s, d


def workspace_for(which: int, M: int, N: int, K: int, mode: int, device="cuda"):
    n = fp8_workspace_size(which, M, N, K, mode)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device)
