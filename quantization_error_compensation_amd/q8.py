"""Python binding of the 8-bit path (include/spear_ec_q8.h).

As in binding.py every spear_ec_q8_* function has the name of the C entry
point it calls, marshals its arguments and raises on a non-zero status; the
functions refuse tensors of another type, shape or layout, since the library
sees bare pointers.  Codes are int8 [rows, width] tensors, scales fp32 [rows].
"""
from __future__ import annotations

import ctypes

from .binding import SPEAR_EC_OUT_F32, _check, load_library
from .kv import _call

SPEAR_EC_Q8_GATED = 8
SPEAR_EC_Q8_GELU = 16

Q8_EXPORTED = (
    "spear_ec_q8_quantize", "spear_ec_q8_dequant_f32", "spear_ec_q8_rmsnorm",
    "spear_ec_q8_workspace_bytes", "spear_ec_q8_linear",
)


class spear_ec_q8_desc(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("flags", ctypes.c_int32)]


_q8_lib = _int8 = _bf16 = _f32 = _stream_of = _device_now = None


def _lib():
    global _q8_lib, _int8, _bf16, _f32, _stream_of, _device_now
    if _q8_lib is None:
        import torch
        lib = load_library()
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        DP = ctypes.POINTER(spear_ec_q8_desc)
        lib.spear_ec_q8_quantize.argtypes = [i32, i32, P, i32, i64, P, P, P]
        lib.spear_ec_q8_dequant_f32.argtypes = [i32, i32, P, P, P, P]
        lib.spear_ec_q8_rmsnorm.argtypes = [i32, i32, P, i64, P, P, P, ctypes.c_double, P, P, P, P]
        lib.spear_ec_q8_workspace_bytes.argtypes = [DP, i32]
        lib.spear_ec_q8_linear.argtypes = [DP, i32, P, P, P, P, P, P, sz, P]
        for name in Q8_EXPORTED:
            getattr(lib, name).restype = ctypes.c_int
        lib.spear_ec_q8_workspace_bytes.restype = sz
        _int8, _bf16, _f32 = torch.int8, torch.bfloat16, torch.float32
        _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _device_now = getattr(torch._C, "_cuda_getDevice", None)
        _q8_lib = lib
    return _q8_lib


_ACTS = {"none": 0, "silu": SPEAR_EC_Q8_GATED, "gelu": SPEAR_EC_Q8_GATED | SPEAR_EC_Q8_GELU}


def make_q8_desc(d_in: int, d_out: int, act: str = "none", out_f32: bool = False) -> spear_ec_q8_desc:
    """A plain product (act "none") or a gated one ("silu", "gelu"), whose
    weights have 2 * d_out rows: first those of the activated projection."""
    if act not in _ACTS:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}")
    return spear_ec_q8_desc(d_in, d_out, _ACTS[act] | (SPEAR_EC_OUT_F32 if out_f32 else 0))


def q8_weight_shape(desc):
    """Shape of a product's weight codes; their scales have one element a row."""
    return desc.d_out * (2 if desc.flags & SPEAR_EC_Q8_GATED else 1), desc.d_in


def alloc_q8(rows, width, device="cuda"):
    """Device tensors for `rows` quantized rows: codes (int8), scales (fp32)."""
    import torch
    return (torch.empty((rows, width), dtype=torch.int8, device=device),
            torch.empty(rows, dtype=torch.float32, device=device))


def alloc_q8_workspace(desc, max_tokens, device="cuda"):
    """Zero-filled workspace for products of up to max_tokens tokens."""
    import torch
    n = spear_ec_q8_workspace_bytes(desc, max_tokens)
    if n == 0:
        raise ValueError("invalid desc or token count")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def spear_ec_q8_workspace_bytes(desc, max_tokens: int) -> int:
    if int(max_tokens) >> 31:   # ctypes would keep its low 32 bits, here and below
        return 0
    return int(_lib().spear_ec_q8_workspace_bytes(ctypes.byref(desc), int(max_tokens)))


# Single-token calls take a few microseconds on the GPU, so the checks below are
# written out in one expression a call: a helper for each tensor costs a third
# of a microsecond apiece.
def _run(fn, dev, stream, *args):
    """fn on the device, on the stream (by default the device's current one)."""
    if stream is None and dev >= 0 and dev == _device_now():
        status = fn(*args, _stream_of(dev))
        if status:
            _check(status)
    else:
        _call(fn, dev, stream, *args)


def _too_large():
    raise ValueError("rows and columns must be fewer than 2^31")


def _sizes(x, shape, name):
    """Rows, columns and row stride of a matrix whose rows may be strided."""
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    rows, width = shape
    if (rows | width) >> 31:
        _too_large()
    if width > 1 and x.stride(1) != 1:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    return rows, width, x.stride(0) if rows > 1 else width


def spear_ec_q8_quantize(x, codes, scales, stream=None):
    """Quantize the rows of x (bf16 or fp32 [rows, width], rows may be strided)."""
    lib = _q8_lib or _lib()
    shape, dev, kind = x.shape, x.get_device(), x.dtype
    rows, width, stride = _sizes(x, shape, "x")
    if (kind is not _bf16 and kind is not _f32) or codes.dtype is not _int8 or scales.dtype is not _f32 or \
            codes.shape != shape or scales.shape != shape[:1] or codes.get_device() != dev or \
            scales.get_device() != dev or not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError("x must be bf16 or fp32, codes contiguous int8 of x's shape and scales contiguous "
                         "fp32 with an element a row, on one device")
    _run(lib.spear_ec_q8_quantize, dev, stream, rows, width, x.data_ptr(), kind is _f32, stride,
         codes.data_ptr(), scales.data_ptr())


def spear_ec_q8_dequant_f32(codes, scales, out, stream=None):
    """Quantized rows as fp32 values [rows, width]."""
    lib = _q8_lib or _lib()
    shape, dev = codes.shape, codes.get_device()
    if len(shape) != 2 or codes.dtype is not _int8 or scales.dtype is not _f32 or out.dtype is not _f32 or \
            scales.shape != shape[:1] or out.shape != shape or scales.get_device() != dev or \
            out.get_device() != dev or not codes.is_contiguous() or not scales.is_contiguous() or \
            not out.is_contiguous():
        raise ValueError("codes must be a contiguous int8 matrix, scales fp32 with an element a row and out "
                         "fp32 of codes' shape, contiguous on one device")
    rows, width = shape
    if (rows | width) >> 31:
        _too_large()
    _run(lib.spear_ec_q8_dequant_f32, dev, stream, rows, width, codes.data_ptr(), scales.data_ptr(),
         out.data_ptr())


def _rows_like(t, shape, dev, name):
    """Pointer of a contiguous bf16 matrix, None for None."""
    if t is None:
        return None
    if t.dtype is not _bf16 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous bf16 of x's shape, on x's device")
    return t.data_ptr()


def spear_ec_q8_rmsnorm(x, residual, sum, weight, eps, y=None, codes=None, scales=None, stream=None):
    """Norm of the rows of x, or of x + residual, which goes to sum (both may
    be None); to y (bf16) and/or quantized to codes and scales."""
    lib = _q8_lib or _lib()
    shape, dev = x.shape, x.get_device()
    rows, width, stride = _sizes(x, shape, "x")
    if x.dtype is not _bf16 or weight.dtype is not _bf16 or weight.shape != shape[1:] or \
            weight.get_device() != dev or not weight.is_contiguous():
        raise ValueError("x must be bf16 and weight contiguous bf16 with an element a column, on one device")
    cp = sp = None
    if codes is not None and scales is not None:
        if codes.dtype is not _int8 or scales.dtype is not _f32 or codes.shape != shape or \
                scales.shape != shape[:1] or codes.get_device() != dev or scales.get_device() != dev or \
                not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes must be contiguous int8 of x's shape and scales contiguous fp32 with an "
                             "element a row, on x's device")
        cp, sp = codes.data_ptr(), scales.data_ptr()
    elif codes is not None or scales is not None:
        raise ValueError("codes and scales are given together or not at all")
    _run(lib.spear_ec_q8_rmsnorm, dev, stream, rows, width, x.data_ptr(), stride,
         _rows_like(residual, shape, dev, "residual"), _rows_like(sum, shape, dev, "sum"), weight.data_ptr(), eps,
         _rows_like(y, shape, dev, "y"), cp, sp)


def spear_ec_q8_linear(desc, xq, xs, wq, ws, y, workspace, stream=None):
    """y = act-gated or plain product of quantized rows: xq int8 [tokens, d_in]
    with scales xs, wq int8 of q8_weight_shape(desc) with scales ws, y bf16 (or
    fp32) [tokens, d_out]."""
    lib = _q8_lib or _lib()
    shape, dev, K, N, flags = xq.shape, xq.get_device(), desc.d_in, desc.d_out, desc.flags
    rows = 2 * N if flags & SPEAR_EC_Q8_GATED else N
    T = shape[0] if len(shape) else -1
    if xq.dtype is not _int8 or wq.dtype is not _int8 or xs.dtype is not _f32 or ws.dtype is not _f32 or \
            shape != (T, K) or wq.shape != (rows, K) or xs.shape != (T,) or ws.shape != (rows,) or \
            wq.get_device() != dev or xs.get_device() != dev or ws.get_device() != dev or \
            not xq.is_contiguous() or not wq.is_contiguous() or not xs.is_contiguous() or not ws.is_contiguous():
        raise ValueError(f"xq must be int8 [tokens, {K}], wq int8 [{rows}, {K}] and their scales fp32 with an "
                         "element a row, contiguous on one device")
    if y.dtype is not (_f32 if flags & SPEAR_EC_OUT_F32 else _bf16) or y.shape != (T, N) or \
            y.get_device() != dev or not y.is_contiguous():
        raise ValueError(f"y must be contiguous of shape [{T}, {N}], bf16 or with out_f32 fp32, on xq's device")
    if workspace is None or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous, on xq's device")
    if T >> 31:
        _too_large()
    _run(lib.spear_ec_q8_linear, dev, stream, desc, T, xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(),
         y.data_ptr(), workspace.data_ptr(), workspace.nbytes)
