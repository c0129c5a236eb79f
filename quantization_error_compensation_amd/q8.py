"""Python binding of the 8-bit path (include/spear_ec_q8.h).

As in binding.py every spear_ec_q8_* function has the name of the C entry
point it calls, marshals its arguments and raises on a non-zero status; the
functions refuse tensors of another type, shape or layout, since the library
sees bare pointers.  Codes are int8 [rows, width] tensors, scales fp32 [rows].
"""
from __future__ import annotations

import ctypes

from .binding import SPEAR_EC_OUT_F32, load_library
from .kv import _call

SPEAR_EC_Q8_GATED = 8
SPEAR_EC_Q8_GELU = 16

Q8_EXPORTED = (
    "spear_ec_q8_quantize", "spear_ec_q8_dequant_f32", "spear_ec_q8_rmsnorm",
    "spear_ec_q8_workspace_bytes", "spear_ec_q8_linear",
)


class spear_ec_q8_desc(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("flags", ctypes.c_int32)]


_q8_lib = None


def _lib():
    global _q8_lib
    if _q8_lib is None:
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
    return int(_lib().spear_ec_q8_workspace_bytes(ctypes.byref(desc), int(max_tokens)))


def _matrix(t, dtype, shape, device, name):
    """Pointer of a contiguous matrix."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be contiguous {dtype} of shape {tuple(shape)} on one device "
                         "with the call's other tensors")
    return t.data_ptr()


def _rows(t, dtypes, name):
    """Shape, row stride and device of a matrix whose rows may be strided."""
    shape = t.shape
    if t.dtype not in dtypes or len(shape) != 2:
        raise ValueError(f"{name} must be a matrix of " + " or ".join(str(d) for d in dtypes))
    row, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return shape, row if shape[0] > 1 else shape[1], t.get_device()


def _codes(codes, scales, shape, device, name):
    import torch
    return (_matrix(codes, torch.int8, shape, device, name),
            _matrix(scales, torch.float32, shape[:1], device, name + "'s scales"))


def spear_ec_q8_quantize(x, codes, scales, stream=None):
    """Quantize the rows of x (bf16 or fp32 [rows, width], rows may be strided)."""
    import torch
    shape, stride, dev = _rows(x, (torch.bfloat16, torch.float32), "x")
    cp, sp = _codes(codes, scales, shape, dev, "codes")
    _call(_lib().spear_ec_q8_quantize, dev, stream, shape[0], shape[1], x.data_ptr(),
          x.dtype is torch.float32, stride, cp, sp)


def spear_ec_q8_dequant_f32(codes, scales, out, stream=None):
    """Quantized rows as fp32 values [rows, width]."""
    import torch
    shape, dev = codes.shape, codes.get_device()
    if len(shape) != 2:
        raise ValueError("codes must be a matrix")
    cp, sp = _codes(codes, scales, shape, dev, "codes")
    _call(_lib().spear_ec_q8_dequant_f32, dev, stream, shape[0], shape[1], cp, sp,
          _matrix(out, torch.float32, shape, dev, "out"))


def spear_ec_q8_rmsnorm(x, residual, sum, weight, eps, y=None, codes=None, scales=None, stream=None):
    """Norm of the rows of x, or of x + residual, which goes to sum (both may
    be None); to y (bf16) and/or quantized to codes and scales."""
    import torch
    bf16 = torch.bfloat16
    shape, stride, dev = _rows(x, (bf16,), "x")
    wp = _matrix(weight, bf16, shape[1:], dev, "weight")
    rp = _matrix(residual, bf16, shape, dev, "residual") if residual is not None else None
    up = _matrix(sum, bf16, shape, dev, "sum") if sum is not None else None
    yp = _matrix(y, bf16, shape, dev, "y") if y is not None else None
    cp = sp = None
    if codes is not None or scales is not None:
        if codes is None or scales is None:
            raise ValueError("codes and scales are given together or not at all")
        cp, sp = _codes(codes, scales, shape, dev, "codes")
    _call(_lib().spear_ec_q8_rmsnorm, dev, stream, shape[0], shape[1], x.data_ptr(), stride, rp, up,
          wp, eps, yp, cp, sp)


def spear_ec_q8_linear(desc, xq, xs, wq, ws, y, workspace, stream=None):
    """y = act-gated or plain product of quantized rows: xq int8 [tokens, d_in]
    with scales xs, wq int8 of q8_weight_shape(desc) with scales ws, y bf16 (or
    fp32) [tokens, d_out]."""
    import torch
    shape, dev = xq.shape, xq.get_device()
    if len(shape) != 2 or shape[1] != desc.d_in:
        raise ValueError("xq must be a matrix of d_in columns")
    flags = desc.flags
    xp, xsp = _codes(xq, xs, shape, dev, "xq")
    wp, wsp = _codes(wq, ws, torch.Size((desc.d_out * (2 if flags & SPEAR_EC_Q8_GATED else 1),
                                         desc.d_in)), dev, "wq")
    yp = _matrix(y, torch.float32 if flags & SPEAR_EC_OUT_F32 else torch.bfloat16,
                 torch.Size((shape[0], desc.d_out)), dev, "y")
    ok = workspace is not None and workspace.get_device() == dev and workspace.is_contiguous()
    if not ok:
        raise ValueError("the workspace must be contiguous, on one device with the call's tensors")
    _call(_lib().spear_ec_q8_linear, dev, stream, desc, shape[0], xp, xsp, wp, wsp, yp,
          workspace.data_ptr(), workspace.nbytes)
