"""Python binding of the 4-bit paged key/value cache (include/spear_ec_kv.h).

As in binding.py every spear_ec_kv_* function has the name of the C entry
point it calls, marshals its arguments and raises on a non-zero status.  Token
arrays are [tokens, heads, head_dim] tensors whose rows may be strided (slices
of one projection's output); the functions refuse tensors of another type,
shape or layout, since the library sees bare pointers.
"""
from __future__ import annotations

import ctypes

from .binding import SPEAR_EC_ZEROS, _check, load_library

SPEAR_EC_WS_BAD_PAGE = 2

KV_EXPORTED = (
    "spear_ec_kv_append", "spear_ec_kv_workspace_bytes", "spear_ec_kv_attention",
    "spear_ec_kv_dequant_f32",
)


class spear_ec_kv_desc(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class spear_ec_kv_batch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("q_offsets", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p)]


class spear_ec_kv_rope(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("rows", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


_kv_lib = None


def _lib():
    global _kv_lib
    if _kv_lib is None:
        lib = load_library()
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        DP, BP = ctypes.POINTER(spear_ec_kv_desc), ctypes.POINTER(spear_ec_kv_batch)
        lib.spear_ec_kv_append.argtypes = [DP, BP, P, i64, P, i64, P, i64,
                                           ctypes.POINTER(spear_ec_kv_rope), P, P, P, P, i64, P]
        lib.spear_ec_kv_append.restype = ctypes.c_int
        lib.spear_ec_kv_workspace_bytes.argtypes = [DP, i32, i32]
        lib.spear_ec_kv_workspace_bytes.restype = sz
        lib.spear_ec_kv_attention.argtypes = [DP, BP, P, i64, P, P, P, ctypes.c_float, i32, P, P, P,
                                              sz, P]
        lib.spear_ec_kv_attention.restype = ctypes.c_int
        lib.spear_ec_kv_dequant_f32.argtypes = [DP, BP, P, P, P, P, P, P]
        lib.spear_ec_kv_dequant_f32.restype = ctypes.c_int
        _kv_lib = lib
    return _kv_lib


def make_kv_desc(q_heads: int, kv_heads: int, head_dim: int, page_tokens: int, pages: int,
                 max_pages: int, zeros: bool) -> spear_ec_kv_desc:
    return spear_ec_kv_desc(q_heads, kv_heads, head_dim, page_tokens, pages, max_pages,
                            SPEAR_EC_ZEROS if zeros else 0)


def make_kv_batch(q_offsets, seq_lens, page_table, tokens: int) -> spear_ec_kv_batch:
    """The batch of int32 device tensors q_offsets [n + 1] (or None: one row a
    sequence), seq_lens [n] and page_table [n, max_pages]; keeps them alive."""
    import torch
    n = int(seq_lens.shape[0])
    shapes = ((q_offsets, (n + 1,)), (seq_lens, (n,)),
              (page_table, (n, int(page_table.shape[1]))))
    for t, shape in shapes:
        if t is None:
            continue
        if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"a batch array must be contiguous int32 of shape {shape}")
    if any(t is not None and t.get_device() != seq_lens.get_device() for t, _ in shapes):
        raise ValueError("the batch arrays must be on one device")
    b = spear_ec_kv_batch(n, int(tokens), None if q_offsets is None else q_offsets.data_ptr(),
                          seq_lens.data_ptr(), page_table.data_ptr())
    b.arrays = (q_offsets, seq_lens, page_table)
    return b


def kv_cache_shapes(desc):
    """Shapes of the cache arrays for a desc: (codes, scales, zeros or None)."""
    blocks = desc.page_tokens // 16
    head = (desc.pages, desc.kv_heads, blocks)
    return ((*head, 16 * desc.head_dim), (*head, 2, 16),
            (*head, 16) if desc.flags & SPEAR_EC_ZEROS else None)


def alloc_kv_cache(desc, device="cuda"):
    """Device tensors for a cache: codes (uint8), scales (fp16), zeros (uint8) or None."""
    import torch
    c, s, z = kv_cache_shapes(desc)
    return (torch.empty(c, dtype=torch.uint8, device=device),
            torch.empty(s, dtype=torch.float16, device=device),
            torch.empty(z, dtype=torch.uint8, device=device) if z else None)


def alloc_kv_workspace(desc, n_seqs, tokens, device="cuda"):
    """Zero-filled workspace for attention calls of up to n_seqs sequences and
    `tokens` rows."""
    import torch
    n = spear_ec_kv_workspace_bytes(desc, n_seqs, tokens)
    if n == 0:
        raise ValueError("invalid desc, sequence or token count")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def spear_ec_kv_workspace_bytes(desc, n_seqs: int, tokens: int) -> int:
    return int(_lib().spear_ec_kv_workspace_bytes(ctypes.byref(desc), int(n_seqs), int(tokens)))


def _call(fn, device, stream, *args):
    """fn on the device, on the stream (by default the device's current one)."""
    import torch
    if device < 0:
        raise ValueError("the tensors must be on the GPU")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if device == torch._C._cuda_getDevice():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status:
        _check(status)


def _rows(t, device, tokens, heads, dim, dtype, name, strided=True):
    """Pointer and row stride of a token array, checked against what the call
    will read or write."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 3 or shape[0] < tokens or shape[1] != heads or \
            shape[2] != dim or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} of shape [>= {tokens}, {heads}, {dim}] on the "
                         "cache's device")
    row, head, one = t.stride()
    if shape[0] <= 1:
        row = heads * dim
    if one != 1 or (head != dim and heads > 1) or (not strided and row != heads * dim):
        raise ValueError(f"{name}'s rows must be contiguous [{heads}, {dim}]")
    return t.data_ptr(), row


def _flat(t, device, elements, size):
    return t.numel() == elements and t.element_size() == size and t.is_contiguous() and \
        t.get_device() == device


def _cache(desc, batch, codes, scales, zeros):
    """Device and pointers of the cache arrays, checked against the desc, as is
    the batch."""
    device = codes.get_device()
    tokens = desc.pages * desc.kv_heads * desc.page_tokens
    ok = _flat(codes, device, tokens * desc.head_dim, 1) and _flat(scales, device, tokens * 2, 2)
    if desc.flags & SPEAR_EC_ZEROS:
        ok = ok and zeros is not None and _flat(zeros, device, tokens, 1)
    if not ok:
        raise ValueError("codes, scales and zeros must have the shapes of kv_cache_shapes(desc), "
                         "on one device")
    arrays = getattr(batch, "arrays", None)
    if arrays and (arrays[2].shape[1] != desc.max_pages or arrays[2].get_device() != device):
        raise ValueError("page_table's rows must have desc.max_pages entries, on the cache's device")
    return device, codes.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr()


def spear_ec_kv_append(desc, batch, q, k, v, cos_sin, codes, scales, zeros, q_out,
                       interleaved=False, stream=None):
    """Rotate q (to q_out) and k by cos_sin (fp32 [rows, dim], or None) and
    store k and v in the cache; q and q_out may be None."""
    import torch
    n, D, H, G, bf16 = batch.tokens, desc.head_dim, desc.q_heads, desc.kv_heads, torch.bfloat16
    dev, cp, sp, zp = _cache(desc, batch, codes, scales, zeros)
    kp, ks = _rows(k, dev, n, G, D, bf16, "k")
    vp, vs = _rows(v, dev, n, G, D, bf16, "v")
    qp, qs = _rows(q, dev, n, H, D, bf16, "q") if q is not None else (None, 0)
    op, os = _rows(q_out, dev, n, H, D, bf16, "q_out") if q_out is not None else (None, 0)
    rope = None
    if cos_sin is not None:
        shape = cos_sin.shape
        if cos_sin.dtype is not torch.float32 or len(shape) != 2 or not cos_sin.is_contiguous() or \
                cos_sin.get_device() != dev:
            raise ValueError("cos_sin must be a contiguous fp32 [rows, dim] on the cache's device")
        rope = spear_ec_kv_rope(cos_sin.data_ptr(), shape[0], shape[1], interleaved)
    _call(_lib().spear_ec_kv_append, dev, stream, desc, batch, qp, qs, kp, ks, vp, vs, rope, cp, sp, zp,
          op, os)


def spear_ec_kv_attention(desc, batch, q, codes, scales, zeros, softmax_scale, out, workspace,
                          lse=None, window=0, stream=None):
    """Attention of q's rows over their sequences' cached tokens, to out (and
    lse, fp32 [tokens, q_heads])."""
    import torch
    n, H, D = batch.tokens, desc.q_heads, desc.head_dim
    dev, cp, sp, zp = _cache(desc, batch, codes, scales, zeros)
    qp, qs = _rows(q, dev, n, H, D, torch.bfloat16, "q")
    op, _ = _rows(out, dev, n, H, D, torch.bfloat16, "out", strided=False)
    lp = None
    if lse is not None:
        shape = lse.shape
        if lse.dtype is not torch.float32 or len(shape) != 2 or shape[0] < n or shape[1] != H or \
                not lse.is_contiguous() or lse.get_device() != dev:
            raise ValueError(f"lse must be contiguous fp32 of shape [>= {n}, {H}] on the cache's device")
        lp = lse.data_ptr()
    wp, size = None, 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous, on the cache's device")
        wp, size = workspace.data_ptr(), workspace.nbytes
    _call(_lib().spear_ec_kv_attention, dev, stream, desc, batch, qp, qs, cp, sp, zp, softmax_scale,
          window, op, lp, wp, size)


def spear_ec_kv_dequant_f32(desc, batch, codes, scales, zeros, k_out, v_out, stream=None):
    """The batch's rows of the cache as fp32 values [tokens, kv_heads, head_dim]."""
    import torch
    n, G, D = batch.tokens, desc.kv_heads, desc.head_dim
    dev, cp, sp, zp = _cache(desc, batch, codes, scales, zeros)
    kp, _ = _rows(k_out, dev, n, G, D, torch.float32, "k_out", strided=False)
    vp, _ = _rows(v_out, dev, n, G, D, torch.float32, "v_out", strided=False)
    _call(_lib().spear_ec_kv_dequant_f32, dev, stream, desc, batch, cp, sp, zp, kp, vp)
