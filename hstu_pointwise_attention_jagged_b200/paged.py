"""ctypes binding of the paged K/V cache calls of libhstu_attn.so (C ABI: include/hstu_paged.h).

Argument marshalling only, as in :mod:`.binding`: every function checks the torch tensors it is
given, passes pointers, sizes, strides and the current CUDA stream to the C entry point of the same
name, and raises :class:`~.binding.HstuError` on a non-zero status.
"""
import ctypes

import torch

from . import binding
from .binding import _check_index, _ptr, _raise_if, _stream_ptr

MAX_AXES = 4

# Every symbol include/hstu_paged.h declares.
EXPORTS = (
    "hstu_rotary",
    "hstu_paged_append",
    "hstu_paged_attn_fwd",
)


class PagedCache(ctypes.Structure):
    """hstu_paged_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("page_table", ctypes.c_void_p), ("table_width", ctypes.c_int32),
                ("table_ld", ctypes.c_int64)]


class Rotation(ctypes.Structure):
    """hstu_rotation_t."""
    _fields_ = [("freqs", ctypes.c_void_p), ("pairs", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("sections", ctypes.c_int32 * MAX_AXES), ("interleaved", ctypes.c_int32),
                ("positions", ctypes.c_void_p), ("positions_ld", ctypes.c_int64)]


_lib = None


def load_library():
    """The library with this module's entry points declared; raises if it has not been built."""
    global _lib
    if _lib is None:
        lib = binding.load_library()
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        rot, cache = ctypes.POINTER(Rotation), ctypes.POINTER(PagedCache)
        lib.hstu_rotary.argtypes = [vp, i64, vp, i64, rot, i32, i32, i32, i32, vp, i64, vp, i64, vp]
        lib.hstu_paged_append.argtypes = [vp, i64, vp, i64, vp, i64, rot, cache, vp, vp, i32, i32, i32, i32, vp, i64, vp]
        f32 = ctypes.c_float
        lib.hstu_paged_attn_fwd.argtypes = [vp, i64, cache, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, f32, vp, i64, vp]
        for name in EXPORTS:
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


def _check_rows(name, t, H=None, d=None, rows=None, device=None):
    """A bf16 CUDA tensor [rows, H, d] with packed heads; returns its row stride in elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != torch.bfloat16 or t.dim() != 3:
        raise TypeError("%s must be a bf16 tensor [rows, H, d]" % name)
    if H is not None and (t.shape[1] != H or t.shape[2] != d):
        raise ValueError("%s has shape %s, expected [*, %d, %d]" % (name, tuple(t.shape), H, d))
    if rows is not None and t.shape[0] != rows:
        raise ValueError("%s has %d rows, expected %d" % (name, t.shape[0], rows))
    if device is not None and t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    n, h, c = t.shape
    if n == 0:
        return h * c
    if (c > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != c):
        raise TypeError("%s must have its heads packed (only the row stride is free)" % name)
    return t.stride(0) if n > 1 else h * c  # the stride of a single row is never used


def _rotation(freqs, sections, positions, interleaved, rows, device, need_positions):
    if not isinstance(freqs, torch.Tensor) or freqs.dtype != torch.float64 or freqs.dim() != 1 or \
            freqs.device != device or not freqs.is_contiguous():
        raise TypeError("freqs must be a contiguous float64 vector on %s" % device)
    sections = [freqs.numel()] if sections is None else [int(n) for n in sections]
    if not 1 <= len(sections) <= MAX_AXES:
        raise ValueError("1 to %d sections, got %d" % (MAX_AXES, len(sections)))
    r = Rotation(freqs=freqs.data_ptr(), pairs=freqs.numel(), axes=len(sections), interleaved=int(bool(interleaved)))
    r.sections[:len(sections)] = sections
    if positions is None:
        if need_positions:
            raise TypeError("positions are required")
        return r
    if not isinstance(positions, torch.Tensor) or positions.device != device or positions.dtype != torch.int32:
        raise TypeError("positions must be an int32 tensor on %s" % device)
    p = positions[None] if positions.dim() == 1 else positions
    if p.dim() != 2 or tuple(p.shape) != (len(sections), rows):
        raise ValueError("positions must be [%d, %d], one row for each axis" % (len(sections), rows))
    if rows > 1 and p.stride(1) != 1:
        raise TypeError("positions of one axis must be contiguous")
    r.positions = positions.data_ptr()
    r.positions_ld = p.stride(0) if len(sections) > 1 else rows
    return r


def _cache(k_cache, v_cache, page_table, B, device):
    """k_cache, v_cache: bf16 [pages, page_size, H, d] views with equal strides, d contiguous."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.bfloat16 or t.dim() != 4:
            raise TypeError("%s must be a bf16 tensor [pages, page_size, H, d] on %s" % (name, device))
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    pages, page_size, H, d = k_cache.shape
    if pages < 1 or page_size < 1 or H < 1 or d < 1:
        raise ValueError("the cache has no rows")
    # The stride of a dimension of one entry is never used.
    strides = []
    for i, n in enumerate((pages, page_size, H)):
        if n > 1 and k_cache.stride(i) != v_cache.stride(i):
            raise ValueError("k_cache and v_cache must have the same strides")
        strides.append(k_cache.stride(i) if n > 1 else d)
    if d > 1 and (k_cache.stride(3) != 1 or v_cache.stride(3) != 1):
        raise TypeError("the last dimension of the cache must be contiguous")
    if not isinstance(page_table, torch.Tensor) or page_table.device != device or page_table.dtype != torch.int32 or \
            page_table.dim() != 2 or page_table.shape[0] != B or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise TypeError("page_table must be an int32 tensor [%d, pages of a user] on %s" % (B, device))
    width = page_table.shape[1]
    return PagedCache(k=k_cache.data_ptr(), v=v_cache.data_ptr(), page_stride=strides[0], row_stride=strides[1],
                      head_stride=strides[2], num_pages=pages, page_size=page_size,
                      page_table=page_table.data_ptr() if page_table.numel() else None,
                      table_width=width, table_ld=page_table.stride(0) if B > 1 and width else width)


def hstu_rotary_freqs(pairs, base=10000.0, device="cuda"):
    """The usual frequencies base^(-i / pairs) of one axis, float64 [pairs] (radians a position)."""
    return (float(base) ** (-torch.arange(pairs, dtype=torch.float64) / max(1, pairs))).to(device)


def hstu_rotary(q, k, positions, freqs, sections=None, interleaved=False, inverse=False, q_out=None, k_out=None,
                stream=None):
    """Rotates q and (unless None) k, bf16 [rows, H, d], by their positions; returns (q_out, k_out).
    ``positions``: int32 [rows] or [axes, rows]; ``sections``: pairs of each axis.  ``inverse`` turns
    back, which is the gradient.  ``q_out`` may be q (in place).  See include/hstu_paged.h."""
    lib = load_library()
    q_ld = _check_rows("q", q)
    rows, H, d = q.shape
    dev = q.device
    k_ld = _check_rows("k", k, H, d, rows, dev) if k is not None else 0
    rot = _rotation(freqs, sections, positions, interleaved, rows, dev, True)
    q_out = torch.empty((rows, H, d), dtype=q.dtype, device=dev) if q_out is None else q_out
    if k is not None and k_out is None:
        k_out = torch.empty((rows, H, d), dtype=q.dtype, device=dev)
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    qo_ld = _check_rows("q_out", q_out, H, d, rows, dev)
    ko_ld = _check_rows("k_out", k_out, H, d, rows, dev) if k is not None else 0
    with torch.cuda.device(dev):
        st = lib.hstu_rotary(_ptr(q), q_ld, _ptr(k), k_ld, ctypes.byref(rot), int(bool(inverse)), H, d, rows,
                             _ptr(q_out), qo_ld, _ptr(k_out), ko_ld, _stream_ptr(stream, dev))
    _raise_if(st, "hstu_rotary")
    return q_out, k_out


def hstu_paged_append(k, v, k_cache, v_cache, page_table, q_offsets, kv_len, q=None, positions=None, freqs=None,
                      sections=None, interleaved=False, q_out=None, stream=None):
    """Writes the new rows k, v (bf16 [total_new, H, d], users packed by q_offsets) to the last places
    of each user's kv_len rows in the paged cache.  With ``freqs`` K is rotated on the way, and q too if
    given; ``positions`` default to the place in the cache.  Returns the rotated q (or None).
    See include/hstu_paged.h."""
    lib = load_library()
    k_ld = _check_rows("k", k)
    total, H, d = k.shape
    dev = k.device
    v_ld = _check_rows("v", v, H, d, total, dev)
    B = q_offsets.numel() - 1
    _check_index("q_offsets", q_offsets, B + 1, dev, optional=False)
    _check_index("kv_len", kv_len, B, dev, optional=False)
    cache = _cache(k_cache, v_cache, page_table, B, dev)
    if k_cache.shape[2:] != k.shape[1:]:
        raise ValueError("the cache holds [%d, %d] rows, k has [%d, %d]" % (*k_cache.shape[2:], H, d))
    if freqs is None and (q is not None or positions is not None or sections is not None):
        raise ValueError("q, positions and sections need freqs")
    rot = None if freqs is None else _rotation(freqs, sections, positions, interleaved, total, dev, False)
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    q_ld = qo_ld = 0
    if q is not None:
        q_ld = _check_rows("q", q, H, d, total, dev)
        q_out = torch.empty((total, H, d), dtype=q.dtype, device=dev) if q_out is None else q_out
        qo_ld = _check_rows("q_out", q_out, H, d, total, dev)
    with torch.cuda.device(dev):
        st = lib.hstu_paged_append(_ptr(q), q_ld, _ptr(k), k_ld, _ptr(v), v_ld,
                                   None if rot is None else ctypes.byref(rot), ctypes.byref(cache), _ptr(q_offsets),
                                   _ptr(kv_len), B, H, d, total, _ptr(q_out), qo_ld, _stream_ptr(stream, dev))
    _raise_if(st, "hstu_paged_append")
    return q_out


def hstu_paged_attn_fwd(q, k_cache, v_cache, page_table, q_offsets, kv_len, num_targets, alpha, N, max_new, max_kv,
                        out=None, stream=None):
    """Attention of each user's new rows q (bf16 [total_new, H, d], packed by q_offsets) over its kv_len rows
    in the paged cache, the new ones included; the last num_targets of them are candidates.  Returns
    ``out``.  See include/hstu_paged.h."""
    lib = load_library()
    q_ld = _check_rows("q", q)
    total, H, d = q.shape
    dev = q.device
    B = q_offsets.numel() - 1
    _check_index("q_offsets", q_offsets, B + 1, dev, optional=False)
    _check_index("kv_len", kv_len, B, dev, optional=False)
    _check_index("num_targets", num_targets, B, dev)
    cache = _cache(k_cache, v_cache, page_table, B, dev)
    if k_cache.shape[2:] != q.shape[1:]:
        raise ValueError("the cache holds [%d, %d] rows, q has [%d, %d]" % (*k_cache.shape[2:], H, d))
    out = torch.empty((total, H, d), dtype=q.dtype, device=dev) if out is None else out
    out_ld = _check_rows("out", out, H, d, total, dev)
    with torch.cuda.device(dev):
        st = lib.hstu_paged_attn_fwd(_ptr(q), q_ld, ctypes.byref(cache), _ptr(q_offsets), _ptr(kv_len), _ptr(num_targets),
                                     B, H, d, total, int(max_new), int(max_kv), float(alpha), float(N), _ptr(out), out_ld,
                                     _stream_ptr(stream, dev))
    _raise_if(st, "hstu_paged_attn_fwd")
    return out
