"""ctypes binding of the paged K/V cache calls of libhstu_attn.so (C ABI: include/hstu_paged.h).

Argument marshalling only, as in :mod:`.binding`: every function checks the torch tensors it is
given, passes pointers, sizes, strides and the current CUDA stream to the C entry point of the same
name, and raises :class:`~.binding.HstuError` on a non-zero status.

A call for a few rows takes the GPU about three microseconds, so the marshalling is kept short: each
check first asks the usual case's questions, and only a tensor that fails them meets the function that finds
out what is wrong; the two argument structs are packed as bytes.
"""
import ctypes
import struct

import torch

from . import binding
from .binding import _raise_if

MAX_AXES = 4

# Every symbol include/hstu_paged.h declares.
EXPORTS = (
    "hstu_rotary",
    "hstu_paged_append",
    "hstu_paged_attn_fwd",
)

# hstu_paged_cache_t and hstu_rotation_t, native alignment.
_CACHE = struct.Struct("@QQqqqiiQiq")
_ROTATION = struct.Struct("@Qii4iiQq")

_BF16, _I32, _F64 = torch.bfloat16, torch.int32, torch.float64
_lib = None


def load_library():
    """The library with this module's entry points declared; raises if it has not been built."""
    global _lib
    if _lib is None:
        lib = binding.load_library()
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        lib.hstu_rotary.argtypes = [vp, i64, vp, i64, vp, i32, i32, i32, i32, vp, i64, vp, i64, vp]
        lib.hstu_paged_append.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, vp]
        lib.hstu_paged_attn_fwd.argtypes = [vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, f32, vp, i64, vp]
        for name in EXPORTS:
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


def _call(name, index, stream, *args):
    """lib.name(*args, stream) with device `index` current; raises on a non-zero status."""
    fn = getattr(_lib, name)
    if torch.cuda.current_device() == index:
        raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
            status = fn(*args, raw)
    if status:
        _raise_if(status, name)


def _first(name, t):
    """Shape, row stride (elements) and device index of the call's first token tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    shape = t.shape
    if t.dtype is not _BF16 or len(shape) != 3:
        raise TypeError("%s must be a bf16 tensor [rows, H, d]" % name)
    index, s = t.get_device(), t.stride()
    if s[2] == 1 and s[1] == shape[2] and shape[0] > 1:
        return shape, s[0], index
    return shape, _row_stride_slow(name, t, shape, index), index


def _row_stride(name, t, shape, index):
    """The row stride (elements) of a bf16 tensor of this shape [rows, H, d] with packed heads."""
    if isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.get_device() == index and t.shape == shape:
        s = t.stride()
        if s[2] == 1 and s[1] == shape[2] and shape[0] > 1:
            return s[0]
    return _row_stride_slow(name, t, shape, index)


def _row_stride_slow(name, t, shape, index):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not _BF16 or t.dim() != 3:
        raise TypeError("%s must be a bf16 tensor [rows, H, d]" % name)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.get_device() != index:
        raise ValueError("%s must be on cuda:%d" % (name, index))
    n, h, c = shape
    if n and ((c > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != c)):
        raise TypeError("%s must have its heads packed (only the row stride is free)" % name)
    return t.stride(0) if n > 1 else h * c  # the stride of a single row is never used


def _output(name, t, shape, index, like, stream):
    """The given output, or a new packed one, and its row stride.  A new one belongs to the stream that the
    call runs on: memory of another stream might still be in use there."""
    if t is not None:
        return t, _row_stride(name, t, shape, index)
    if stream is None:
        t = torch.empty_like(like, memory_format=torch.contiguous_format)
    else:
        with torch.cuda.stream(stream):
            t = torch.empty_like(like, memory_format=torch.contiguous_format)
    return t, shape[1] * shape[2]


def _index(name, t, n, index):
    """Address of a contiguous int32 vector of n elements on the device."""
    if isinstance(t, torch.Tensor) and t.dtype is _I32 and t.get_device() == index and t.shape == (n,) and \
            (n < 2 or t.stride(0) == 1):
        return t.data_ptr()
    raise TypeError("%s must be a contiguous int32 tensor of %d elements on cuda:%d" % (name, n, index))


def _users(q_offsets):
    if not isinstance(q_offsets, torch.Tensor) or q_offsets.dim() != 1 or q_offsets.shape[0] < 1:
        raise TypeError("q_offsets must be an int32 vector of one element more than there are users")
    return q_offsets.shape[0] - 1


def _rotation(freqs, sections, positions, interleaved, rows, index, need_positions):
    """hstu_rotation_t as bytes."""
    if not isinstance(freqs, torch.Tensor) or freqs.dtype is not _F64 or freqs.dim() != 1 or \
            freqs.get_device() != index or not freqs.is_contiguous():
        raise TypeError("freqs must be a contiguous float64 vector on cuda:%d" % index)
    pairs = freqs.shape[0]
    sections = (pairs,) if sections is None else tuple(int(n) for n in sections)
    axes = len(sections)
    if not 1 <= axes <= MAX_AXES:
        raise ValueError("1 to %d sections, got %d" % (MAX_AXES, axes))
    at, ld = 0, 0
    if positions is None:
        if need_positions:
            raise TypeError("positions are required")
    else:
        if not isinstance(positions, torch.Tensor) or positions.get_device() != index or positions.dtype is not _I32:
            raise TypeError("positions must be an int32 tensor on cuda:%d" % index)
        if positions.shape != (axes, rows) and (axes > 1 or positions.shape != (rows,)):
            raise ValueError("positions must be [%d, %d], one row for each axis" % (axes, rows))
        if rows > 1 and positions.stride(-1) != 1:
            raise TypeError("positions of one axis must be contiguous")
        at, ld = positions.data_ptr(), positions.stride(0) if axes > 1 else rows
    return _ROTATION.pack(freqs.data_ptr(), pairs, axes, *sections, *(0,) * (MAX_AXES - axes), 1 if interleaved else 0, at, ld)


def _cache(k_cache, v_cache, page_table, B, H, d, index):
    """hstu_paged_cache_t as bytes, of bf16 [pages, page_size, H, d] views with equal strides, d contiguous."""
    if not (isinstance(k_cache, torch.Tensor) and isinstance(v_cache, torch.Tensor) and k_cache.dtype is _BF16 and
            v_cache.dtype is _BF16 and k_cache.get_device() == index and v_cache.get_device() == index and
            k_cache.dim() == 4):
        raise TypeError("k_cache and v_cache must be bf16 tensors [pages, page_size, H, d] on cuda:%d" % index)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if shape[2] != H or shape[3] != d:
        raise ValueError("the cache holds [%d, %d] rows, the new rows are [%d, %d]" % (shape[2], shape[3], H, d))
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks != vs or 1 in shape:
        if 0 in shape:
            raise ValueError("the cache has no rows")
        # The stride of a dimension of one entry is never used.
        ks, vs = ([s if n > 1 else (d if i < 3 else 1) for i, (s, n) in enumerate(zip(x, shape))] for x in (ks, vs))
        if ks != vs:
            raise ValueError("k_cache and v_cache must have the same strides")
    if ks[3] != 1:
        raise TypeError("the last dimension of the cache must be contiguous")
    if not isinstance(page_table, torch.Tensor) or page_table.get_device() != index or page_table.dtype is not _I32 or \
            page_table.dim() != 2 or page_table.shape[0] != B:
        raise TypeError("page_table must be an int32 tensor [%d, pages of a user] on cuda:%d" % (B, index))
    width, ts = page_table.shape[1], page_table.stride()
    if width > 1 and ts[1] != 1:
        raise TypeError("a user's entries of page_table must be contiguous")
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), ks[0], ks[1], ks[2], shape[0], shape[1],
                       page_table.data_ptr(), width, ts[0] if B > 1 and width else width)


def hstu_rotary_freqs(pairs, base=10000.0, device="cuda"):
    """The usual frequencies base^(-i / pairs) of one axis, float64 [pairs] (radians a position)."""
    return (float(base) ** (-torch.arange(pairs, dtype=torch.float64) / max(1, pairs))).to(device)


def hstu_rotary(q, k, positions, freqs, sections=None, interleaved=False, inverse=False, q_out=None, k_out=None,
                stream=None):
    """Rotates q and (unless None) k, bf16 [rows, H, d], by their positions; returns (q_out, k_out).
    ``positions``: int32 [rows] or [axes, rows]; ``sections``: pairs of each axis.  ``inverse`` turns
    back, which is the gradient.  ``q_out`` may be q (in place).  See include/hstu_paged.h."""
    load_library()
    shape, q_ld, index = _first("q", q)
    rows, H, d = shape
    rot = _rotation(freqs, sections, positions, interleaved, rows, index, True)
    q_out, qo_ld = _output("q_out", q_out, shape, index, q, stream)
    k_ld = ko_ld = k_at = ko_at = 0
    if k is not None:
        k_ld = _row_stride("k", k, shape, index)
        k_out, ko_ld = _output("k_out", k_out, shape, index, q, stream)
        k_at, ko_at = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    _call("hstu_rotary", index, stream, q.data_ptr(), q_ld, k_at, k_ld, rot, 1 if inverse else 0, H, d, rows,
          q_out.data_ptr(), qo_ld, ko_at, ko_ld)
    return q_out, k_out


def hstu_paged_append(k, v, k_cache, v_cache, page_table, q_offsets, kv_len, q=None, positions=None, freqs=None,
                      sections=None, interleaved=False, q_out=None, stream=None):
    """Writes the new rows k, v (bf16 [total_new, H, d], users packed by q_offsets) to the last places
    of each user's kv_len rows in the paged cache.  With ``freqs`` K is rotated on the way, and q too if
    given; ``positions`` default to the place in the cache.  Returns the rotated q (or None).
    See include/hstu_paged.h."""
    load_library()
    shape, k_ld, index = _first("k", k)
    total, H, d = shape
    v_ld = _row_stride("v", v, shape, index)
    B = _users(q_offsets)
    off, lens = _index("q_offsets", q_offsets, B + 1, index), _index("kv_len", kv_len, B, index)
    cache = _cache(k_cache, v_cache, page_table, B, H, d, index)
    rot, q_ld, qo_ld, q_at, qo_at = None, 0, 0, 0, 0
    if freqs is not None:
        rot = _rotation(freqs, sections, positions, interleaved, total, index, False)
    elif q is not None or positions is not None or sections is not None:
        raise ValueError("q, positions and sections need freqs")
    if q is not None:
        q_ld = _row_stride("q", q, shape, index)
        q_out, qo_ld = _output("q_out", q_out, shape, index, q, stream)
        q_at, qo_at = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    _call("hstu_paged_append", index, stream, q_at, q_ld, k.data_ptr(), k_ld, v.data_ptr(), v_ld, rot, cache, off, lens,
          B, H, d, total, qo_at, qo_ld)
    return q_out


def hstu_paged_attn_fwd(q, k_cache, v_cache, page_table, q_offsets, kv_len, num_targets, alpha, N, max_new, max_kv,
                        out=None, stream=None):
    """Attention of each user's new rows q (bf16 [total_new, H, d], packed by q_offsets) over its kv_len rows
    in the paged cache, the new ones included; the last num_targets of them are candidates.  Returns
    ``out``.  See include/hstu_paged.h."""
    load_library()
    shape, q_ld, index = _first("q", q)
    total, H, d = shape
    B = _users(q_offsets)
    off, lens = _index("q_offsets", q_offsets, B + 1, index), _index("kv_len", kv_len, B, index)
    targets = 0 if num_targets is None else _index("num_targets", num_targets, B, index)
    cache = _cache(k_cache, v_cache, page_table, B, H, d, index)
    out, out_ld = _output("out", out, shape, index, q, stream)
    _call("hstu_paged_attn_fwd", index, stream, q.data_ptr(), q_ld, cache, off, lens, targets, B, H, d, total, max_new,
          max_kv, alpha, N, out.data_ptr(), out_ld)
    return out
