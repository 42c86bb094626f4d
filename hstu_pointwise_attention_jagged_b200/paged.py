"""Binding of the paged K/V cache calls of libhstu_attn.so (C ABI: include/hstu_paged.h).

The functions marshal torch tensors into the C entry points of the same names, as :mod:`.binding`
does, with the same checks and errors (:class:`~.binding.HstuError` on a non-zero status).  They are
written in C++ (``csrc/paged_binding.cpp``): a call for a few rows takes the GPU about three microseconds,
and in Python its marshalling took 13 to 16.  If the library has not been built, importing this module or the
first call raises.
"""
import ctypes
import os

import torch

from . import binding, build

_REBUILD = "(run __graft_entry__.build() or python -m hstu_pointwise_attention_jagged_b200.build)"
# The module uses torch's C++ interface, which another torch need not have.
if build.module_built_for() not in (None, build.built_for()):
    raise RuntimeError("_paged_native.so was built for %s, this is %s %s" % (build.module_built_for(), build.built_for(),
                                                                             _REBUILD))
try:
    from . import _paged_native
except ImportError as e:
    raise RuntimeError("_paged_native.so %s %s" % (
        "could not be loaded: %s" % e if os.path.exists(build.MODULE) else "is not built", _REBUILD)) from e

MAX_AXES = 4

# Every symbol include/hstu_paged.h declares.
EXPORTS = (
    "hstu_rotary",
    "hstu_paged_append",
    "hstu_paged_attn_fwd",
    "hstu_paged_selfcheck_fwd_timeout",
)

hstu_rotary = _paged_native.hstu_rotary
hstu_paged_append = _paged_native.hstu_paged_append
hstu_paged_attn_fwd = _paged_native.hstu_paged_attn_fwd
hstu_paged_selfcheck_fwd_timeout = _paged_native.hstu_paged_selfcheck_fwd_timeout

_lib = None


def load_library():
    """The library, with its entry points of include/hstu_paged.h declared and handed to the marshalling
    module; raises if it has not been built."""
    global _lib
    if _lib is None:
        lib = binding.load_library()
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        lib.hstu_rotary.argtypes = [vp, i64, vp, i64, vp, i32, i32, i32, i32, vp, i64, vp, i64, vp]
        lib.hstu_paged_append.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, vp]
        lib.hstu_paged_attn_fwd.argtypes = [vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, f32, vp, i64, vp]
        lib.hstu_paged_selfcheck_fwd_timeout.argtypes = lib.hstu_paged_attn_fwd.argtypes[:-1] + [ctypes.c_uint64, vp]
        for name in EXPORTS:
            getattr(lib, name).restype = ctypes.c_int
        _paged_native.bind(binding.HstuError, *(ctypes.cast(getattr(lib, name), vp).value for name in EXPORTS))
        _lib = lib
    return _lib


def hstu_rotary_freqs(pairs, base=10000.0, device="cuda"):
    """The usual frequencies base^(-i / pairs) of one axis, float64 [pairs] (radians a position)."""
    return (float(base) ** (-torch.arange(pairs, dtype=torch.float64) / max(1, pairs))).to(device)
