"""CPU: the functions include/hstu_paged.h declares are exported, and their host-side argument checks
answer synchronously without touching a GPU."""
import ctypes
import os
import re

import pytest

class PagedCache(ctypes.Structure):
    """hstu_paged_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("page_table", ctypes.c_void_p), ("table_width", ctypes.c_int32),
                ("table_ld", ctypes.c_int64)]


class Rotation(ctypes.Structure):
    """hstu_rotation_t."""
    _fields_ = [("freqs", ctypes.c_void_p), ("pairs", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("sections", ctypes.c_int32 * 4), ("interleaved", ctypes.c_int32),
                ("positions", ctypes.c_void_p), ("positions_ld", ctypes.c_int64)]


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "hstu_paged.h")
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib(cuda_lib):
    from hstu_pointwise_attention_jagged_b200 import paged
    return paged.load_library()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\w[\w ]*\s+\**(hstu_\w+)\s*\(", text, flags=re.M)))


def test_exports(lib):
    from hstu_pointwise_attention_jagged_b200 import binding, paged
    assert declared() == sorted(paged.EXPORTS)
    out = os.popen("nm -D --defined-only %s" % binding.library_path()).read()
    for name in declared():
        assert re.search(r"\sT %s$" % name, out, re.M), name


def test_marshalling_refuses_without_a_gpu(lib):
    """The checks come before any GPU work: CPU tensors, wrong types, unknown and missing arguments."""
    import torch
    from hstu_pointwise_attention_jagged_b200 import hstu_paged_append, hstu_paged_attn_fwd, hstu_rotary
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: hstu_rotary(x, None, i, torch.zeros(32, dtype=torch.float64)),
                 lambda: hstu_rotary("q", None, i, i), lambda: hstu_rotary(x, None, i), lambda: hstu_rotary(),
                 lambda: hstu_rotary(x, None, i, i, angle=3), lambda: hstu_rotary(x, None, i, i, q=x),
                 lambda: hstu_rotary(*[x] * 11),
                 lambda: hstu_paged_append(x, x, x, x, i, i, i), lambda: hstu_paged_append(x, x, x, x, i, kv_len=i),
                 lambda: hstu_paged_attn_fwd(x, x, x, i, i, i, None, 1.0, 1.0, 4, 4),
                 lambda: hstu_paged_attn_fwd(None, x, x, i, i, i, None, 1.0, 1.0, 4, 4)):
        with pytest.raises(TypeError):
            call()


def _rotation(**kw):
    a = dict(freqs=1 << 12, pairs=32, axes=1, interleaved=0, positions=1 << 13, positions_ld=0)
    sections = kw.pop("sections", [32])
    a.update(kw)
    r = Rotation(**a)
    r.sections[:len(sections)] = sections
    return r


def _cache(**kw):
    a = dict(k=1 << 30, v=1 << 31, page_stride=16 * 128, row_stride=128, head_stride=64, num_pages=8, page_size=16,
             page_table=1 << 12, table_width=4, table_ld=4)
    a.update(kw)
    return PagedCache(**a)


def _rotary(lib, rot=None, **kw):
    a = dict(q=1 << 20, q_ld=128, k=None, k_ld=0, inverse=0, H=2, d=64, rows=16, qo=1 << 24, qo_ld=128, ko=None, ko_ld=0)
    a.update(kw)
    vp = ctypes.c_void_p
    r = _rotation() if rot is None else rot
    return lib.hstu_rotary(vp(a["q"]), a["q_ld"], vp(a["k"]), a["k_ld"], ctypes.byref(r) if r else None, a["inverse"],
                           a["H"], a["d"], a["rows"], vp(a["qo"]), a["qo_ld"], vp(a["ko"]), a["ko_ld"], None)


def test_rotary_refusals(lib):
    assert _rotary(lib, rows=0) == OK
    for kw in (dict(q=None), dict(qo=None), dict(H=0), dict(rows=-1), dict(inverse=2), dict(q_ld=127), dict(ko=1 << 25),
               dict(k=1 << 25), dict(qo=(1 << 20) + 256 * 4), dict(k=1 << 25, k_ld=128, ko=1 << 20, ko_ld=128),
               dict(qo=1 << 20, qo_ld=256)):
        assert _rotary(lib, **kw) == INVALID, kw
    for kw in (dict(d=48), dict(d=256), dict(q=(1 << 20) + 8), dict(qo=(1 << 24) + 2), dict(q_ld=132)):
        assert _rotary(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(pairs=0), dict(pairs=40, sections=[40]), dict(sections=[31]), dict(axes=0), dict(axes=5),
               dict(axes=2, sections=[40, -8]), dict(axes=2, sections=[16, 16], positions_ld=15), dict(freqs=None),
               dict(positions=None)):
        assert _rotary(lib, _rotation(**kw)) == INVALID, kw
    for kw in (dict(pairs=12, sections=[12]), dict(freqs=(1 << 12) + 4), dict(positions=(1 << 13) + 2)):
        assert _rotary(lib, _rotation(**kw)) == UNSUPPORTED, kw


def _append(lib, cache=None, rot=None, **kw):
    a = dict(q=None, q_ld=0, k=1 << 20, k_ld=128, v=1 << 22, v_ld=128, off=1 << 12, kv=1 << 12, B=2, H=2, d=64, total=16,
             qo=None, qo_ld=0)
    a.update(kw)
    vp = ctypes.c_void_p
    c = _cache() if cache is None else cache
    return lib.hstu_paged_append(vp(a["q"]), a["q_ld"], vp(a["k"]), a["k_ld"], vp(a["v"]), a["v_ld"],
                                 ctypes.byref(rot) if rot else None, ctypes.byref(c), vp(a["off"]), vp(a["kv"]), a["B"],
                                 a["H"], a["d"], a["total"], vp(a["qo"]), a["qo_ld"], None)


def test_append_refusals(lib):
    assert _append(lib, total=0) == OK and _append(lib, total=0, B=0) == OK and _append(lib, B=0) == INVALID
    for kw in (dict(k=None), dict(v=None), dict(off=None), dict(kv=None), dict(B=-1), dict(H=0), dict(total=-1), dict(k_ld=120),
               dict(q=1 << 24, q_ld=128, qo=1 << 25, qo_ld=128), dict(q=1 << 24, q_ld=128), dict(k=1 << 30),
               dict(v=(1 << 31) + 4096)):
        assert _append(lib, **kw) == INVALID, kw
    assert _append(lib, rot=_rotation(), q=1 << 24, q_ld=128, qo=1 << 20, qo_ld=128) == INVALID  # q_out over k
    for kw in (dict(d=80), dict(k=(1 << 20) + 8), dict(v_ld=130)):
        assert _append(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(k=None), dict(num_pages=0), dict(table_ld=3), dict(page_table=None), dict(row_stride=32), dict(v=1 << 30),
               dict(page_stride=0)):
        assert _append(lib, _cache(**kw)) == INVALID, kw
    for kw in (dict(page_size=12), dict(page_size=4), dict(page_size=2048), dict(head_stride=68), dict(k=(1 << 30) + 8),
               dict(page_stride=1 << 40)):
        assert _append(lib, _cache(**kw)) == UNSUPPORTED, kw


def _attn(lib, cache=None, **kw):
    a = dict(q=1 << 20, q_ld=128, off=1 << 12, kv=1 << 12, nt=None, B=2, H=2, d=64, total=16, max_new=8, max_kv=64, alpha=1.0,
             N=16.0, out=1 << 24, out_ld=128)
    a.update(kw)
    vp = ctypes.c_void_p
    c = _cache() if cache is None else cache
    return lib.hstu_paged_attn_fwd(vp(a["q"]), a["q_ld"], ctypes.byref(c), vp(a["off"]), vp(a["kv"]), vp(a["nt"]), a["B"],
                                   a["H"], a["d"], a["total"], a["max_new"], a["max_kv"], a["alpha"], a["N"], vp(a["out"]),
                                   a["out_ld"], None)


def test_attn_refusals(lib):
    assert _attn(lib, total=0) == OK and _attn(lib, total=0, B=0) == OK and _attn(lib, B=0) == INVALID
    for kw in (dict(q=None), dict(out=None), dict(off=None), dict(kv=None), dict(B=-1), dict(H=0), dict(total=-1),
               dict(max_new=-1), dict(max_kv=-1), dict(alpha=float("nan")), dict(alpha=float("inf")), dict(N=0.0),
               dict(N=float("inf")), dict(q_ld=64), dict(out_ld=100), dict(out=1 << 20), dict(out=1 << 30),
               dict(out=(1 << 31) + 64)):
        assert _attn(lib, **kw) == INVALID, kw
    for kw in (dict(d=16), dict(q=(1 << 20) + 2), dict(out=(1 << 24) + 8), dict(out_ld=129), dict(max_kv=2 ** 31 - 1)):
        assert _attn(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(v=None), dict(num_pages=0), dict(table_width=5)):
        assert _attn(lib, _cache(**kw)) == INVALID, kw
    for kw in (dict(page_size=24), dict(row_stride=129)):
        assert _attn(lib, _cache(**kw)) == UNSUPPORTED, kw


def test_selfcheck_limit_refusals(lib):
    """Limits of 0 and above one second, and hstu_paged_attn_fwd's own refusals with a limit in range."""
    c = _cache()
    vp, u64 = ctypes.c_void_p, ctypes.c_uint64

    def call(limit, B=2, rows=8, q=0x10000):
        return lib.hstu_paged_selfcheck_fwd_timeout(vp(q), 128, ctypes.byref(c), vp(0x20000), vp(0x30000), vp(0), B, 2, 64,
                                                    rows, 4, 64, 1.0, 1.0, vp(0x40000), 128, u64(limit), vp(0))

    for limit in (0, 10 ** 9 + 1, 2 ** 63):
        assert call(limit) == INVALID
    assert call(1000, rows=0) == OK
    assert call(1000, B=-1) == INVALID
    assert call(1000, q=0x10002) == UNSUPPORTED


def test_extents_beyond_any_memory(lib):
    """Strides whose extents would not fit 64 bits are refused, not wrapped into small ones."""
    huge = 1 << 61
    assert _rotary(lib, q_ld=huge) == UNSUPPORTED and _rotary(lib, qo_ld=huge, rows=1 << 30) == UNSUPPORTED
    assert _append(lib, k_ld=huge) == UNSUPPORTED and _append(lib, v_ld=huge) == UNSUPPORTED
    assert _attn(lib, q_ld=huge) == UNSUPPORTED and _attn(lib, out_ld=huge) == UNSUPPORTED
    for call in (_append, _attn):
        assert call(lib, _cache(num_pages=1 << 30, page_stride=1 << 34)) == UNSUPPORTED
