"""GPU: hstu_paged_append: V copied exactly, K and Q rotated as hstu_rotary rotates them (bit for bit),
every row at its place of the table, and nothing else in the pool touched."""
import numpy as np
import pytest
import torch

from gpu_util import dev_i32
from hstu_pointwise_attention_jagged_b200 import binding, paged
from paged_util import Pool, bf16_normal, offsets_of

pytestmark = pytest.mark.gpu

CASES = [  # cached, new rows, page, H, d, layout
    ([0], [1], 16, 1, 32, "rows"),
    ([5, 0, 100, 31], [1, 0, 7, 1], 32, 2, 64, "heads"),
    ([3000] * 5, [1] * 5, 16, 4, 128, "rows"),
    ([0, 129, 64, 0, 7], [300, 0, 64, 0, 1000], 8, 3, 128, "halves"),
    ([10, 2000], [1500, 49], 1024, 2, 64, "rows"),
    ([17] * 40, list(range(40)), 128, 8, 32, "heads"),
    ([9, 1, 70], [3, 60, 1], 32, 3, 128, "padded"),
]


def _setup(cached, new, page, H, d, layout, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cached, new = np.asarray(cached), np.asarray(new)
    pool = Pool(cached + new, page, H, d, layout, seed)
    total = int(new.sum())
    q, k, v = (bf16_normal(gen, total, H, d) for _ in range(3))
    return pool, q, k, v, offsets_of(new), dev_i32(cached + new)


def _bits(t):
    return t.contiguous().view(torch.int16)


def _expect(pool, cached, new, k, v):
    """The pool after the call, from its state now."""
    ek, ev = pool.k.clone(), pool.v.clone()
    at = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        if n:
            idx = pool.where(b, c, c + n)
            ek[idx], ev[idx] = k[at:at + n], v[at:at + n]
        at += n
    return ek, ev


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("rotate", [None, "place", "axes"])
def test_append(case, rotate):
    cached, new, page, H, d, layout = case
    pool, q, k, v, off, kv = _setup(*case)
    kw = {}
    wk, wq = k, None
    if rotate:
        place = np.concatenate([np.arange(c, c + n) for c, n in zip(cached, new)]).astype(np.int32)
        pairs = d // 2 if rotate == "place" else d // 4
        f = paged.hstu_rotary_freqs(pairs)
        if rotate == "place":
            pos, kw = place[None], dict(q=q, freqs=f)
        else:
            pos = np.stack([place, 1_700_000_000 + 97 * place]).astype(np.int32)
            kw = dict(q=q, freqs=f, sections=[pairs // 2, pairs // 2], positions=dev_i32(pos).view(pos.shape),
                      interleaved=True)
        wq, wk = paged.hstu_rotary(q, k, dev_i32(pos).view(pos.shape), f, kw.get("sections"), kw.get("interleaved", False))
    ek, ev = _expect(pool, cached, new, wk, v)
    got = paged.hstu_paged_append(k, v, pool.k, pool.v, pool.table, off, kv, **kw)
    assert binding.hstu_attn_get_error() == 0
    assert torch.equal(_bits(pool.k), _bits(ek)) and torch.equal(_bits(pool.v), _bits(ev))
    assert (got is None) == (wq is None)
    if wq is not None:
        assert torch.equal(got, wq)


def test_strided_inputs_and_in_place_q():
    cached, new, page, H, d, layout = CASES[3]
    pool, q, k, v, off, kv = _setup(*CASES[3])
    wide = torch.stack([q, v, q, k], 1).contiguous()
    f = paged.hstu_rotary_freqs(d // 2)
    place = dev_i32(np.concatenate([np.arange(c, c + n) for c, n in zip(cached, new)]))
    wq, wk = paged.hstu_rotary(q, k, place, f)
    ek, ev = _expect(pool, cached, new, wk, v)
    out = paged.hstu_paged_append(wide[:, 3], wide[:, 1], pool.k, pool.v, pool.table, off, kv, q=wide[:, 2], freqs=f,
                                  q_out=wide[:, 2])
    assert torch.equal(_bits(pool.k), _bits(ek)) and torch.equal(_bits(pool.v), _bits(ev))
    assert torch.equal(out, wq) and torch.equal(wide[:, 0], q) and torch.equal(wide[:, 1], v) and torch.equal(wide[:, 3], k)


def test_more_users_than_one_scan():
    """Past the size up to which a block scans all offsets, rows search for their users; empty users among them."""
    rng = np.random.default_rng(3)
    new = rng.integers(0, 4, 3000)
    cached = rng.integers(0, 40, 3000)
    pool, q, k, v, off, kv = _setup(cached, new, 8, 1, 32, "rows", 4)
    ek, ev = _expect(pool, cached, new, k, v)
    paged.hstu_paged_append(k, v, pool.k, pool.v, pool.table, off, kv)
    assert binding.hstu_attn_get_error() == 0
    assert torch.equal(_bits(pool.k), _bits(ek)) and torch.equal(_bits(pool.v), _bits(ev))


def test_wide_table_of_another_pitch():
    pool, q, k, v, off, kv = _setup(*CASES[1])
    cached, new = CASES[1][:2]
    ek, ev = _expect(pool, cached, new, k, v)
    loose = torch.full((4, pool.table.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    loose[:, :pool.table.shape[1]] = pool.table
    paged.hstu_paged_append(k, v, pool.k, pool.v, loose[:, :pool.table.shape[1]], off, kv)
    assert torch.equal(_bits(pool.k), _bits(ek)) and torch.equal(_bits(pool.v), _bits(ev))


def test_bad_users_and_pages_are_skipped_and_reported():
    cached, new = [20, 20, 20, 20, 20], [4, 4, 4, 4, 4]
    pool, q, k, v, off, kv = _setup(cached, new, 8, 2, 64, "rows", 5)
    ek, ev = _expect(pool, cached, new, k, v)
    kv_bad = kv.clone()
    kv_bad[1] = 3          # shorter than its new rows
    kv_bad[2] = 1 << 20    # more pages than the table has
    table = pool.table.clone()
    table[3, 2] = pool.pages      # one past the pool: position 16..23 of user 3
    table[4, 2] = -1
    skipped = [1, 2, 3, 4]
    for b in skipped:
        at = pool.where(b, 20, 24)
        ek[at], ev[at] = pool.k[at], pool.v[at]
    f = paged.hstu_rotary_freqs(32)
    q_out = torch.full_like(q, 5.0)
    before = pool.k.clone()
    paged.hstu_paged_append(k, v, pool.k, pool.v, table, off, kv_bad)
    assert binding.hstu_attn_get_error() == 4
    assert torch.equal(_bits(pool.k), _bits(ek)) and torch.equal(_bits(pool.v), _bits(ev))
    pool.k.copy_(before)
    paged.hstu_paged_append(k, v, pool.k, pool.v, table, off, kv_bad, q=q, freqs=f, q_out=q_out)
    assert binding.hstu_attn_get_error() == 4
    assert binding.hstu_attn_get_error() == 0
    assert torch.all(q_out[4:12] == 5.0)  # skipped users
    # Offsets that do not end at the last row: reported, the consistent users are written.
    off_bad = off.clone()
    off_bad[5] = 19
    paged.hstu_paged_append(k, v, pool.k, pool.v, pool.table, off_bad, kv)
    assert binding.hstu_attn_get_error() == 4


def test_decreasing_offsets():
    """Offsets that step back: reported; nothing but cache rows that the offsets and lengths name is written."""
    cached, new = [20, 20, 20], [4, 4, 4]
    pool, q, k, v, off, kv = _setup(cached, new, 8, 2, 64, "rows", 6)
    at = [pool.where(b, 20, 24) for b in range(3)]
    paged.hstu_paged_append(k, v, pool.k, pool.v, pool.table, dev_i32([0, 8, 4, 12]), kv)
    assert binding.hstu_attn_get_error() == 4
    for b in (1, 2):
        pool.k[at[b]] = float("nan")
    for idx in (pool.where(0, 16, 24), pool.where(2, 16, 24)):
        pool.k[idx] = float("nan")
    assert torch.isnan(pool.k).all()


def test_capture_and_other_stream():
    pool, q, k, v, off, kv = _setup(*CASES[2])
    cached, new = CASES[2][:2]
    ek, ev = _expect(pool, cached, new, k, v)
    buf = torch.zeros_like(k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        paged.hstu_paged_append(buf, v, pool.k, pool.v, pool.table, off, kv)
    buf.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(_bits(pool.k), _bits(ek)) and torch.equal(_bits(pool.v), _bits(ev))
    pool.k.fill_(float("nan"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    paged.hstu_paged_append(k, v, pool.k, pool.v, pool.table, off, kv, stream=s)
    s.synchronize()
    assert torch.equal(_bits(pool.k), _bits(ek))


def test_nothing_to_do():
    pool, q, k, v, off, kv = _setup([5, 6], [0, 0], 16, 1, 32, "rows")
    paged.hstu_paged_append(k, v, pool.k, pool.v, pool.table, off, kv)
    assert torch.isnan(pool.k).all() and torch.isnan(pool.v).all()


def test_refusals():
    pool, q, k, v, off, kv = _setup(*CASES[1])
    args = (k, v, pool.k, pool.v, pool.table, off, kv)
    with pytest.raises(ValueError):
        paged.hstu_paged_append(*args, q=q)  # nothing to rotate it with
    with pytest.raises(TypeError):
        paged.hstu_paged_append(k, v, pool.k.float(), pool.v, pool.table, off, kv)
    with pytest.raises(ValueError):
        paged.hstu_paged_append(k, v, pool.k, pool.v.contiguous(), pool.table, off, kv)
    with pytest.raises(TypeError):
        paged.hstu_paged_append(k, v, pool.k, pool.v, pool.table[:3], off, kv)
    with pytest.raises(TypeError):
        paged.hstu_paged_append(k, v, pool.k, pool.v, pool.table, off.long(), kv)
    with pytest.raises(binding.HstuError) as e:  # page size 12
        c = torch.zeros((4, 12, 2, 64), dtype=torch.bfloat16, device="cuda")
        paged.hstu_paged_append(k, v, c, c.clone(), pool.table, off, kv)
    assert e.value.status == 2
    with pytest.raises(binding.HstuError) as e:  # K and V in one place
        paged.hstu_paged_append(k, v, pool.k, pool.k, pool.table, off, kv)
    assert e.value.status == 1
    flat = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.HstuError) as e:  # rows that lie in the cache
        paged.hstu_paged_append(flat.view(-1, 2, 64)[:k.shape[0]], v, flat, flat.clone(), pool.table, off, kv)
    assert e.value.status == 1
