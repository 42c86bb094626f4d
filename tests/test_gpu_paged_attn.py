"""GPU: hstu_paged_attn_fwd against fp64 (tests/paged_util.dense64, element by element within the
bound derived there; the oracle for long users), over every layout and page size, with NaN in all
places of the pool that no user owns."""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_util import assert_parity, dev_i32, to_f64
from hstu_pointwise_attention_jagged_b200 import binding, paged
from paged_util import Pool, bf16_normal, dense64, offsets_of

pytestmark = pytest.mark.gpu


LONG = 1 << 20  # a bound on the lengths that makes more than 16 rows a user take the tcgen05 kernel


class Batch:
    """users: (cached rows, new rows, candidates among them).  bound: max_kv, if not the longest length."""

    def __init__(self, users, page, H, d, layout="rows", seed=1, scale=1.0, alpha=None, bound=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.users, self.H, self.d = users, H, d
        lengths = [c + n for c, n, _ in users]
        new = [n for _, n, _ in users]
        self.pool = Pool(lengths, page, H, d, layout, seed)
        self.kv = [(bf16_normal(gen, L, H, d) * scale, bf16_normal(gen, L, H, d)) for L in lengths]
        for b, (k, v) in enumerate(self.kv):
            if lengths[b]:
                self.pool.put(b, 0, k, v)
        self.q = bf16_normal(gen, sum(new), H, d) * scale
        self.off, self.kv_len = offsets_of(new), dev_i32(lengths)
        self.nt = dev_i32([t for _, _, t in users])
        self.alpha, self.N = 1 / math.sqrt(d) if alpha is None else alpha, float(max(lengths + [1]))
        self.max_new, self.max_kv = max(new + [0]), bound or max(lengths + [0])
        self.starts = np.concatenate([[0], np.cumsum(new)])

    def run(self, **kw):
        p = self.pool
        a = dict(q=self.q, table=p.table, off=self.off, kv=self.kv_len, nt=self.nt, max_new=self.max_new,
                 max_kv=self.max_kv, out=None, k=p.k, v=p.v)
        a.update(kw)
        return paged.hstu_paged_attn_fwd(a["q"], a["k"], a["v"], a["table"], a["off"], a["kv"], a["nt"], self.alpha,
                                         self.N, a["max_new"], a["max_kv"], out=a["out"], stream=a.get("stream"))

    def check(self, out, only=None):
        got = to_f64(out)
        for b, (c, n, t) in enumerate(self.users):
            if n == 0 or (only is not None and b not in only):
                continue
            s = slice(self.starts[b], self.starts[b + 1])
            k, v = (to_f64(x) for x in self.kv[b])
            want, bound = dense64(to_f64(self.q[s]), k, v, c, n, t, self.alpha, self.N)
            err = np.abs(got[s] - want)
            assert (err <= bound).all(), (b, self.users[b], float((err / bound).max()), np.argwhere(~(err <= bound))[0])


# (users, page, H, layout)
SMALL = [
    ([(0, 1, 0)], 16, 1, "rows"),
    ([(0, 1, 1), (1, 1, 0), (5, 0, 0), (63, 1, 0), (64, 1, 1), (127, 1, 0), (128, 1, 1)], 8, 2, "rows"),
    ([(300, 1, 0)] * 9, 32, 4, "heads"),
    ([(700, 4, 3), (0, 0, 0), (255, 16, 0), (256, 16, 16), (257, 13, 5)], 16, 3, "halves"),
    ([(2000, 1, 0), (3, 2, 1), (4100, 1, 1)], 128, 1, "rows"),
    ([(100, 3, 1), (33, 1, 0)], 16, 3, "padded"),
    ([(1500, 7, 2), (90, 9, 9)], 1024, 2, "heads"),
]
LARGE = [
    ([(0, 17, 0)], 16, 1, "rows"),
    ([(0, 17, 0), (127, 1, 1), (0, 1, 0), (128, 16, 2), (5, 0, 0), (3, 64, 64)], 8, 2, "rows"),
    ([(300, 64, 3), (2000, 33, 33), (1, 63, 0)], 32, 1, "halves"),
    ([(0, 300, 40), (129, 128, 0), (128, 129, 1), (1000, 0, 0), (7, 257, 257), (513, 1, 0)], 16, 2, "rows"),
    ([(0, 128, 128), (384, 127, 3), (640, 200, 100)], 64, 3, "heads"),
    ([(900, 600, 500), (0, 64, 0)], 256, 1, "halves"),
    ([(1300, 40, 0)], 8, 4, "rows"),
    ([(1000, 300, 40), (77, 130, 0)], 32, 2, "padded"),
    ([(250, 33, 20)] * 30, 32, 2, "rows"),
    ([(100, 1100, 1000)], 1024, 2, "heads"),
]


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(SMALL)))
def test_few_rows(case, d):
    users, page, H, layout = SMALL[case]
    x = Batch(users, page, H, d, layout, seed=case + 1)
    x.check(x.run())
    x.check(x.run(max_kv=200000))  # a bound that makes it equal runs of tiles
    assert binding.hstu_attn_get_error() == 0


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(LARGE)))
def test_many_rows(case, d):
    users, page, H, layout = LARGE[case]
    x = Batch(users, page, H, d, layout, seed=case + 11)
    x.check(x.run())
    x.check(x.run(max_new=5000, max_kv=LONG))
    assert binding.hstu_attn_get_error() == 0


@pytest.mark.parametrize("users", [300, 1024, 1025, 5000])
def test_many_users_of_few_rows(users):
    """Ragged histories, some users without new rows, over the sizes at which the kernel's form changes."""
    rng = np.random.default_rng(users)
    new = rng.integers(0, 3, users)
    cached = np.minimum((30 * rng.lognormal(0, 1.5, users)).astype(int), 700)
    x = Batch([(int(c), int(n), int(rng.integers(0, n + 1))) for c, n in zip(cached, new)], 16, 1, 32, seed=users)
    x.check(x.run(), only=set(rng.choice(users, 200).tolist()) | {0, users - 1})
    assert binding.hstu_attn_get_error() == 0
    big = [(int(c), int(n), 0) for c, n in zip(cached, 20 * new)]  # the same through the tcgen05 kernel
    x = Batch(big, 16, 1, 32, seed=users + 1, bound=LONG)
    x.check(x.run(), only=set(rng.choice(users, 200).tolist()) | {0, users - 1})


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("new,bound", [(3, None), (150, None), (150, LONG)])
def test_page_sizes(page, new, bound):
    x = Batch([(page - 1, new, 1), (page, new, 0), (2 * page + 5, new, new)], page, 2, 64, "rows", seed=page, bound=bound)
    x.check(x.run())


@pytest.mark.parametrize("new", [16, 17, 64, 127, 128, 129])
def test_bounds_larger_than_the_batch(new):
    """max_new and max_kv are bounds: a looser one gives the same rows (within the error bound)."""
    x = Batch([(200, new, 5), (0, new, 0), (77, 1, 0)], 16, 2, 64, "rows", seed=new)
    x.check(x.run())
    x.check(x.run(max_new=4 * new, max_kv=20000))
    x.check(x.run(max_new=4 * new, max_kv=LONG))


@pytest.mark.parametrize("users", [[(5000, 1, 0), (40, 1, 1)], [(5000, 200, 100), (40, 60, 1)]])
def test_large_scores_and_alpha(users):
    """Scores of size 30 (SiLU near 0 and near x), a negative alpha, and alpha = 0."""
    x = Batch(users, 16, 1, 64, scale=3.0, alpha=0.5, seed=3)
    x.check(x.run())
    x.check(x.run(max_kv=LONG))
    for alpha in (-0.25, 0.0):
        x = Batch(users, 16, 1, 64, alpha=alpha, seed=4)
        x.check(x.run())
        x.check(x.run(max_kv=LONG))


@pytest.mark.parametrize("users,H,d,page", [([(33000, 2, 1)], 1, 128, 16), ([(20000, 1, 0), (12000, 16, 8)], 2, 64, 64),
                                            ([(9000, 700, 500), (30, 10, 0)], 2, 128, 32), ([(16000, 130, 0)], 1, 32, 128)])
def test_long_users(users, H, d, page):
    x = Batch(users, page, H, d, seed=9)
    out = to_f64(x.run())
    k, v = (np.concatenate([to_f64(a[i]) for a in x.kv]) for i in (0, 1))
    seq = np.concatenate([[0], np.cumsum([c + n for c, n, _ in users])]).astype(np.int32)
    want = oracle.fwd_cached(to_f64(x.q).astype(np.float32), k.astype(np.float32), v.astype(np.float32), seq,
                             np.array([t for _, _, t in users], np.int32), np.array([c for c, _, _ in users], np.int32),
                             x.alpha, x.N)
    assert_parity(out, want, what="paged long d=%d" % d, users=np.repeat(np.arange(len(users)), [n for _, n, _ in users]))


@pytest.mark.parametrize("new,bound", [(2, None), (140, None), (140, LONG)])
def test_equals_the_contiguous_call(new, bound):
    """The same batch through hstu_attn_fwd_cached: within both calls' error bound of fp64."""
    users = [(321, new, 1), (0, new, 0), (1000, new, new)]
    x = Batch(users, 16, 4, 128, seed=21, bound=bound)
    out = x.run()
    x.check(out)
    k, v = (torch.cat([a[i] for a in x.kv]) for i in (0, 1))
    seq = offsets_of([c + n for c, n, _ in users])
    x.check(binding.hstu_attn_fwd_cached(x.q, k, v, seq, x.nt, dev_i32([c for c, _, _ in users]), x.alpha, x.N, int(x.kv_len.max())))


@pytest.mark.parametrize("new,bound", [(3, None), (60, None), (60, LONG)])
def test_no_targets_argument_strides_and_guard_rows(new, bound):
    users = [(100, new, 0), (0, 0, 0), (17, new, 0)]
    x = Batch(users, 16, 2, 64, seed=5, bound=bound)
    want = x.run()
    x.check(want)
    assert torch.equal(x.run(nt=None), want)
    # q as a column block of a wider matrix, out as a row block of a larger one with guard rows
    total = x.q.shape[0]
    wide = torch.full((total, 3, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = x.q
    big = torch.full((total + 2, 2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    x.run(q=wide[:, 1], out=big[1:-1, 1])
    assert torch.equal(big[1:-1, 1], want)
    assert torch.all(big[0] == 7.0) and torch.all(big[-1] == 7.0) and torch.all(big[:, 0] == 7.0)


@pytest.mark.parametrize("new,long,bound", [(4, 2222, None), (4, 23000, None), (200, 2222, None), (200, 2222, LONG),
                                            (700, 9000, None)])
def test_deterministic_replayed_and_on_another_stream(new, long, bound):
    x = Batch([(600, new, 3), (long, new, new // 2), (0, new, 1)], 32, 4 if long < 9000 else 1, 128, seed=6, bound=bound)
    want = x.run()
    x.check(want)
    for _ in range(5):
        assert torch.equal(x.run(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = x.run(stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    # Two captured calls, replayed on two streams at once: they share nothing.
    graphs, outs = [], []
    for _ in range(2):
        out = torch.zeros_like(x.q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(out=out)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # The same graph on new lengths: user 0 forgets its candidates and its last rows.
    x.kv_len[0] -= 5
    again = x.run()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], again)


@pytest.mark.parametrize("new,bound", [(3, None), (40, None), (100, LONG)])
def test_a_user_does_not_see_its_neighbours_rows(new, bound):
    """q, K and V of one user are NaN: the others' outputs are what they were, bit for bit."""
    x = Batch([(77, new, 1), (130, new, 2), (40, new, 0)], 16, 2, 64, seed=12, bound=bound)
    want = x.run()
    x.check(want)
    x.q[x.starts[1]:x.starts[2]] = float("nan")
    x.pool.put(1, 0, *(torch.full_like(a, float("inf")) for a in x.kv[1]))
    got = x.run()
    assert torch.equal(got[:x.starts[1]], want[:x.starts[1]]) and torch.equal(got[x.starts[2]:], want[x.starts[2]:])


@pytest.mark.parametrize("new,bound", [(3, None), (40, None), (100, LONG)])
def test_decreasing_offsets(new, bound):
    """Offsets that step back: reported; the users before the step are computed, nothing else is touched
    beyond the rows the offsets name."""
    x = Batch([(50, new, 1)] * 4, 16, 2, 64, seed=13, bound=bound)
    off = dev_i32([0, new, 3 * new, 2 * new, 4 * new])
    big = torch.full((4 * new + 8, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    x.run(off=off, out=big[4:-4])
    assert binding.hstu_attn_get_error() == 4
    x.check(big[4:-4], only=[0])
    assert torch.all(big[:4] == 5.0) and torch.all(big[-4:] == 5.0)


@pytest.mark.parametrize("new,bound", [(2, None), (90, None), (90, LONG)])
def test_shared_prefix_pages(new, bound):
    """Two users whose first pages are the same pages."""
    x = Batch([(64, new, 1), (64, new, 1)], 16, 2, 64, seed=7, bound=bound)
    p = x.pool
    p.table_h[1, :4] = p.table_h[0, :4]
    table = dev_i32(p.table_h).view(p.table_h.shape)
    x.kv[1] = tuple(torch.cat([x.kv[0][i][:64], x.kv[1][i][64:]]) for i in (0, 1))
    x.check(x.run(table=table))


@pytest.mark.parametrize("new,bound", [(3, None), (50, None), (50, LONG)])
def test_bad_users_and_pages(new, bound):
    users = [(50, new, 1)] * 6
    x = Batch(users, 16, 2, 64, seed=8, bound=bound)
    kv = x.kv_len.clone()
    kv[1] = new - 1                      # shorter than its new rows
    nt = x.nt.clone()
    nt[2] = new + 1                      # more candidates than new rows
    nt[3] = -1
    kv[4] = 2 * LONG                     # longer than max_kv and its pages
    out = torch.full_like(x.q, 5.0)
    x.run(kv=kv, nt=nt, out=out)
    assert binding.hstu_attn_get_error() == 4
    assert binding.hstu_attn_get_error() == 0
    x.check(out, only=[0, 5])
    assert torch.all(out[x.starts[1]:x.starts[5]] == 5.0)
    # more new rows than max_new
    out.fill_(5.0)
    x.run(out=out, max_new=new - 1)
    assert binding.hstu_attn_get_error() == 4
    assert torch.all(out == 5.0)
    # offsets that do not end at the last row
    off = x.off.clone()
    off[6] -= 1
    x.run(off=off)
    assert binding.hstu_attn_get_error() == 4
    # a table entry outside the pool counts as a page of zeros
    for bad in (-1, x.pool.pages, 2 ** 31 - 1, -2 ** 31):
        table = x.pool.table.clone()
        table[0, 1] = bad
        k, v = (a.clone() for a in x.kv[0])
        k[16:32], v[16:32] = 0, 0
        keep, x.kv[0] = x.kv[0], (k, v)
        out = x.run(table=table)
        assert binding.hstu_attn_get_error() == 4
        x.check(out)
        x.kv[0] = keep


@pytest.mark.parametrize("users", [[(1200, 300, 20)] * 14, [(1200, 300, 0)] * 7 + [(0, 0, 0)] + [(900 + 40 * i, 290, 290) for i in range(8)],
                                   [(100 * i, 129 + 30 * i, 0) for i in range(1, 13)]], ids=["equal", "two kinds", "ragged"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_whole_items_and_pieces_in_one_plan(users, d):
    """A little more work than one round of whole items: the plan may cut the first users' items and leave the
    others whole."""
    x = Batch(users, 32, 4, d, seed=17, bound=LONG)
    out = x.run()
    x.check(out, only={0, 1, 3, len(users) - 1})
    assert torch.equal(out, x.run())


@pytest.mark.parametrize("page,d", [(16, 128), (256, 64), (8, 32)])
def test_abort_path_then_recovers(page, d):
    """The many-row kernel with every wait limited to 1 us: waits run out in the middle of it, it drains and
    returns, the device reports the timeout once, and a normal call is right afterwards."""
    x = Batch([(600, 129, 20), (300, 40, 3), (40, 300, 2)], page, 2, d, seed=15, bound=LONG)
    p = x.pool
    assert binding.hstu_attn_get_error() == 0
    for _ in range(2):
        paged.hstu_paged_selfcheck_fwd_timeout(x.q, p.k, p.v, p.table, x.off, x.kv_len, x.nt, x.alpha, x.N, x.max_new, x.max_kv,
                                               1000)
        assert binding.hstu_attn_get_error() == 5  # HSTU_ERR_TIMEOUT
        assert binding.hstu_attn_get_error() == 0
    x.check(x.run())
    assert binding.hstu_attn_get_error() == 0
    for bad in (0, 10 ** 9 + 1, -5):
        with pytest.raises(binding.HstuError) as e:
            paged.hstu_paged_selfcheck_fwd_timeout(x.q, p.k, p.v, p.table, x.off, x.kv_len, x.nt, x.alpha, x.N, x.max_new,
                                                   x.max_kv, limit_ns=bad)
        assert e.value.status == 1


@pytest.mark.parametrize("page,d", [(1024, 32), (256, 64), (64, 64), (128, 128), (64, 128), (32, 32)])
def test_many_short_pieces_with_few_copies_a_tile(page, d):
    """Few copies a tile leave a producer warp without one; it must not fall behind the others.  Short
    pieces of many users, repeated: no wait runs out (each would be reported) and nothing changes."""
    rng = np.random.default_rng(page + d)
    users = [(int(rng.integers(0, 300)), int(rng.choice([0, 1, 17, 40, 129])), 0) for _ in range(32)]
    x = Batch(users, page, 6, d, seed=14, bound=LONG)
    want = x.run()
    x.check(want)
    for _ in range(300):
        got = x.run()
    assert binding.hstu_attn_get_error() == 0
    assert torch.equal(got, want)


def test_nothing_to_do():
    x = Batch([(5, 0, 0), (0, 0, 0)], 16, 1, 32)
    assert x.run().shape == (0, 1, 32)


@pytest.mark.parametrize("new,bound", [(1, None), (40, None), (40, LONG)])
def test_cache_past_32_bit_offsets(new, bound):
    """Pages whose element offsets do not fit 32 bits: a pool of 2^32 elements' reach, a few pages of it used."""
    H, d, page = 2, 128, 16
    rows = (1 << 32) // (H * d) // page + 40
    k = torch.empty((rows, page, H, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    x = Batch([(70, new, 0)], page, H, d, seed=10, bound=bound)
    x.pool.table_h[0, :(70 + new + page - 1) // page] = rows - 1 - 3 * np.arange((70 + new + page - 1) // page)
    x.pool.k, x.pool.v = k, v
    x.pool.put(0, 0, *x.kv[0])
    table = dev_i32(x.pool.table_h).view(x.pool.table_h.shape)
    x.check(x.run(table=table))
    paged.hstu_paged_append(x.kv[0][0][70:], x.kv[0][1][70:], k, v, table, x.off, x.kv_len)
    x.check(x.run(table=table))
    assert binding.hstu_attn_get_error() == 0


def test_refusals():
    x = Batch([(50, 3, 1)], 16, 2, 64)
    with pytest.raises(binding.HstuError) as e:
        x.run(out=x.q)
    assert e.value.status == 1
    with pytest.raises(binding.HstuError) as e:
        x.run(max_new=-1)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        x.run(q=x.q[:, :1].contiguous())
    with pytest.raises(TypeError):
        x.run(q=x.q.half())
    with pytest.raises(TypeError):
        x.run(nt=x.nt.long())
    with pytest.raises(ValueError):
        x.run(v=x.pool.v[:-1])
