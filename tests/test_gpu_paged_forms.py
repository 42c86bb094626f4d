"""GPU: the forms of the paged attention's kernels that only batches of many users, or of certain amounts of
work, reach; each test also shows that its form ran.

Few rows a user: equal runs of tiles take a workspace, clusters take none, which a captured call's allocations tell.
Many rows a user: whether an item was cut is seen in its sums.  V holds +2^60 in one tile and -2^60 in the next, the
last two of the history, and 1 elsewhere: one fp32 sum over all tiles loses what came before them, while a piece's
own sum keeps it."""
import numpy as np
import pytest
import torch

from gpu_util import to_f64
from hstu_pointwise_attention_jagged_b200 import binding
from test_gpu_paged_attn import LONG, Batch

pytestmark = pytest.mark.gpu


def allocations(call):
    """Bytes of each allocation node of the captured call."""
    from cuda.bindings import runtime as rt
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    handle = rt.cudaGraph_t(graph.raw_cuda_graph())
    err, _, count = rt.cudaGraphGetNodes(handle, 0)
    assert err == rt.cudaError_t.cudaSuccess
    err, nodes, count = rt.cudaGraphGetNodes(handle, count)
    assert err == rt.cudaError_t.cudaSuccess
    kinds = [(node, rt.cudaGraphNodeGetType(node)[1]) for node in nodes[:count]]
    return [int(rt.cudaGraphMemAllocNodeGetParams(node)[1].bytesize) for node, kind in kinds
            if kind == rt.cudaGraphNodeType.cudaGraphNodeTypeMemAlloc]


def _ragged(users, most, longest, seed):
    """Up to `most` new rows for each user on lognormal histories; long runs of users bring none."""
    rng = np.random.default_rng(seed)
    new = rng.integers(0, most + 1, users)
    for at in (0, users // 3, users - users // 8):  # the first, some in the middle and the last users
        new[at:at + users // 8] = 0
    new[users // 2] = most
    cached = np.minimum((longest / 8 * rng.lognormal(0, 1.5, users)).astype(int), longest)
    return [(int(c), int(n), int(rng.integers(0, n + 1))) for c, n in zip(cached, new)]


@pytest.mark.parametrize("d,H,most,longest", [(32, 1, 2, 700), (32, 3, 12, 300), (64, 2, 8, 500), (128, 1, 16, 300)])
@pytest.mark.parametrize("users", [129, 300, 1000, 1024, 1025, 5000])
def test_equal_runs_of_many_users(users, d, H, most, longest):
    """Up to 1024 users as equal runs of tiles (a bound on the lengths that makes them long), more as clusters."""
    batch = _ragged(users, most, longest, users + d)
    x = Batch(batch, 16, H, d, seed=users)
    wide = dict(max_kv=200000)
    assert (allocations(lambda: x.run(**wide)) != []) == (users <= 1024)
    out = x.run(**wide)
    rng = np.random.default_rng(users)
    x.check(out, only=set(rng.choice(users, 250 if users > 250 else users, replace=False).tolist()) | {0, users // 2, users - 1})
    assert torch.equal(x.run(**wide), out)
    assert binding.hstu_attn_get_error() == 0


@pytest.mark.parametrize("d,longest", [(128, 3000), (64, 6000)])
def test_equal_runs_of_many_long_users(d, longest):
    """More than 128 users, so that a thread scans several, of many tiles each; no bound but the lengths."""
    batch = _ragged(200, 3, longest, d)
    batch[100] = (longest, 3, 1)
    x = Batch(batch, 32, 2, d, "heads", seed=d)
    assert allocations(x.run) != []
    x.check(x.run())
    assert binding.hstu_attn_get_error() == 0


@pytest.mark.parametrize("place", [0, 500, 1023])
def test_equal_runs_of_one_user_among_many(place):
    """Every other user brings no rows, whether it has a history or not."""
    batch = [(int(i % 3) * 40, 0, 0) for i in range(1024)]
    batch[place] = (9000, 5, 2)
    x = Batch(batch, 16, 2, 64, seed=place + 1)
    assert allocations(x.run) != []
    x.check(x.run())
    assert binding.hstu_attn_get_error() == 0


@pytest.mark.parametrize("users", [255, 256, 257, 1025, 5000])
def test_many_rows_of_many_users(users):
    """The plan with and without its per-user values on chip; no user is reported."""
    batch = [(c, 20 * n, 0) for c, n, _ in _ragged(users, 3, 400, users)]
    x = Batch(batch, 16, 1, 32, seed=users, bound=LONG)
    out = x.run()
    assert binding.hstu_attn_get_error() == 0
    rng = np.random.default_rng(users)
    x.check(out, only=set(rng.choice(users, 200, replace=False).tolist()) | {0, users - 1})
    assert torch.equal(x.run(), out)


# users (all new rows are candidates on whole tiles of history), H, and whether some items are cut, some whole
CUTS = {
    "equal": ([(3072, 300, 300)] * 16, 4, True, True),
    "one user": ([(8192, 200, 200)], 4, True, False),
    "ragged": ([(128 * (4 + 2 * i), 129 + 30 * i, 129 + 30 * i) for i in range(1, 15)], 4, True, True),
    "mixed": ([(128 * (8 + (5 * i) % 13), 60 + (71 * i) % 400, 60 + (71 * i) % 400) for i in range(20)], 4, True, True),
    "many": ([(384, 128, 128)] * 160, 4, False, True),
}


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("case", list(CUTS))
def test_cut_and_whole_items(case, d):
    users, H, some_cut, some_whole = CUTS[case]
    x = Batch(users, 64, H, d, seed=len(users), bound=LONG)
    x.check(x.run())
    x.q.fill_(1.0)
    x.alpha, x.N = 1.0 / d, 1.0  # every score is 1
    for b, (c, n, _) in enumerate(users):
        v = torch.ones((c + n, H, d), dtype=torch.bfloat16, device="cuda")
        v[c - 256:c - 128, :, 0] = 2.0 ** 60
        v[c - 128:c, :, 0] = -2.0 ** 60
        x.pool.put(b, 0, torch.ones_like(v), v)
    out = x.run()
    assert binding.hstu_attn_get_error() == 0
    assert torch.equal(x.run(), out)
    out = to_f64(out)
    weight = 1.0 / (1.0 + np.exp(-1.0))
    cut = []
    for b, (c, n, _) in enumerate(users):
        for at in range(int(x.starts[b]), int(x.starts[b + 1]), 128):
            item = out[at:min(at + 128, int(x.starts[b + 1]))]
            assert (item == item[:1]).all()  # every row of a block sees the same
            # The other columns: c + 1 weights of one size, each off by 2^-8 and the tanh's 2^-10.9 / 2, and a rounding.
            assert (np.abs(item[..., 1:] / (weight * (c + 1)) - 1.0) < 2.0 ** -8 * 2 + 2.0 ** -10.9).all()
            kept = item[0, :, 0]
            lost = np.abs(kept - weight) < 0.01  # the row itself
            assert (lost | (kept > 90.0)).all()  # or at least one whole tile before the last piece
            cut += (~lost).tolist()
    assert any(cut) == some_cut and any(not c for c in cut) == some_whole, (sum(cut), len(cut))
