"""GPU: what the paged attention takes from the library's memory pool, read from a captured call's allocation
nodes, against the bound that include/hstu_paged.h states."""
import pytest
import torch

from gpu_util import dev_i32
from hstu_pointwise_attention_jagged_b200 import binding, paged

pytestmark = pytest.mark.gpu


class Call:
    """`users` users with `new` new rows on `cached` rows; all of them read the same pages."""

    def __init__(self, users, cached, new, H, d, max_kv=None, page=128):
        L = cached + new
        pages = -(-L // page)
        gen = torch.Generator(device="cuda").manual_seed(1)
        self.k, self.v = (torch.randn((pages, page, H, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
        self.q = torch.randn((users * new, H, d), generator=gen, device="cuda").to(torch.bfloat16)
        self.table = dev_i32([list(range(pages))] * users)
        self.off, self.kv_len = dev_i32([new * b for b in range(users + 1)]), dev_i32([L] * users)
        self.new, self.max_kv = new, max_kv or L
        self.out = torch.empty_like(self.q)

    def run(self, stream=None):
        return paged.hstu_paged_attn_fwd(self.q, self.k, self.v, self.table, self.off, self.kv_len, None, 0.1, 100.0,
                                         self.new, self.max_kv, out=self.out, stream=stream)

    def workspace(self):
        """Bytes of each allocation of the captured call."""
        from cuda.bindings import runtime as rt
        self.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(graph):
            self.run()
        handle = rt.cudaGraph_t(graph.raw_cuda_graph())
        err, _, count = rt.cudaGraphGetNodes(handle, 0)
        assert err == rt.cudaError_t.cudaSuccess
        err, nodes, count = rt.cudaGraphGetNodes(handle, count)
        sizes = []
        for node in nodes[:count]:
            err, kind = rt.cudaGraphNodeGetType(node)
            assert err == rt.cudaError_t.cudaSuccess
            if kind == rt.cudaGraphNodeType.cudaGraphNodeTypeMemAlloc:
                err, params = rt.cudaGraphMemAllocNodeGetParams(node)
                assert err == rt.cudaError_t.cudaSuccess
                sizes.append(int(params.bytesize))
        return sizes


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# users, cached, new, H, d, max_kv, pieces a call may be cut into at most (None: four for each SM)
CASES = [
    (16, 3000, 2348, 4, 128, None, 0),       # 304 blocks of 4 heads: too many to cut
    (1, 20000, 20000, 4, 64, None, 0),       # one user's 157 blocks
    (300, 500, 40, 2, 64, 1 << 20, 0),       # more users than the plan keeps on chip
    (20, 100, 129, 4, 128, 380, 160 * 2),    # room for 160 items of at most 4 tiles
    (1, 1000, 100, 2, 32, 1 << 20, 2 * 16),  # one item a head, any length
    (16, 3000, 300, 4, 128, None, None),
    (64, 400, 24, 4, 128, 100000, None),
]


@pytest.mark.parametrize("case", CASES)
def test_workspace_of_many_rows(case):
    users, cached, new, H, d, max_kv, pieces = case
    call = Call(users, cached, new, H, d, max_kv)
    items = H * (users * new // 128 + users)
    if pieces is None:
        pieces = 4 * _sms()
    sizes = call.workspace()
    assert len(sizes) == 1
    # The queue holds the pieces too; counters and padding come on top.
    assert sizes[0] <= 48 * items + pieces * (512 * d + 48 + 16) + 4 * (users + 1) + 2048, sizes
    assert binding.hstu_attn_get_error() == 0


def test_workspace_of_few_rows():
    assert Call(8, 300, 3, 2, 64).workspace() == []
    sizes = Call(64, 4000, 1, 4, 128, 40000).workspace()
    assert len(sizes) == 1 and sizes[0] <= 256 * 128 * _sms() + 8 * 64 * 4 + 512


def test_pool_keeps_two_concurrent_workspaces():
    """Two calls in flight on two streams, each with the largest workspace: a synchronisation gives none of their
    memory back, so the next ones find it there."""
    calls = [Call(16, 3000, 300, 4, 128) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    free = []
    for _ in range(3):
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        for call, stream in zip(calls, streams):
            with torch.cuda.stream(stream):
                torch.cuda._sleep(40_000_000)  # some 20 ms: neither call ends before the other has its memory
                call.run()
        during = torch.cuda.mem_get_info()[0]
        torch.cuda.synchronize()
        free.append((before, during, torch.cuda.mem_get_info()[0]))
    # The first pair of calls may still grow the pool; from then on it neither shrinks nor grows.
    assert all(after == during for _, during, after in free), free
    assert all(during == before for before, during, _ in free[1:]), free
    assert binding.hstu_attn_get_error() == 0
