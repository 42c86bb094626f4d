"""hstu_paged_append refuses caches in which one element belongs to two places, and takes every layout in which
K and V only interleave."""
import numpy as np
import pytest

from test_paged_abi import INVALID, _append, _cache, lib  # noqa: F401  (lib: fixture)

K = 1 << 30  # address of K; pages of 16 rows, 2 heads, d = 64: 4096 bytes a page, 8 pages


@pytest.mark.parametrize("shift", [16, 64, 128, 256, 4096, 7 * 4096, 7 * 4096 + 15 * 256 + 128 + 112])
def test_v_shifted_into_k_is_refused(lib, shift):
    """V begins inside K: at another column, head, row or page."""
    for sign in (1, -1):
        assert _append(lib, _cache(v=K + sign * shift)) == INVALID, (sign, shift)


def test_interleaved_k_and_v_that_meet_are_refused(lib):
    """Halves of [pages, 2, 16, 2, 64] (a page of either at every second 4096 bytes), V off by some rows."""
    for shift in (4096 - 256, 4096 + 256, 4096 + 128, 15 * 4096 - 16):
        assert _append(lib, _cache(page_stride=2 * 2048, v=K + shift)) == INVALID, shift


@pytest.mark.parametrize("strides", [dict(row_stride=64, head_stride=64), dict(row_stride=120),
                                     dict(page_stride=2048 - 8), dict(page_stride=64), dict(row_stride=64, head_stride=512)])
def test_rows_that_share_elements_are_refused(lib, strides):
    assert _append(lib, _cache(**strides)) == INVALID, strides


def _layouts(torch, pages, page, H, d):
    def full(*shape):
        return torch.full(shape, 3.0, dtype=torch.bfloat16, device="cuda")
    a = full(pages, page, 2, H, d)
    yield "rows by turns", a, a[:, :, 0], a[:, :, 1]
    a = full(pages, page, H, 2, d)
    yield "heads by turns", a, a[:, :, :, 0], a[:, :, :, 1]
    a = full(pages, page, H, 2 * d)
    yield "columns by turns", a, a[..., d:], a[..., :d]
    a = full(2, page, pages, H, d)
    yield "pages within rows", a, a[0].transpose(0, 1), a[1].transpose(0, 1)
    a = full(H, 2, pages, page, d)
    yield "heads outermost", a, a[:, 0].permute(1, 2, 0, 3), a[:, 1].permute(1, 2, 0, 3)
    a = full(pages * page + 1, 2, H, d)
    yield "V a row behind K", a, a[:-1, 0].view(pages, page, H, d), a[1:, 1].view(pages, page, H, d)


@pytest.mark.gpu
@pytest.mark.parametrize("H,pages", [(2, 5), (1, 5), (3, 1)])
def test_layouts_that_only_interleave(H, pages):
    """Every row at its place, and nothing else of the tensor that both are part of touched."""
    import torch

    from gpu_util import dev_i32
    from hstu_pointwise_attention_jagged_b200 import binding, paged
    from paged_util import bf16_normal
    page, d = 8, 64
    n = pages * page - 3
    gen = torch.Generator(device="cuda").manual_seed(H)
    k, v = (bf16_normal(gen, n, H, d) for _ in range(2))
    order = np.random.default_rng(pages).permutation(pages).astype(np.int32)
    table = dev_i32(order).view(1, pages)
    at = torch.from_numpy(order[np.arange(n) // page].astype(np.int64)).cuda(), torch.from_numpy(np.arange(n) % page).cuda()
    layouts = [x[0] for x in _layouts(torch, pages, page, H, d)]
    for i, name in enumerate(layouts):
        _, want, wk, wv = list(_layouts(torch, pages, page, H, d))[i]
        wk[at], wv[at] = k, v
        _, got, ck, cv = list(_layouts(torch, pages, page, H, d))[i]
        paged.hstu_paged_append(k, v, ck, cv, table, dev_i32([0, n]), dev_i32([n]))
        assert binding.hstu_attn_get_error() == 0
        assert torch.equal(got, want), name
