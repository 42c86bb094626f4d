"""GPU: the rotation's angles at far positions, for frequencies of both signs.  A pair (1, 0) becomes
(cos t, sin t), and where one of them is near zero its bf16 value resolves the angle itself."""
import numpy as np
import pytest
import torch

from gpu_util import dev_i32, to_f64
from hstu_pointwise_attention_jagged_b200 import binding, paged
from paged_util import Pool, bf16_normal, offsets_of, rotate64, rotation_bound

pytestmark = pytest.mark.gpu

# Error of the angle for |freq| <= 1 and |pos| <= 2^31, in radians: the two fp64 roundings of freq / 2 pi (the
# constant's and the product's), 2^-53 each of at most 0.1592 turns, times the position, 4.8e-7; the 2^-64 turns
# cut off from it, times the position, 7.3e-10; the 2^-32 turns cut off from the product, 1.5e-9; and its rounding
# to fp32, 2^-25 turns, 1.9e-7: 6.7e-7 in all.  The pair's other entry is zero, so nothing is added to the
# product with 1; sincospif is good to two steps (2^-22 of the value), and the value is rounded to bf16 once, 2^-8.
ANGLE = 6.7e-7
VALUE = 2.0 ** -8 + 2.0 ** -21


def _far(rows, pairs, seed):
    rng = np.random.default_rng(seed)
    pos = (rng.integers(2 ** 31 - 2 ** 27, 2 ** 31, rows) * rng.choice([-1, 1], rows)).astype(np.int32)
    return pos, rng.uniform(0.5, 1.0, pairs)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_angles_at_far_positions(sign, inverse):
    rows, pairs = 60000, 64
    pos, freqs = _far(rows, pairs, 3)
    freqs = sign * freqs
    x = torch.zeros((rows, 1, 2 * pairs), dtype=torch.bfloat16, device="cuda")
    x[..., :pairs] = 1.0
    got, _ = paged.hstu_rotary(x, None, dev_i32(pos), torch.from_numpy(freqs).cuda(), inverse=inverse)
    got = to_f64(got)[:, 0]
    t = pos.astype(np.longdouble)[:, None] * freqs.astype(np.longdouble) * (-1 if inverse else 1)
    for have, want in ((got[:, :pairs], np.cos(t)), (got[:, pairs:], np.sin(t))):
        want = want.astype(np.float64)
        err, bound = np.abs(have - want), ANGLE + np.abs(want) * VALUE
        assert (err <= bound).all(), (float((err / bound).max()), int((err > bound).sum()))


def test_negative_frequencies_in_both_calls():
    """hstu_rotary by negative frequencies against the formula, and hstu_paged_append bit for bit like it."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    rows, H, d = 333, 2, 64
    q, k, v = (bf16_normal(gen, rows, H, d) for _ in range(3))
    pos, freqs = _far(rows, d // 2, 4)
    freqs[::2] *= -1
    p, f = dev_i32(pos), torch.from_numpy(freqs).cuda()
    wq, wk = paged.hstu_rotary(q, k, p, f)
    for got, x in ((wq, q), (wk, k)):
        want = rotate64(to_f64(x), pos[None], freqs, [d // 2])
        assert (np.abs(to_f64(got) - want) <= rotation_bound(to_f64(x), want, d // 2, False)).all()
    pool = Pool([rows], 16, H, d, seed=3)
    out = paged.hstu_paged_append(k, v, pool.k, pool.v, pool.table, offsets_of([rows]), dev_i32([rows]), q=q, positions=p,
                                  freqs=f)
    assert binding.hstu_attn_get_error() == 0
    assert torch.equal(out, wq) and torch.equal(pool.rows(0, 0, rows)[0], wk)
