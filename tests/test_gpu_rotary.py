"""GPU: hstu_rotary against the formula in 64 bits (tests/paged_util.py), element by element within
the bound that function derives, and its inverse as the gradient: against the formula and against
the differences of the (linear) forward along every column."""
import numpy as np
import pytest
import torch

from gpu_util import dev_i32, to_f64
from hstu_pointwise_attention_jagged_b200 import binding, paged
from paged_util import bf16_normal, rotate64, rotation_bound

pytestmark = pytest.mark.gpu


def _case(rows, H, d, pairs, axes, seed, far=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    q, k = bf16_normal(gen, rows, H, d), bf16_normal(gen, rows, H, d)
    cut = np.sort(rng.integers(0, pairs + 1, axes - 1))
    sections = np.diff(np.concatenate([[0], cut, [pairs]])).astype(int).tolist()
    hi = 2 ** 31 - 1 if far else 20000
    pos = rng.integers(-hi if far else 0, hi, size=(axes, rows), endpoint=True).astype(np.int32)
    if far and rows > 1:
        pos[:, 0], pos[:, -1] = -2 ** 31, 2 ** 31 - 1
    freqs = 10000.0 ** (-np.arange(pairs) / pairs)
    return q, k, pos, freqs, sections


def _check(got, x, pos, freqs, sections, interleaved, inverse):
    x64 = to_f64(x)
    want = rotate64(x64, pos, freqs, sections, interleaved, inverse)
    err = np.abs(to_f64(got) - want)
    bound = rotation_bound(x64, want, len(freqs), interleaved)
    assert (err <= bound).all(), float((err / bound).max())
    if 2 * len(freqs) < x.shape[2]:
        assert torch.equal(got[..., 2 * len(freqs):], x[..., 2 * len(freqs):])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,H,d,pairs,axes", [(1, 1, 32, 8, 1), (1, 4, 128, 64, 2), (17, 3, 64, 32, 1), (300, 2, 32, 16, 4),
                                                 (1000, 5, 128, 24, 3), (2049, 1, 128, 64, 1), (33, 16, 64, 8, 2),
                                                 (5000, 2, 64, 32, 2), (7, 70, 128, 64, 1)])
def test_rotary_matches_formula(rows, H, d, pairs, axes, interleaved):
    q, k, pos, freqs, sections = _case(rows, H, d, pairs, axes, rows + d)
    f = torch.from_numpy(freqs).cuda()
    for inverse in (False, True):
        qo, ko = paged.hstu_rotary(q, k, dev_i32(pos).view(pos.shape), f, sections, interleaved, inverse)
        _check(qo, q, pos, freqs, sections, interleaved, inverse)
        _check(ko, k, pos, freqs, sections, interleaved, inverse)


def test_far_positions():
    """Positions over the whole int32 range, where an fp32 angle would have no digit left."""
    q, k, pos, freqs, sections = _case(512, 2, 64, 32, 2, 5, far=True)
    qo, _ = paged.hstu_rotary(q, k, dev_i32(pos).view(pos.shape), torch.from_numpy(freqs).cuda(), sections)
    _check(qo, q, pos, freqs, sections, False, False)


def test_q_alone_one_axis_vector():
    q, _, pos, freqs, _ = _case(50, 2, 64, 16, 1, 6)
    qo, ko = paged.hstu_rotary(q, None, dev_i32(pos[0]), torch.from_numpy(freqs).cuda())
    assert ko is None
    _check(qo, q, pos, freqs, [16], False, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_and_in_place(interleaved):
    """Q and K as columns of one [U | V | Q | K] buffer: out of place, then in place; U and V stay."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    rows, H, d = 777, 4, 128
    wide = bf16_normal(gen, rows, 4, H, d)
    before = wide.clone()
    _, _, pos, freqs, sections = _case(rows, H, d, 64, 2, 9)
    p, f = dev_i32(pos).view(pos.shape), torch.from_numpy(freqs).cuda()
    qo, ko = paged.hstu_rotary(wide[:, 2], wide[:, 3], p, f, sections, interleaved)
    assert torch.equal(wide, before)
    _check(qo, before[:, 2], pos, freqs, sections, interleaved, False)
    _check(ko, before[:, 3], pos, freqs, sections, interleaved, False)
    paged.hstu_rotary(wide[:, 2], wide[:, 3], p, f, sections, interleaved, q_out=wide[:, 2], k_out=wide[:, 3])
    assert torch.equal(wide[:, :2], before[:, :2])
    assert torch.equal(wide[:, 2], qo) and torch.equal(wide[:, 3], ko)
    # positions with a row stride of their own
    loose = torch.zeros((2, rows + 5), dtype=torch.int32, device="cuda")
    loose[:, :rows] = p
    again, _ = paged.hstu_rotary(before[:, 2], None, loose[:, :rows], f, sections, interleaved)
    assert torch.equal(again, qo)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_by_differences(interleaved):
    """The forward is linear: along column c its difference quotient is rot(e_c), for any step.  So
    the gradient of <g, rot(x)> in column c is <g, rot(e_c)>, which the inverse of g must give.  Bound:
    rot(e_c) has two entries, each rounded to bf16 (2^-8 of it, at most 1), against g; the gradient is
    rounded once more."""
    H, d, pairs = 1, 32, 16
    gen = torch.Generator(device="cuda").manual_seed(11)
    g = bf16_normal(gen, d, H, d)          # row c: the loss gradient used with e_c
    pos = np.full((1, d), 1234, np.int32)
    freqs = 10000.0 ** (-np.arange(pairs) / pairs)
    f = torch.from_numpy(freqs).cuda()
    eye = torch.eye(d, device="cuda").to(torch.bfloat16)[:, None, :].contiguous()
    grad, _ = paged.hstu_rotary(g, None, dev_i32(pos).view(pos.shape), f, [pairs], interleaved, inverse=True)
    for step in (1.0, 0.25):
        up, _ = paged.hstu_rotary(eye * step, None, dev_i32(pos).view(pos.shape), f, [pairs], interleaved)
        down, _ = paged.hstu_rotary(eye * -step, None, dev_i32(pos).view(pos.shape), f, [pairs], interleaved)
        quotient = (to_f64(up) - to_f64(down)) / (2 * step)
        want = (to_f64(g) * quotient).sum(-1)[:, 0]
        got = to_f64(grad)[np.arange(d), 0, np.arange(d)]
        gmax = np.abs(to_f64(g)).max(-1)[:, 0]
        assert (np.abs(got - want) <= 2 * gmax * 2.0 ** -8 + np.abs(want) * 2.0 ** -8 + 1e-6).all()


def test_round_trip_and_determinism():
    q, k, pos, freqs, sections = _case(400, 3, 64, 32, 1, 13)
    p, f = dev_i32(pos).view(pos.shape), torch.from_numpy(freqs).cuda()
    a, b = paged.hstu_rotary(q, k, p, f, sections)
    a2, b2 = paged.hstu_rotary(q, k, p, f, sections)
    assert torch.equal(a, a2) and torch.equal(b, b2)
    back, _ = paged.hstu_rotary(a, None, p, f, sections, inverse=True)
    # Two roundings to bf16 of a pair of norm r: each entry off by at most 2 * 2^-8 * r (and the angles).
    x = to_f64(q)
    r = np.sqrt(x[..., :32] ** 2 + x[..., 32:] ** 2)
    assert (np.abs(to_f64(back) - x) <= 2.5 * 2.0 ** -8 * np.concatenate([r, r], -1) + 1e-6).all()


def test_other_stream_and_graph():
    q, k, pos, freqs, sections = _case(600, 2, 128, 64, 2, 14)
    p, f = dev_i32(pos).view(pos.shape), torch.from_numpy(freqs).cuda()
    want, _ = paged.hstu_rotary(q, None, p, f, sections)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = paged.hstu_rotary(q, None, p, f, sections, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    buf, out = q.clone(), torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        paged.hstu_rotary(buf, None, p, f, sections, q_out=out)
    buf.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, paged.hstu_rotary(k, None, p, f, sections)[0])


def test_empty_and_non_finite():
    f = paged.hstu_rotary_freqs(16)
    q = torch.empty((0, 2, 32), dtype=torch.bfloat16, device="cuda")
    qo, ko = paged.hstu_rotary(q, q, torch.empty(0, dtype=torch.int32, device="cuda"), f)
    assert qo.shape == (0, 2, 32) and ko.shape == (0, 2, 32)
    # A NaN stays in its pair: other rows, heads and pairs are untouched by it.
    q = torch.ones((3, 2, 32), dtype=torch.bfloat16, device="cuda")
    q[1, 0, 5] = float("nan")
    qo, _ = paged.hstu_rotary(q, None, dev_i32(np.arange(3)), f)
    bad = torch.isnan(qo)
    assert bad[1, 0, 5] and bad[1, 0, 21] and int(bad.sum()) == 2


def test_refusals():
    q = torch.zeros((8, 2, 64), dtype=torch.bfloat16, device="cuda")
    f, pos = paged.hstu_rotary_freqs(32), dev_i32(np.arange(8))
    with pytest.raises(TypeError):
        paged.hstu_rotary(q.float(), None, pos, f)
    with pytest.raises(TypeError):
        paged.hstu_rotary(q, None, pos, f.float())
    with pytest.raises(ValueError):
        paged.hstu_rotary(q, None, dev_i32(np.arange(9)), f)
    with pytest.raises(ValueError):
        paged.hstu_rotary(q, torch.zeros((8, 3, 64), dtype=torch.bfloat16, device="cuda"), pos, f)
    with pytest.raises(TypeError):
        paged.hstu_rotary(q.transpose(0, 1), None, dev_i32(np.arange(2)), f)
    for bad in (dict(sections=[31]), dict(sections=[40, -8])):
        with pytest.raises((binding.HstuError, ValueError)):
            paged.hstu_rotary(q, None, dev_i32(np.zeros((len(bad["sections"]), 8))).view(-1, 8), f, **bad)
    with pytest.raises(binding.HstuError) as e:  # 2 * pairs > d
        paged.hstu_rotary(q, None, pos, paged.hstu_rotary_freqs(40))
    assert e.value.status == 1
    with pytest.raises(binding.HstuError) as e:  # pairs not a multiple of 8
        paged.hstu_rotary(q, None, pos, paged.hstu_rotary_freqs(12))
    assert e.value.status == 2
    with pytest.raises(binding.HstuError) as e:  # output over the other input
        paged.hstu_rotary(q, q.clone(), pos, f, k_out=q)
    assert e.value.status == 1
    big = torch.zeros((16, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.HstuError) as e:  # shifted over its own input
        paged.hstu_rotary(big[:8], None, pos, f, q_out=big[4:12])
    assert e.value.status == 1
    with pytest.raises(binding.HstuError) as e:  # head size
        paged.hstu_rotary(torch.zeros((8, 2, 96), dtype=torch.bfloat16, device="cuda"), None, pos, f)
    assert e.value.status == 2
