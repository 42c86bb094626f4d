"""GPU: the paged calls together, as a serving process uses them, against the framework's calls on whole
sequences.  Requests arrive in rounds; each brings some new events and candidates of every user.
hstu_paged_append writes both (rotating K and Q), hstu_paged_attn_fwd scores them, and the candidates are
forgotten by keeping only the history's length, so the next round overwrites them.  The result of
every round is what hstu_attn_fwd gives on the whole sequence with Q and K rotated by hstu_rotary:
both are compared with fp64 on the same rotated rows, within the bound of paged_util.dense64."""
import math

import numpy as np
import pytest
import torch

from gpu_util import dev_i32, to_f64
from hstu_pointwise_attention_jagged_b200 import (hstu_attn_fwd, hstu_attn_get_error, hstu_paged_append,
                                                  hstu_paged_attn_fwd, hstu_rotary, hstu_rotary_freqs)
from paged_util import Pool, bf16_normal, dense64, offsets_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,page,layout", [(64, 16, "rows"), (128, 64, "heads"), (32, 8, "halves")])
def test_serving_rounds(d, page, layout):
    H, users = 2, 5
    rng = np.random.default_rng(d)
    gen = torch.Generator(device="cuda").manual_seed(d)
    rounds = [([200, 0, 37, 1, 512], [0, 0, 3, 1, 0]), ([1, 1, 1, 1, 1], [2, 0, 5, 0, 1]), ([0, 130, 4, 0, 9], [300, 8, 0, 0, 40]),
              ([1, 0, 0, 2, 1], [0, 0, 0, 0, 0])]
    history = [sum(r[0][b] for r in rounds) for b in range(users)]
    pool = Pool([h + 320 for h in history], page, H, d, layout, seed=d)
    freqs = torch.cat([hstu_rotary_freqs(d // 4), 2 * math.pi / (60.0 * hstu_rotary_freqs(d // 4, 1e5).reciprocal())])
    sections = [d // 4, d // 4]
    kept = [[torch.empty((0, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(users)]
    length = np.zeros(users, np.int64)
    alpha, N = 1 / math.sqrt(d), 700.0
    for events, cands in rounds:
        events, cands = np.array(events), np.array(cands)
        new = events + cands
        total = int(new.sum())
        q, k, v = (bf16_normal(gen, total, H, d) for _ in range(3))
        # a candidate stands at the next place of its user's history; times are seconds
        place = np.concatenate([np.r_[np.arange(L, L + e), np.full(t, L + e)] for L, e, t in zip(length, events, cands)])
        when = 1_700_000_000 + rng.integers(0, 10 ** 8, total)
        pos = dev_i32(np.stack([place, when])).view(2, total)
        kv_len, off = dev_i32(length + new), offsets_of(new)
        qr = hstu_paged_append(k, v, pool.k, pool.v, pool.table, off, kv_len, q=q, positions=pos, freqs=freqs,
                               sections=sections)
        out = hstu_paged_attn_fwd(qr, pool.k, pool.v, pool.table, off, kv_len, dev_i32(cands), alpha, N, int(new.max()),
                                  int((length + new).max()))
        assert hstu_attn_get_error() == 0
        q2, k2 = hstu_rotary(q, k, pos, freqs, sections)
        assert torch.equal(q2, qr)
        # whole sequences: kept history, then this round's rows
        starts = np.concatenate([[0], np.cumsum(new)])
        seqs = []
        for b in range(users):
            mine = slice(starts[b], starts[b + 1])
            seqs.append((torch.cat([kept[b][0], k2[mine]]), torch.cat([kept[b][1], v[mine]])))
            gk, gv = pool.rows(b, 0, int(length[b] + new[b]))
            assert torch.equal(gk, seqs[b][0]) and torch.equal(gv, seqs[b][1])
        kf, vf = (torch.cat([s[i] for s in seqs]) for i in (0, 1))
        qf = torch.cat([torch.cat([torch.zeros_like(kept[b][0]), q2[starts[b]:starts[b + 1]]]) for b in range(users)])
        whole = hstu_attn_fwd(qf, kf, vf, offsets_of(length + new), dev_i32(cands), alpha, N, int((length + new).max()))
        row = 0
        for b in range(users):
            mine, L, n = slice(starts[b], starts[b + 1]), int(length[b]), int(new[b])
            if n:
                want, bound = dense64(to_f64(q2[mine]), to_f64(seqs[b][0]), to_f64(seqs[b][1]), L, n, int(cands[b]), alpha, N)
                assert (np.abs(to_f64(out[mine]) - want) <= bound).all()
                assert (np.abs(to_f64(whole[row + L:row + L + n]) - want) <= bound).all()
            row += L + n
            kept[b] = [s[:L + int(events[b])] for s in seqs[b]]
        length = length + events
