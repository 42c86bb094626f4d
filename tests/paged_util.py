"""Helpers of the paged-cache and rotation tests: a plain fp64 rotation, random page pools, and the
jagged K/V that a page pool holds."""
import numpy as np
import torch

from gpu_util import dev_i32


def rotate64(x, positions, freqs, sections, interleaved=False, inverse=False):
    """x: [rows, H, d] float64; positions: [axes, rows]; the formula of include/hstu_paged.h, pair by pair."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    n = len(freqs)
    axis = [a for a, k in enumerate(sections) for _ in range(k)]
    for i in range(n):
        # Long double: a 31-bit position times a frequency carries 2^-53 of its size in fp64.
        t = positions[axis[i]].astype(np.longdouble) * np.longdouble(freqs[i])
        c, s = np.cos(t).astype(np.float64)[:, None], np.sin(t).astype(np.float64)[:, None]
        if inverse:
            s = -s
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        y[..., lo] = x[..., lo] * c - x[..., hi] * s
        y[..., hi] = x[..., lo] * s + x[..., hi] * c
    return y


def rotation_bound(x, want, pairs, interleaved):
    """Largest error a correct rotation makes, element by element.  The value is rounded to bf16 once
    (half a step: 2^-8 of it).  Before that, times the pair's |x| + |y|: the angle in turns carries the two
    fp64 roundings of freq / 2 pi, 2^-53 each of at most 2^28.4 turns (positions below 2^31,
    frequencies up to 1), 5.2e-7 radians, and the 2^-32 turns cut off below its upper half, 1.5e-9; rounded to
    fp32 it is off by another 2^-25 turns, 1.9e-7; sincospif by two steps, 1.2e-7; and three fp32
    operations by 2^-24 each, 1.8e-7: 1.02e-6 < 2^-19.5 in all."""
    x = np.abs(np.asarray(x, np.float64))
    s = np.zeros_like(x)
    for i in range(pairs):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        s[..., lo] = s[..., hi] = x[..., lo] + x[..., hi]
    pre = s * 2.0 ** -19.5
    return pre + (np.abs(want) + pre) * 2.0 ** -8 + 1e-38


def bf16_normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


class Pool:
    """A page pool with every user's pages in random places; unused table entries are -1 or garbage.

    layout: "rows" [pages, P, H, d], "heads" [pages, H, P, d], "halves" K and V as the two halves of
    [pages, 2, P, H, d], "padded" rows, heads and pages with gaps between them."""

    def __init__(self, lengths, page, H, d, layout="rows", seed=0, spare=3, fill=float("nan"), extra_width=2):
        rng = np.random.default_rng(seed)
        self.lengths = np.asarray(lengths, np.int64)
        self.page, self.H, self.d = page, H, d
        need = -(-self.lengths // page)
        self.pages = int(need.sum()) + spare
        order = rng.permutation(self.pages)
        width = int(need.max(initial=0)) + extra_width
        table = rng.integers(-5, 1 << 30, size=(len(lengths), width)).astype(np.int32)  # garbage where unused
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += int(n)
        self.table_h = table
        self.table = dev_i32(table).view(table.shape)
        if layout == "rows":
            self.k, self.v = (torch.full((self.pages, page, H, d), fill, dtype=torch.bfloat16, device="cuda")
                              for _ in range(2))
        elif layout == "heads":
            self.k, self.v = (torch.full((self.pages, H, page, d), fill, dtype=torch.bfloat16, device="cuda")
                              .transpose(1, 2) for _ in range(2))
        elif layout == "padded":
            self.k, self.v = (torch.full((self.pages, page + 3, H + 1, d + 8), fill, dtype=torch.bfloat16,
                                         device="cuda")[:, :page, :H, :d] for _ in range(2))
        else:
            both = torch.full((self.pages, 2, page, H, d), fill, dtype=torch.bfloat16, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]

    def where(self, b, lo, hi):
        """(page, row) index tensors of user b's positions [lo, hi)."""
        j = np.arange(lo, hi)
        pages = self.table_h[b, j // self.page].astype(np.int64)
        return torch.from_numpy(pages).cuda(), torch.from_numpy(j % self.page).cuda()

    def put(self, b, lo, k, v):
        at = self.where(b, lo, lo + k.shape[0])
        self.k[at] = k
        self.v[at] = v

    def rows(self, b, lo, hi):
        at = self.where(b, lo, hi)
        return self.k[at], self.v[at]


def offsets_of(counts):
    return dev_i32(np.concatenate([[0], np.cumsum(counts)]))


def dense64(q, k, v, c, n, T, alpha, N):
    """One user in fp64: q [n, H, d] at positions c .. c + n, k and v [c + n, H, d], the last T rows
    candidates.  Returns the outputs and a bound on a correct kernel's error, element by element.

    The bound: p = silu(x) is rounded to bf16 for its product with v (half a step, 2^-8 of p); it is
    formed as h + h tanh(h), h = x / 2, with a tanh good to 2^-10.9 (PTX tanh.approx.f32), which moves
    p by at most 2^-10.9 |h|; scores are fp32 sums of d products (d 2^-24 of the sum of their sizes,
    and |silu'| < 1.1), outputs fp32 sums of L terms (L 2^-24 of the sum of their sizes); the output
    is rounded once (2^-8 of it)."""
    L, U = c + n, c + n - T
    i, j = np.arange(c, L)[:, None], np.arange(L)[None, :]
    seen = np.where(i < U, j <= i, (j < U) | (j == i))
    want, bound = np.zeros(q.shape), np.zeros(q.shape)
    d = q.shape[2]
    for h in range(q.shape[1]):
        x = alpha * (q[:, h] @ k[:, h].T)
        size = abs(alpha) * (np.abs(q[:, h]) @ np.abs(k[:, h]).T)
        p = np.where(seen, x / (1.0 + np.exp(-x)), 0.0)
        want[:, h] = p @ v[:, h] / N
        off = np.where(seen, (np.abs(p) * (2.0 ** -8 + L * 2.0 ** -24) + np.abs(x) / 2 * 2.0 ** -10.9
                              + 1.1 * (d + 2) * 2.0 ** -24 * size), 0.0)
        bound[:, h] = off @ np.abs(v[:, h]) / N
    return want, bound + (np.abs(want) + bound) * 2.0 ** -8 + 1e-38
