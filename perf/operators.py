"""Cases and plain forms of the paged K/V cache operators: the position rotation (and its gradient), appending rows
to a paged cache with the rotation applied on the way, and the target-aware SiLU attention that reads the cache.

``run`` computes an operator with elementary torch operations in 32 bits (angles in 64), or, with ``own`` set, calls
the library.  ``exact`` computes the same results in 64 bits, one user at a time."""
import math
import random

import torch

own = False


# --------------------------------------------------------------------------------------------- cases
def _rotary(name, rows, heads, d, rot_dim, axes, interleaved, inverse, strided):
    return {"name": name, "op": "rotary", "rows": rows, "heads": heads, "d": d, "rot_dim": rot_dim, "axes": axes,
            "interleaved": interleaved, "inverse": inverse, "strided": strided}


def _cache(op, name, users, heads, d, page, history, new, targets, ragged, **more):
    """history, new, targets: rows a user has cached, brings as history and brings as candidates (upper bounds where
    ragged: then histories are lognormal and the other two uniform, zero among them)."""
    return {"name": name, "op": op, "users": users, "heads": heads, "d": d, "page": page, "history": history,
            "new": new, "targets": targets, "ragged": ragged, "lens": 1, **more}


def listed():
    return [
        # Training: Q and K of the DLRMv3-shaped batch (8 users x 4096 rows) on their way to the attention, columns of
        # the layer's [U | V | Q | K] buffer, rotated by position and by event time.
        _rotary("rotary dlrmv3", 8 * 4096, 4, 128, 128, 2, False, False, True),
        # Training: the gradients of the same for the long-history batch, packed, pairs side by side.
        _rotary("rotary grad long", 4 * 8704, 8, 64, 64, 1, True, True, False),
        # The tiny batch's few hundred rows, half of each head rotated: the latency of one launch.
        _rotary("rotary tiny", 211, 2, 32, 16, 1, False, False, False),
        # Serving: every user's one new event.
        _cache("append", "append token", 64, 4, 128, 16, 4096, 1, 0, False, rotate=True, axes=1, strided=True,
               head_major=False),
        # Serving: 300 new events and 2048 candidates for each of 16 users, straight from the projection's columns.
        _cache("append", "append streaming", 16, 4, 128, 64, 3000, 300, 2048, False, rotate=True, axes=2, strided=True,
               head_major=False),
        # Filling a cache from whole ragged histories, head-major pages, no rotation.
        _cache("append", "append ragged", 64, 8, 64, 32, 0, 4096, 16, True, rotate=False, axes=1, strided=False,
               head_major=True),
        # The smallest call: four short users, one new token each.
        _cache("attn", "attn tiny token", 4, 2, 32, 16, 64, 1, 0, False, head_major=False),
        # One new token for each of 64 users of lognormal history: a pass over the cached K and V.
        _cache("attn", "attn token", 64, 4, 128, 16, 4096, 1, 0, True, head_major=False),
        # A few events and candidates for each user.
        _cache("attn", "attn few", 16, 4, 128, 32, 3000, 4, 8, False, head_major=True),
        # 300 new events on a cached history, no candidates.
        _cache("attn", "attn chunk", 16, 4, 128, 64, 3000, 300, 0, False, head_major=False),
        # The streaming batch: 300 new events and 2048 candidates on 3000 cached rows.
        _cache("attn", "attn streaming", 16, 4, 128, 64, 3000, 300, 2048, False, head_major=False),
        # Long histories, 512 candidates a user, small heads.
        _cache("attn", "attn long", 4, 8, 64, 128, 8192, 0, 512, False, head_major=False),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attn", "attn"])
    d = rng.choice([32, 64, 128])
    heads = rng.randint(1, 8)
    if op == "rotary":
        rows = _spread(rng, 1, 8 * 4096 * 512 // (heads * d))
        rot_dim = rng.choice([16 * n for n in range(1, d // 16 + 1)])
        return _rotary("", min(rows, 8 * 4096), heads, d, rot_dim, rng.randint(1, 3), rng.random() < 0.5,
                       rng.random() < 0.5, rng.random() < 0.5)
    users = _spread(rng, 1, 64)
    page = rng.choice([8, 16, 32, 64, 128, 256])
    history = _spread(rng, 1, 8192) if rng.random() < 0.9 else 0
    new = _spread(rng, 1, 2048) if rng.random() < 0.6 else rng.randint(1, 16)
    targets = _spread(rng, 1, 2048) if rng.random() < 0.5 else 0
    # No more rows, and no more (query, key) pairs of the padded batch, than the largest listed case has.
    while users > 1 and (users * (history + new + targets) * heads * d > 16 * 5348 * 512 or
                         users * heads * (new + targets) * (history + new + targets) > 16 * 4 * 2348 * 5348):
        users = max(1, users * 3 // 4)
    case = _cache(op, "", users, heads, d, page, history, new, targets, rng.random() < 0.6,
                  head_major=rng.random() < 0.3)
    case["lens"] = rng.randint(1, 1 << 30)
    if op == "append":
        case.update(rotate=rng.random() < 0.7, axes=rng.randint(1, 2), strided=rng.random() < 0.5)
    return case


def _lengths(case):
    """Cached rows, new rows (candidates among them) and candidates of every user."""
    rng = random.Random(case["lens"])
    users, history, new, targets = (case[k] for k in ("users", "history", "new", "targets"))
    if not case["ragged"]:
        return [history] * users, [new + targets] * users, [targets] * users
    cached, fresh, cands = [], [], []
    for _ in range(users):
        cached.append(min(history, int(history / 4 * rng.lognormvariate(0.0, 1.0))))
        n = new if new <= 1 else rng.randint(0, new)
        t = rng.randint(0, targets)
        fresh.append(n + t)
        cands.append(t)
    if not any(fresh):
        fresh[0] = 1
    return cached, fresh, cands


def _sections(pairs, axes):
    """How many of the pairs each axis turns: equal runs, the first one taking the rest."""
    return [pairs - (axes - 1) * (pairs // axes)] + [pairs // axes] * (axes - 1)


# --------------------------------------------------------------------------------------------- inputs
def _freqs(sections, device):
    """Radians a step: 10000^(-i/n) for the position axis, periods of a minute to ten years for the others (seconds)."""
    out = []
    for a, n in enumerate(sections):
        i = torch.arange(n, dtype=torch.float64) / max(1, n)
        out.append(10000.0 ** -i if a == 0 else 2 * math.pi / (60.0 * (10 * 365.25 * 1440.0) ** i))
    return torch.cat(out).to(device)


def _positions(starts, counts, axes, gen, device):
    """int32 [axes, rows]: the row's place in its history, then unix times that grow along it."""
    counts_t = torch.tensor(counts, device=device)
    rows = int(counts_t.sum())
    first = torch.cumsum(counts_t, 0) - counts_t
    place = torch.arange(rows, device=device) - torch.repeat_interleave(first - torch.tensor(starts, device=device), counts_t)
    times = [1_700_000_000 + torch.cumsum(torch.randint(0, 3000, (rows,), generator=gen, device=device), 0)
             for _ in range(axes - 1)]
    return torch.stack([place] + times).to(torch.int32)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32).to(torch.bfloat16)


def _tokens(gen, count, rows, heads, d, strided):
    """`count` tensors [rows, heads, d]: columns of one wide projection, or packed."""
    if strided:
        wide = _normal(gen, rows, 4, heads, d)
        return [wide[:, 3 - i] for i in range(count)]
    return [_normal(gen, rows, heads, d) for _ in range(count)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 1009 + 17)
    heads, d = case["heads"], case["d"]
    if case["op"] == "rotary":
        q, k = _tokens(gen, 2, case["rows"], heads, d, case["strided"])
        sections = _sections(case["rot_dim"] // 2, case["axes"])
        return {"case": case, "q": q, "k": k, "sections": sections, "freqs": _freqs(sections, dev),
                "positions": _positions([0], [case["rows"]], case["axes"], gen, dev)}
    page = case["page"]
    cached, fresh, cands = _lengths(case)
    total = [c + n for c, n in zip(cached, fresh)]
    pages = [(t + page - 1) // page for t in total]
    used, width = sum(pages), max(1, max(pages))
    pool = used + used // 4 + 1
    # Pages in any order; table entries past a user's last page name no page.
    order = torch.randperm(pool, generator=gen, device=dev)[:used].to(torch.int32)
    slot = torch.arange(width, device=dev)[None, :] < torch.tensor(pages, device=dev)[:, None]
    table = torch.full((case["users"], width), -1, dtype=torch.int32, device=dev)
    table[slot] = order
    offsets = torch.tensor([0] + fresh, device=dev).cumsum(0).to(torch.int32)
    st = {"case": case, "table": table, "q_offsets": offsets, "kv_len": torch.tensor(total, dtype=torch.int32, device=dev),
          "num_targets": torch.tensor(cands, dtype=torch.int32, device=dev), "max_new": max(fresh), "max_kv": max(total),
          "total_new": sum(fresh), "cached": torch.tensor(cached, device=dev), "alpha": 1.0 / math.sqrt(d), "N": float(max(total))}
    shape = (pool, heads, page, d) if case["head_major"] else (pool, page, heads, d)
    caches = [_normal(gen, *shape) for _ in range(2)]
    if case["head_major"]:
        caches = [c.transpose(1, 2) for c in caches]
    st["k_cache"], st["v_cache"] = caches
    if case["op"] == "append":
        st["q"], st["k"], st["v"] = _tokens(gen, 3, sum(fresh), heads, d, case["strided"])
        sections = _sections(d // 2, case["axes"])
        st["sections"], st["freqs"] = sections, _freqs(sections, dev)
        # With one axis the place in the cache is the position; a second axis brings its own numbers.
        st["positions"] = _positions(cached, fresh, case["axes"], gen, dev) if case["axes"] > 1 else None
        return st
    st["q"] = _normal(gen, sum(fresh), heads, d)
    # What lies behind a user's last row was never written.
    last = torch.tensor(total, device=dev) - 1
    tail = torch.arange(page, device=dev)[None, :] > (last % page)[:, None]
    where = table.gather(1, (last.clamp(min=0) // page)[:, None])[:, 0].long()
    for c in caches:
        rows, cols = torch.nonzero(tail & (last >= 0)[:, None], as_tuple=True)
        c[where[rows], cols] = float("nan")
    return st


# --------------------------------------------------------------------------------------------- plain forms
def _turn(x, positions, freqs, sections, interleaved, inverse):
    """x with its pairs turned: positions [axes, rows], x [rows, heads, d]."""
    pairs = freqs.numel()
    axis = torch.cat([torch.full((n,), a, device=x.device) for a, n in enumerate(sections)])
    angle = (positions.double()[axis] * freqs[:, None]).t()
    cos = torch.cos(angle).float()[:, None, :]
    sin = torch.sin(angle).float()[:, None, :] * (-1.0 if inverse else 1.0)
    y = x.float().clone()
    a, b = (y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2]) if interleaved else (y[..., :pairs], y[..., pairs:2 * pairs])
    turned = a * cos - b * sin, a * sin + b * cos
    a.copy_(turned[0])
    b.copy_(turned[1])
    return y.to(torch.bfloat16)


def _row_users(st):
    """User of every new row and the row's place in the user's cache."""
    counts = st["q_offsets"].diff().long()
    user = torch.repeat_interleave(torch.arange(counts.numel(), device=counts.device), counts, output_size=st["total_new"])
    place = torch.arange(st["total_new"], device=counts.device) - st["q_offsets"][user] + st["kv_len"][user] - counts[user]
    return user, place


def _plain_append(st):
    case, page = st["case"], st["case"]["page"]
    user, place = _row_users(st)
    q, k = st["q"], st["k"]
    if case["rotate"]:
        positions = place[None] if st["positions"] is None else st["positions"]
        q = _turn(q, positions, st["freqs"], st["sections"], False, False)
        k = _turn(k, positions, st["freqs"], st["sections"], False, False)
    at = st["table"][user, place // page].long(), place % page
    st["k_cache"][at] = k
    st["v_cache"][at] = st["v"]
    return (q if case["rotate"] else None), st["k_cache"], st["v_cache"]


def _plain_attn(st):
    page, n_max, l_max = st["case"]["page"], st["max_new"], st["max_kv"]
    dev = st["q"].device
    counts = st["q_offsets"].diff().long()
    length = st["kv_len"].long()
    hist = length - st["num_targets"]
    key = torch.arange(l_max, device=dev)
    held = key[None, :] < length[:, None]
    at = st["table"][:, (key // page).clamp(max=st["table"].shape[1] - 1)].long().clamp(min=0), (key % page)[None, :]
    k = torch.where(held[..., None, None], st["k_cache"][at], 0).float().permute(0, 2, 3, 1)
    v = torch.where(held[..., None, None], st["v_cache"][at], 0).float().permute(0, 2, 1, 3)
    row = torch.arange(n_max, device=dev)
    q = st["q"][(st["q_offsets"][:-1, None] + row[None, :]).clamp(max=st["total_new"] - 1).long()].float()
    x = torch.matmul(q.permute(0, 2, 1, 3), k) * st["alpha"]
    place = (length - counts)[:, None] + row[None, :]
    sees = torch.minimum(place + 1, hist[:, None])
    seen = (key[None, None, :] < sees[..., None]) | (key[None, None, :] == place[..., None])
    p = torch.where(seen[:, None], x / (1.0 + torch.exp(-x)), 0.0)
    out = torch.matmul(p, v) / st["N"]
    user, at = _row_users(st)
    return out.permute(0, 2, 1, 3)[user, at - (length - counts)[user]].to(torch.bfloat16)


def run(st):
    case = st["case"]
    if own:
        import hstu_pointwise_attention_jagged_b200 as hstu
        if case["op"] == "rotary":
            return hstu.hstu_rotary(st["q"], st["k"], st["positions"], st["freqs"], sections=st["sections"],
                                    interleaved=case["interleaved"], inverse=case["inverse"])
        if case["op"] == "append":
            turn = {"q": st["q"], "freqs": st["freqs"], "sections": st["sections"], "positions": st["positions"]}
            q = hstu.hstu_paged_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["q_offsets"],
                                       st["kv_len"], **(turn if case["rotate"] else {}))
            return q, st["k_cache"], st["v_cache"]
        return hstu.hstu_paged_attn_fwd(st["q"], st["k_cache"], st["v_cache"], st["table"], st["q_offsets"],
                                        st["kv_len"], st["num_targets"], st["alpha"], st["N"], st["max_new"], st["max_kv"])
    if case["op"] == "rotary":
        return tuple(_turn(x, st["positions"], st["freqs"], st["sections"], case["interleaved"], case["inverse"])
                     for x in (st["q"], st["k"]))
    return _plain_append(st) if case["op"] == "append" else _plain_attn(st)


# --------------------------------------------------------------------------------------------- work
def work(case):
    row = case["heads"] * case["d"] * 2  # bytes of one bf16 row of all heads
    if case["op"] == "rotary":
        return {"bytes": 4 * case["rows"] * row + 4 * case["rows"] * case["axes"],
                "flops": 3 * 2 * case["rows"] * case["heads"] * case["rot_dim"]}
    cached, fresh, cands = _lengths(case)
    new = sum(fresh)
    if case["op"] == "append":
        tensors = 6 if case["rotate"] else 4
        return {"bytes": tensors * new * row + 8 * case["users"] + (4 * new * case["axes"] if case["axes"] > 1 else 0),
                "flops": 3 * 2 * new * row // 2 if case["rotate"] else 0}
    pairs = 0
    for c, n, t in zip(cached, fresh, cands):
        u = c + n - t
        pairs += (u * (u + 1) - c * (c + 1)) // 2 + t * (u + 1)
    held = sum(c + n for c, n in zip(cached, fresh) if n)
    return {"bytes": 2 * new * row + 2 * held * row + 4 * held // case["page"], "flops": 4 * case["d"] * case["heads"] * pairs}


# --------------------------------------------------------------------------------------------- 64 bits
def _exact_turn(x, positions, freqs, sections, interleaved, sign):
    x = x.double()
    y = x.clone()
    pairs = freqs.numel()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for i in range(pairs):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        t = (positions[axis[i]].double() * freqs[i] * sign)[:, None]
        y[..., lo] = x[..., lo] * t.cos() - x[..., hi] * t.sin()
        y[..., hi] = x[..., lo] * t.sin() + x[..., hi] * t.cos()
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return tuple(_exact_turn(x, st["positions"], st["freqs"], st["sections"], case["interleaved"],
                                 -1.0 if case["inverse"] else 1.0) for x in (st["q"], st["k"]))
    cached, fresh, cands = _lengths(case)
    page, begin = case["page"], 0
    if case["op"] == "append":
        k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
        outs = []
        for b, (c, n) in enumerate(zip(cached, fresh)):
            place = torch.arange(c, c + n, device=k_cache.device)
            mine = slice(begin, begin + n)
            begin += n
            q, k = st["q"][mine].double(), st["k"][mine].double()
            if case["rotate"]:
                pos = place[None] if st["positions"] is None else st["positions"][:, mine]
                q, k = (_exact_turn(x, pos, st["freqs"], st["sections"], False, 1.0) for x in (q, k))
            outs.append(q)
            pages = st["table"][b].long()[place // page]
            k_cache[pages, place % page] = k
            v_cache[pages, place % page] = st["v"][mine].double()
        return (torch.cat(outs) if case["rotate"] else None), k_cache, v_cache
    outs = []
    for b, (c, n, t) in enumerate(zip(cached, fresh, cands)):
        j = torch.arange(c + n, device=st["q"].device)
        pages = st["table"][b].long()[j // page]
        k, v = (x[pages, j % page].double().transpose(0, 1) for x in (st["k_cache"], st["v_cache"]))
        q = st["q"][begin:begin + n].double().transpose(0, 1)
        begin += n
        i = torch.arange(c, c + n, device=q.device)[:, None]
        u = c + n - t
        visible = ((j[None] <= i) & (j[None] < u)) | (j[None] == i)
        x = (q @ k.transpose(1, 2)) * st["alpha"]
        w = torch.sigmoid(x).mul_(x).mul_(visible)
        outs.append(((w @ v) / st["N"]).transpose(0, 1))
    return torch.cat(outs)
