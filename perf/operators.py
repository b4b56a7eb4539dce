"""Measured cases of the bounded-history operators: attention over a sliding
window and a few first tokens that stay visible (sinks), read from the
factored paged cache, for single tokens and for prompt chunks, and the page
tables and slot maps that keep such a cache.

``run`` computes a case with elementary torch operations, or, where ``own``
is true, with the library's operators.
"""
import math

import torch

own = False

D_H = 128          # head width of every tensor-core configuration
FP8_SCALE = 2.0 ** -5


def listed():
    return [
        # one conversation on one stream, the smallest call: latency
        {"name": "decode_one", "op": "decode", "dtype": "bf16", "B": 1, "H": 16, "r": 48, "d_h": D_H, "page": 64,
         "len_lo": 1500, "len_hi": 1500, "window": 512, "sinks": 4},
        # a few requests whose first tokens are younger than the window: odd lengths, some of one token
        {"name": "decode_young", "op": "decode", "dtype": "bf16", "B": 7, "H": 16, "r": 48, "d_h": D_H, "page": 64,
         "len_lo": 1, "len_hi": 901, "window": 640, "sinks": 5},
        # an fp32 cache of a small layer
        {"name": "decode_f32", "op": "decode", "dtype": "f32", "B": 6, "H": 8, "r": 16, "d_h": 64, "page": 32,
         "len_lo": 100, "len_hi": 1900, "window": 500, "sinks": 3},
        # the ordinary serving batch: long histories, a window of 1024
        {"name": "decode_batch", "op": "decode", "dtype": "bf16", "B": 16, "H": 16, "r": 48, "d_h": D_H, "page": 64,
         "len_lo": 4096, "len_hi": 4096, "window": 1024, "sinks": 4},
        # the ragged batch: lengths shorter and longer than the window
        {"name": "decode_ragged", "op": "decode", "dtype": "bf16", "B": 64, "H": 16, "r": 56, "d_h": D_H, "page": 64,
         "len_lo": 256, "len_hi": 8192, "window": 4000, "sinks": 16},
        # an 8-bit cache
        {"name": "decode_fp8", "op": "decode", "dtype": "fp8", "B": 32, "H": 16, "r": 48, "d_h": D_H, "page": 64,
         "len_lo": 3000, "len_hi": 5001, "window": 2048, "sinks": 64},
        # few requests, a long window over a long history
        {"name": "decode_long", "op": "decode", "dtype": "bf16", "B": 4, "H": 32, "r": 32, "d_h": D_H, "page": 64,
         "len_lo": 32768, "len_hi": 32768, "window": 8192, "sinks": 128},
        # one chunk of a long prompt, its history in the cache
        {"name": "prefill_chunk", "op": "prefill", "dtype": "bf16", "B": 1, "H": 16, "r": 48, "d_h": D_H, "page": 64,
         "d": 2048, "rows_lo": 512, "rows_hi": 512, "start_lo": 3001, "start_hi": 3001, "window": 1024, "sinks": 4},
        # prompts of different lengths, some with a history
        {"name": "prefill_ragged", "op": "prefill", "dtype": "bf16", "B": 6, "H": 16, "r": 48, "d_h": D_H, "page": 64,
         "d": 1024, "rows_lo": 33, "rows_hi": 1501, "start_lo": 0, "start_hi": 1900, "window": 700, "sinks": 16},
        # whole prompts
        {"name": "prefill_batch", "op": "prefill", "dtype": "bf16", "B": 8, "H": 16, "r": 48, "d_h": D_H, "page": 64,
         "d": 2048, "rows_lo": 2048, "rows_hi": 2048, "start_lo": 0, "start_hi": 0, "window": 1024, "sinks": 4},
        # the page plan of a decode step: one new token for each request, a few requests end
        {"name": "plan_step", "op": "plan", "B": 64, "page": 64, "max_pages": 512, "len_lo": 100, "len_hi": 30000,
         "new_lo": 1, "new_hi": 1, "retire": 3, "window": 4096, "sinks": 4},
        # the page plan of a large mixed step: chunks of prompts among single tokens
        {"name": "plan_mixed", "op": "plan", "B": 1500, "page": 64, "max_pages": 256, "len_lo": 0, "len_hi": 9000,
         "new_lo": 1, "new_hi": 999, "retire": 40, "window": 2000, "sinks": 70},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "prefill", "prefill", "plan"])
    if op == "decode":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp8", "f32"])
        window, sinks = _log(rng, 60, 8192), rng.choice([0, 1, 4, 16, 31, 128])
        if dtype == "f32":
            H, r, d_h = rng.choice([(4, 4, 16), (8, 16, 64), (6, 8, 32)])
            window = min(window, 1000)
        else:
            (H, r), d_h = rng.choice([(16, 48), (16, 56), (32, 32), (16, 32), (16, 64)]), D_H
        B = max(1, min(_log(rng, 1, 96), 150000 // window, 24 if dtype == "f32" else 96))
        lo = _log(rng, 1, 9000)
        return {"op": op, "dtype": dtype, "B": B, "H": H, "r": r, "d_h": d_h, "page": rng.choice([32, 64, 128]),
                "len_lo": lo, "len_hi": lo + rng.randrange(0, 6000), "window": window, "sinks": sinks}
    if op == "prefill":
        B, hi = rng.randrange(1, 6), _log(rng, 20, 1500)
        lo = rng.randrange(1, hi + 1)
        start = rng.choice([0, rng.randrange(1, 1500)])
        return {"op": op, "dtype": "bf16", "B": B, "H": 16, "r": rng.choice([32, 48, 56]), "d_h": D_H, "page": 64,
                "d": rng.choice([512, 1024, 2048]), "rows_lo": lo, "rows_hi": hi, "start_lo": start,
                "start_hi": start + rng.randrange(0, 300), "window": _log(rng, 40, 1500),
                "sinks": rng.choice([0, 1, 4, 16, 130])}
    B, lo = _log(rng, 1, 1500), rng.randrange(0, 3000)
    window = rng.choice([0, _log(rng, 100, 6000)])
    return {"op": "plan", "B": B, "page": rng.choice([16, 32, 64]), "max_pages": 600, "len_lo": lo,
            "len_hi": lo + rng.randrange(1, 5500), "new_lo": rng.choice([0, 1]), "new_hi": _log(rng, 1, 999),
            "retire": rng.randrange(0, 1 + B // 8), "window": window, "sinks": rng.choice([0, 4, 100])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _spread(lo, hi, B):
    """B whole numbers spread evenly over [lo, hi]."""
    return [lo + (hi - lo) * (2 * b + 1) // (2 * B) for b in range(B)]


def _pages(n, page):
    return (n + page - 1) // page


def _dead(length, c):
    """Leading pages that no query at a position >= length sees (the pages of the sinks apart)."""
    return max(0, (length - c["window"] + 1) // c["page"]) if c["window"] else 0


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, std, dtype, g):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def _pool_fill(shape, c, g):
    if c["dtype"] == "fp8":
        x = torch.randn(shape, device="cuda", generator=g) / FP8_SCALE
        return x.clamp(-448, 448).to(torch.float8_e4m3fn)
    return _normal(shape, 1.0, torch.float32 if c["dtype"] == "f32" else torch.bfloat16, g)


def _live(c, first, last):
    """Page indexes of a request that holds rows for queries at positions first .. last - 1."""
    kept = min(_pages(c["sinks"], c["page"]), _pages(last, c["page"]))
    lo = max(kept, _dead(first, c))
    return list(range(kept)) + list(range(lo, _pages(last, c["page"])))


def _most(c, history, rows):
    """A number of pages that the live rows of requests with at most `history` rows and then rows[b] new ones fit in."""
    if c["window"]:
        history = min(history, c["window"])
    return sum(_pages(c["sinks"], c["page"]) + _pages(history + n, c["page"]) + 2 for n in rows)


def _table(c, firsts, lasts, max_pages, pool, g):
    """Page table whose live entries are pages of a shuffled pool and whose others are -1."""
    index = [(b, p) for b, (f, e) in enumerate(zip(firsts, lasts)) for p in _live(c, f, e)]
    table = torch.full((len(firsts), max_pages), -1, dtype=torch.int32)
    at = torch.tensor(index, dtype=torch.int64).view(-1, 2)
    ids = torch.randperm(pool, generator=g, device="cuda")[:len(index)].cpu().to(torch.int32)
    table[at[:, 0], at[:, 1]] = ids
    return table.cuda()


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    order = torch.randperm(c["B"], device="cuda", generator=g).tolist()
    if c["op"] == "plan":
        return _prepare_plan(c, g, order)
    H, r, d_h, page = c["H"], c["r"], c["d_h"], c["page"]
    act = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = {"c": c, "B_K": _normal((H, d_h, r), r ** -0.5, act, g), "B_V": _normal((H, d_h, r), r ** -0.5, act, g),
         "scale": (FP8_SCALE,) * 4 if c["dtype"] == "fp8" else (1.0,) * 4}
    if c["op"] == "decode":
        spread = _spread(c["len_lo"], c["len_hi"], c["B"])
        lens = [spread[i] for i in order]
        pool = _most(c, c["len_hi"], [1] * c["B"])
        s["page_table"] = _table(c, [n - 1 for n in lens], lens, _pages(max(lens), page), pool, g)
        s["seq_lens"], s["max_len"] = _i32(lens), max(lens)
        s["q"] = _normal((c["B"], H, d_h), 1.0, act, g)
    else:
        starts, rows = _spread(c["start_lo"], c["start_hi"], c["B"]), _spread(c["rows_lo"], c["rows_hi"], c["B"])
        starts, rows = starts[::-1], [rows[i] for i in order]
        ends = [a + n for a, n in zip(starts, rows)]
        pool = _most(c, c["start_hi"], rows)
        s["page_table"] = _table(c, starts, ends, _pages(max(ends), page), pool, g)
        s["start_pos"], s["max_len"] = _i32(starts), max(ends)
        s["cu_rows"] = _i32([sum(rows[:b]) for b in range(c["B"] + 1)])
        n, d = sum(rows), c["d"]
        # activations and weights of unit and 1/d variance: cache rows like a layer's, of unit variance
        s["X"], s["Q"] = _normal((n, d), 1.0, act, g), _normal((n, H, d_h), 1.0, act, g)
        s["W_S_K"], s["W_S_V"] = _normal((d_h, d), d ** -0.5, act, g), _normal((d_h, d), d ** -0.5, act, g)
        s["U_K"], s["U_V"] = _normal((H, r, d), d ** -0.5, act, g), _normal((H, r, d), d ** -0.5, act, g)
    s["S_K"], s["S_V"] = _pool_fill((pool, page, d_h), c, g), _pool_fill((pool, page, d_h), c, g)
    s["R_K"], s["R_V"] = _pool_fill((pool, page, H, r), c, g), _pool_fill((pool, page, H, r), c, g)
    return s


def _prepare_plan(c, g, order):
    B, page = c["B"], c["page"]
    spread, news = _spread(c["len_lo"], c["len_hi"], B), _spread(c["new_lo"], c["new_hi"], B)
    lens, new = [spread[i] for i in order], news[:]
    for b in range(c["retire"]):
        new[b * B // max(1, c["retire"])] = -1
    used = _most(c, c["len_hi"], [0] * B)
    table = _table(c, lens, lens, c["max_pages"], used, g)
    rows = sum(max(0, n) for n in new)
    free = torch.randperm(sum(_pages(max(0, n), page) + 1 for n in new), device="cuda", generator=g).to(torch.int32) + used
    pool = used + free.numel()
    return {"c": c, "seq_lens": _i32(lens), "new_rows": _i32(new), "page_table": table,
            "free_pages": torch.cat([free, torch.full((used,), -1, dtype=torch.int32, device="cuda")]),
            "n_free": _i32([free.numel()]), "free_out": torch.full((pool,), -1, dtype=torch.int32, device="cuda"),
            "max_rows": rows + 5}


# ---------------------------------------------------------------------------
# What a pass needs
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "plan":
        lens, news = _spread(c["len_lo"], c["len_hi"], c["B"]), _spread(c["new_lo"], c["new_hi"], c["B"])
        need = sum(_pages(n + k, c["page"]) - _pages(n, c["page"]) for n, k in zip(lens, news))
        # lengths and counts in, lengths and row offsets out; position, request and slot of each row; new table
        # entries and the ids they come from
        return {"bytes": 16 * c["B"] + 12 * sum(news) + 8 * need, "flops": 0}
    H, r, d_h = c["H"], c["r"], c["d_h"]
    eb = {"f32": 4, "bf16": 2, "fp8": 1}[c["dtype"]]
    ab = 4 if c["dtype"] == "f32" else 2
    row = 2 * (d_h + H * r) * eb
    seen = lambda n: n if c["window"] + c["sinks"] >= n else c["window"] + c["sinks"]  # noqa: E731
    bases = 2 * H * d_h * r * ab
    pair = 4 * H * (d_h + r)
    if c["op"] == "decode":
        rows = sum(seen(n) for n in _spread(c["len_lo"], c["len_hi"], c["B"]))
        return {"bytes": rows * row + bases + 2 * c["B"] * H * d_h * ab, "flops": rows * pair + 4 * c["B"] * H * d_h * r}
    starts, rows = _spread(c["start_lo"], c["start_hi"], c["B"])[::-1], _spread(c["rows_lo"], c["rows_hi"], c["B"])
    n, pairs, old, width = sum(rows), 0, 0, 2 * (d_h + H * r)
    for a, k in zip(starts, rows):
        full = max(0, min(k, c["window"] + c["sinks"] - a))  # rows that still see everything
        pairs += full * a + full * (full + 1) // 2 + (k - full) * (c["window"] + c["sinks"])
        old += min(a, c["window"] + c["sinks"])
    return {"bytes": n * (c["d"] * 2 + width * 2 + 2 * H * d_h * 2) + c["d"] * width * 2 + bases + old * row,
            "flops": 2 * n * c["d"] * width + pairs * pair + 4 * n * H * d_h * r}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    c = state["c"]
    if own:
        return _own(state)
    if c["op"] == "decode":
        return _plain_decode(state)
    if c["op"] == "prefill":
        return _plain_prefill(state)
    return _plain_plan(state)


def _own(s):
    from rank_kv_attention_gb300 import api
    c = s["c"]
    if c["op"] == "plan":
        p = api.page_plan(s["seq_lens"], s["new_rows"], s["page_table"], s["free_pages"], s["n_free"], c["page"],
                          s["max_rows"], free_out=s["free_out"], window=c["window"], sinks=c["sinks"])
        return [p.seq_lens, p.cu_rows, p.positions, p.seq_ids, p.slots, s["page_table"], s["free_out"], p.n_free]
    cache = api.PagedCache(s["S_K"], s["S_V"], s["R_K"], s["R_V"], s["scale"])
    if c["op"] == "decode":
        return api.decode_window(s["q"], cache, s["B_K"], s["B_V"], s["seq_lens"], s["page_table"], s["max_len"],
                                 c["window"], c["sinks"])
    out = api.prefill_window(s["X"], s["Q"], s["cu_rows"], s["start_pos"], s["max_len"], s["W_S_K"], s["W_S_V"],
                             s["U_K"], s["U_V"], s["B_K"], s["B_V"], cache, s["page_table"], c["window"], c["sinks"])
    return [out, s["S_K"], s["S_V"], s["R_K"], s["R_V"]]


def _rows_of(pool, rows, scale):
    """Rows of a pool as fp32 values (8-bit codes times their scale)."""
    flat = pool.view(-1, *pool.shape[2:])
    if pool.dtype == torch.float8_e4m3fn:
        return flat.view(torch.uint8)[rows].view(torch.float8_e4m3fn).float() * scale
    return flat[rows].float()


def _plain_decode(s):
    c, page = s["c"], s["c"]["page"]
    n = s["seq_lens"].long()[:, None]
    first = (n - c["window"]).clamp(min=0)
    kept = torch.minimum(first, torch.full_like(first, c["sinks"]))   # sink rows before the window
    k = torch.arange(min(s["max_len"], c["window"] + c["sinks"]), device=n.device)[None]
    j = torch.where(k < kept, k, first + k - kept)                     # the k-th visible row
    seen = j < n
    j = torch.where(seen, j, n - 1)
    rows = s["page_table"].long().gather(1, j // page) * page + j % page
    q, B_K, B_V, sc = s["q"].float(), s["B_K"].float(), s["B_V"].float(), s["scale"]
    score = torch.einsum("bhd,bkd->bhk", q, _rows_of(s["S_K"], rows, sc[0]))
    score += torch.einsum("bhr,bkhr->bhk", torch.einsum("bhd,hdr->bhr", q, B_K), _rows_of(s["R_K"], rows, sc[2]))
    score = (score * c["d_h"] ** -0.5).masked_fill(~seen[:, None], -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    o = torch.einsum("bhk,bkd->bhd", w, _rows_of(s["S_V"], rows, sc[1]))
    private = torch.einsum("bhk,bkhr->bhr", w, _rows_of(s["R_V"], rows, sc[3]))
    return (o + torch.einsum("bhr,hdr->bhd", private, B_V)).to(s["q"].dtype)


def _plain_prefill(s):
    c, page = s["c"], s["c"]["page"]
    cu, start, X = s["cu_rows"].long(), s["start_pos"].long(), s["X"]
    n, dev = X.shape[0], X.device
    i = torch.arange(n, device=dev)
    b = torch.searchsorted(cu[1:], i, right=True)
    pos = start[b] + i - cu[b]
    table = s["page_table"].long()
    rows = table[b, pos // page] * page + pos % page
    x = X.float()
    put = lambda pool, w: pool.view(-1, w.reshape(-1, w.shape[-1]).shape[0]).index_copy_(  # noqa: E731
        0, rows, (x @ w.float().reshape(-1, w.shape[-1]).T).to(pool.dtype))
    put(s["S_K"], s["W_S_K"]), put(s["S_V"], s["W_S_V"]), put(s["R_K"], s["U_K"]), put(s["R_V"], s["U_V"])
    # each request's rows and keys, padded to the longest
    at = torch.arange(s["max_len"], device=dev)
    live = table[:, at // page] * page + at % page
    live = torch.where(live < 0, 0, live)                              # pages without an id are out of every window
    lens = cu[1:] - cu[:-1]
    t = torch.arange(c["rows_hi"], device=dev)
    there = t[None] < lens[:, None]
    src = torch.where(there, cu[:-1, None] + t[None], 0)
    qpos = start[:, None] + t[None]
    gap = qpos[:, :, None] - at[None, None]
    seen = (gap >= 0) & ((gap < c["window"]) | (at[None, None] < c["sinks"]))
    q = s["Q"][src].float()
    score = torch.einsum("bthd,bkd->bhtk", q, _rows_of(s["S_K"], live, 1.0))
    p = torch.einsum("bthd,hdr->bthr", q, s["B_K"].float())
    score += torch.einsum("bthr,bkhr->bhtk", p, _rows_of(s["R_K"], live, 1.0))
    score.mul_(c["d_h"] ** -0.5).masked_fill_(~seen[:, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    score.div_(score.sum(-1, keepdim=True))
    o = torch.einsum("bhtk,bkd->bthd", score, _rows_of(s["S_V"], live, 1.0))
    private = torch.einsum("bhtk,bkhr->bthr", score, _rows_of(s["R_V"], live, 1.0))
    o += torch.einsum("bthr,hdr->bthd", private, s["B_V"].float())
    return [o[there].to(s["Q"].dtype), s["S_K"], s["S_V"], s["R_K"], s["R_V"]]


def _plain_plan(s):
    c, page, dev = s["c"], s["c"]["page"], s["seq_lens"].device
    L, new, table = s["seq_lens"].long(), s["new_rows"].long(), s["page_table"]
    B, room = L.numel(), table.shape[1] * page
    pages = lambda x: (x + page - 1) // page  # noqa: E731
    ok = (L >= 0) & (L <= room) & (new >= -1) & (L + new.clamp(min=0) <= room)
    ends, want = ok & (new == -1), torch.where(ok, new.clamp(min=0), 0)
    need = pages(L + want) - pages(L)
    grant = (want.cumsum(0) <= s["max_rows"]) & ((need == 0) | (need.cumsum(0) <= s["n_free"]))
    rows, need = torch.where(grant, want, 0), torch.where(grant, need, 0)
    grown = torch.where(ends, 0, L + rows)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), rows.cumsum(0)])
    # new table entries, from the end of the free list
    k = torch.arange(int(s["max_rows"]), device=dev)
    off = need.cumsum(0)
    kb = torch.searchsorted(off, k, right=True).clamp(max=B - 1)
    new_page = k < off[-1]
    kb, k = kb[new_page], k[new_page]
    n_free = s["n_free"].long()
    table[kb, pages(L)[kb] + k - (off - need)[kb]] = s["free_pages"][n_free - 1 - k]
    # pages that no later query sees, and those of requests that end
    sp = pages(torch.tensor(c["sinks"], device=dev)) if c["window"] else torch.zeros((), dtype=torch.int64, device=dev)
    dead = lambda n: torch.maximum(  # noqa: E731
        sp, ((n - c["window"] + 1) // page).clamp(min=0) if c["window"] else torch.zeros_like(n))
    held = pages(L)
    lo = dead(L)
    hi = torch.where(ends, torch.maximum(held, lo), torch.where(rows > 0, dead(L + rows), lo))
    front = torch.where(ends, torch.minimum(sp, held), 0)              # the sinks' pages of requests that end
    count = front + hi - lo
    out_b = torch.repeat_interleave(torch.arange(B, device=dev), count)
    j = torch.arange(out_b.numel(), device=dev) - (count.cumsum(0) - count)[out_b]
    column = torch.where(j < front[out_b], j, lo[out_b] + j - front[out_b])
    back = table.long()[out_b, column]
    left = n_free - off[-1]
    f = torch.arange(s["free_out"].numel(), device=dev)
    s["free_out"].copy_(torch.where(f < left, s["free_pages"].long(), s["free_out"].long()))
    s["free_out"].index_copy_(0, left + torch.arange(back.numel(), device=dev), back.int())
    # the rows
    i = torch.arange(int(s["max_rows"]), device=dev)
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=B - 1)
    row = i < cu[-1]
    pos = torch.where(row, L[b] + i - cu[b], 0)
    slot = table.long()[b, pos // page] * page + pos % page
    cut = lambda v: torch.where(row, v, -1).int()  # noqa: E731
    return [grown.int(), cu.int(), cut(pos), cut(b), cut(slot), table, s["free_out"], (left + back.numel()).int()]


# ---------------------------------------------------------------------------
# The definition in 64 bits: keys and values written out for each head, then
# one softmax over the rows that the mask leaves
# ---------------------------------------------------------------------------
def _expanded(pool_s, pool_r, basis, ids, scale_s, scale_r):
    """S + R B^T of the cache rows `ids`, by head: [H, rows, d_h]."""
    pick = lambda pool: _picked(pool.reshape(-1, *pool.shape[2:]), ids)  # noqa: E731
    wide = torch.matmul(pick(pool_r).transpose(0, 1) * scale_r, basis.double().transpose(1, 2))
    return pick(pool_s)[None] * scale_s + wide


def _picked(rows, ids):
    if rows.dtype == torch.float8_e4m3fn:
        return rows.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
    return rows[ids].double()


def _attend(q, keys, values, seen):
    """q [t, H, d], keys and values [H, k, d], seen [t, k]."""
    logits = torch.matmul(q.double().transpose(0, 1), keys.transpose(1, 2)) / math.sqrt(q.shape[-1])
    logits[:, ~seen] = -math.inf
    return torch.matmul(torch.softmax(logits, dim=-1), values).transpose(0, 1)


def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None
    s = prepare(c, seed)
    page, table, sc = c["page"], s["page_table"].tolist(), s["scale"]
    if c["op"] == "decode":
        out = []
        for b, n in enumerate(s["seq_lens"].tolist()):
            vis = [j for j in range(n) if j >= n - c["window"] or j < c["sinks"]]
            ids = torch.tensor([table[b][j // page] * page + j % page for j in vis], device="cuda")
            keys = _expanded(s["S_K"], s["R_K"], s["B_K"], ids, sc[0], sc[2])
            values = _expanded(s["S_V"], s["R_V"], s["B_V"], ids, sc[1], sc[3])
            out.append(_attend(s["q"][b:b + 1], keys, values, torch.ones(1, len(vis), dtype=torch.bool, device="cuda")))
        return torch.cat(out)
    cu, starts, x = s["cu_rows"].tolist(), s["start_pos"].tolist(), s["X"].double()
    wide = {k: x @ s[w].double().reshape(-1, c["d"]).T
            for k, w in (("S_K", "W_S_K"), ("S_V", "W_S_V"), ("R_K", "U_K"), ("R_V", "U_V"))}
    pools = {k: s[k].double() for k in wide}
    for b, a in enumerate(starts):
        ids = torch.tensor([table[b][j // page] * page + j % page for j in range(a, a + cu[b + 1] - cu[b])], device="cuda")
        for k in wide:
            new = wide[k][cu[b]:cu[b + 1]].reshape(-1, *s[k].shape[2:])
            s[k].view(-1, *s[k].shape[2:])[ids] = new.to(s[k].dtype)   # what the cache holds
            pools[k].view(-1, *s[k].shape[2:])[ids] = new
    out = []
    for b, a in enumerate(starts):
        end = a + cu[b + 1] - cu[b]
        for t0 in range(a, end, 512):
            t = torch.arange(t0, min(end, t0 + 512), device="cuda")
            lo = max(0, t0 - c["window"] + 1)
            js = sorted(set(range(min(c["sinks"], end))) | set(range(lo, int(t[-1]) + 1)))
            j = torch.tensor(js, device="cuda")
            ids = torch.tensor([table[b][k // page] * page + k % page for k in js], device="cuda")
            gap = t[:, None] - j[None]
            seen = (gap >= 0) & ((gap < c["window"]) | (j[None] < c["sinks"]))
            q = s["Q"][cu[b] + t0 - a:cu[b] + int(t[-1]) + 1 - a]
            out.append(_attend(q, _expanded(s["S_K"], s["R_K"], s["B_K"], ids, 1.0, 1.0),
                               _expanded(s["S_V"], s["R_V"], s["B_V"], ids, 1.0, 1.0), seen))
    return [torch.cat(out), pools["S_K"], pools["S_V"], pools["R_K"], pools["R_V"]]
