"""Attention over a sliding window with sinks, and the page plan of such a
cache: plain float64 / integer definitions.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path imports this module.

A query at position t sees row j when j <= t and (j > t - window or
j < sinks); over the visible rows it is the textbook attention of
``lrkv_oracle.attend`` on the materialised keys and values.  The page plan
walks the requests one by one with an ordinary list of free pages.
"""
from __future__ import annotations

import numpy as np

from .grouped import group_of
from .lrkv_oracle import attend, expand_head


def visible(t, window, sinks):
    """Positions that the query at position t sees, in order."""
    return [j for j in range(t + 1) if j > t - window or j < sinks]


def pool_rows(pool, pages, positions, page_size):
    """Rows of one request at the given positions, read page by page."""
    pool = np.asarray(pool, np.float64)
    if not positions:
        return np.zeros((0,) + pool.shape[2:])
    return np.stack([pool[int(pages[j // page_size]), j % page_size] for j in positions])


def attend_query(q, S_K, S_V, R_K, R_V, B_K, B_V, pages, t, page_size, window, sinks, N_K=None):
    """Output [H, d_h] of one query at position t of a request.

    q: [H, d_h]; S pools [pages, page_size, d_h] or [.., G, d_h]; R pools
    [pages, page_size, H, r]; N_K: stored reciprocal key norms or None.
    """
    seen = visible(t, window, sinks)
    sk, sv, rk, rv = (pool_rows(p, pages, seen, page_size) for p in (S_K, S_V, R_K, R_V))
    if sk.ndim == 2:
        sk, sv = sk[:, None], sv[:, None]
    H, G = q.shape[0], sk.shape[1]
    nk = None if N_K is None else pool_rows(N_K, pages, seen, page_size)
    out = np.empty(q.shape)
    for h in range(H):
        g = group_of(h, H, G)
        K = expand_head(sk[:, g], rk[:, h], B_K[h])
        if nk is not None:
            K = K * nk[:, h][:, None]
        out[h] = attend(q[h], K, expand_head(sv[:, g], rv[:, h], B_V[h]))
    return out


def page_plan(seq_lens, new_rows, page_table, free_pages, page_size, num_pages, window, sinks, max_rows):
    """One step of the page plan, request by request.

    free_pages: list of free ids, the last one handed out first.  Returns a
    dict with the new lengths, cu_rows, positions, seq_ids, slots, the page
    table, the free list and which requests were refused or invalid.
    """
    table = np.array(page_table, copy=True)
    B, max_pages = table.shape
    room = max_pages * page_size
    free = list(free_pages)
    n_free = len(free)
    pages = lambda n: -(-n // page_size)
    sp = pages(min(sinks, room)) if window else 0

    def sight(L):
        """First page a query at a position >= L may still see beyond the sinks' pages."""
        p = 0
        while window and (p + 1) * page_size <= L - window + 1:
            p += 1
        return max(sp, p) if window else 0

    lens, cu, pos, ids, slots, back = [], [0], [], [], [], []
    refused, invalid = [], []
    asked_rows = asked_pages = 0
    for b in range(B):
        L, n = int(seq_lens[b]), int(new_rows[b])
        if L < 0 or L > room or n < -1 or L + max(n, 0) > room:
            invalid.append(b)
            n = 0
            lens.append(L)
        elif n == -1:
            held = pages(L)
            back += [int(table[b, p]) for p in range(held) if p < sp or p >= sight(L)]
            lens.append(0)
        else:
            need = pages(L + n) - pages(L)
            asked_rows += n
            asked_pages += need
            if n and (asked_rows > max_rows or (need and asked_pages > n_free)):
                refused.append(b)
                n = 0
            else:
                for p in range(pages(L), pages(L + n)):
                    table[b, p] = free.pop()
                if n:
                    back += [int(table[b, p]) for p in range(sight(L), sight(L + n))]
            lens.append(L + n)
        for t in range(L, L + max(n, 0)):
            pos.append(t)
            ids.append(b)
            slots.append(int(table[b, t // page_size]) * page_size + t % page_size)
        cu.append(len(pos))
    return dict(seq_lens=lens, cu_rows=cu, positions=pos, seq_ids=ids, slots=slots, page_table=table,
                free=free + back, refused=refused, invalid=invalid)
