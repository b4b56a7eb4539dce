"""Block-scaled 8-bit cache: plain float64 / integer definitions.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path imports this module.

A pool holds E4M3 codes and, for each block of ``block`` consecutive tokens of a
page and each head (shared rows: each group), one exponent e, stored as the byte
e + 127; a value is code * 2^e.  A block's exponent is the least one whose 448 *
2^e reaches the largest finite magnitude written to it; when later rows of the
block need more, it grows and the codes of the rows before them are rounded to
the coarser scale.
"""
from __future__ import annotations

import math

import numpy as np

from .fp8 import E4M3_NAN, e4m3_decode, e4m3_encode
from .grouped import group_of
from .lrkv_oracle import attend, expand_head

MIN_EXP, MAX_EXP = -117, 119
POOLS = ("S_K", "S_V", "R_K", "R_V")


def needed_exp(a):
    """Least exponent in range with a <= 448 * 2^e."""
    e = MIN_EXP
    while e < MAX_EXP and a > math.ldexp(448.0, e):
        e += 1
    return e


def exp_of(byte):
    """Exponent that a stored byte stands for."""
    return np.clip(np.asarray(byte, np.int64) - 127, MIN_EXP, MAX_EXP)


def encode(x, e):
    """Codes of x / 2^e; what is not finite becomes the NaN code."""
    x = np.asarray(x, np.float64)
    ok = np.isfinite(x)
    return np.where(ok, e4m3_encode(np.where(ok, x, 0.0) * 2.0 ** -e), np.uint8(E4M3_NAN)).astype(np.uint8)


class Cache:
    """Codes [pages, page_size, heads, width] and exponent bytes [pages, blocks, heads] of the four pools."""

    def __init__(self, codes, exps):
        self.codes, self.exps = dict(codes), dict(exps)
        self.page_size = self.codes["R_K"].shape[1]
        self.block = self.page_size // self.exps["R_K"].shape[1]

    def copy(self):
        return Cache({k: v.copy() for k, v in self.codes.items()}, {k: v.copy() for k, v in self.exps.items()})

    def row(self, name, page, slot):
        """Values [heads, width] of one row."""
        e = exp_of(self.exps[name][page, slot // self.block])
        return e4m3_decode(self.codes[name][page, slot]) * 2.0 ** e.astype(np.float64)[:, None]


def places(cu_rows, start_pos, table, page_size, num_pages):
    """(row, request, position, page or None) of every row that a request owns; page None: skipped."""
    max_len = table.shape[1] * page_size
    for b in range(len(start_pos)):
        for i in range(cu_rows[b], cu_rows[b + 1]):
            pos = int(start_pos[b]) + i - int(cu_rows[b])
            page = int(table[b, pos // page_size]) if 0 <= pos < max_len else -1
            yield i, b, pos, page if 0 <= page < num_pages else None


def write(cache, rows, cu_rows, start_pos, table):
    """Quantise rows (name -> [n, heads, width]) into the cache."""
    units = {}  # (request, block of its positions) -> rows
    for i, b, pos, page in places(cu_rows, start_pos, table, cache.page_size, len(cache.codes["R_K"])):
        if page is not None:
            units.setdefault((b, pos // cache.block), []).append((i, pos, page))
    for unit in units.values():
        page, slot = unit[0][2], unit[0][1] % cache.page_size
        blk, before = slot // cache.block, slot % cache.block
        for name in POOLS:
            for h in range(cache.codes[name].shape[2]):
                x = np.stack([rows[name][i, h] for i, _, _ in unit]).astype(np.float64)
                finite = np.abs(x[np.isfinite(x)])
                e = needed_exp(finite.max(initial=0.0))
                if before:
                    old = int(exp_of(cache.exps[name][page, blk, h]))
                    e = max(e, old)
                    if e > old:
                        c = cache.codes[name][page, slot - before:slot, h]
                        c[...] = encode(e4m3_decode(c) * 2.0 ** old, e)
                if before == 0 or e > old:
                    cache.exps[name][page, blk, h] = e + 127
                for k, (_, pos, _) in enumerate(unit):
                    cache.codes[name][page, pos % cache.page_size, h] = encode(x[k], e)


def read(cache, name, cu_rows, start_pos, table, out):
    """Values of the rows into out [n, heads, width]; others stay."""
    for i, _, pos, page in places(cu_rows, start_pos, table, cache.page_size, len(cache.codes["R_K"])):
        if page is not None:
            out[i] = cache.row(name, page, pos % cache.page_size)
    return out


def history(cache, pages, n):
    """name -> values [rows, heads, width] of positions 0 .. n - 1 of a request, without rows on pages out of the pool."""
    ps, count = cache.page_size, len(cache.codes["R_K"])
    at = [(int(pages[j // ps]), j % ps) for j in range(n)]
    at = [(p, s) for p, s in at if 0 <= p < count]
    return {k: np.stack([cache.row(k, p, s) for p, s in at]) if at else np.zeros((0,) + cache.codes[k].shape[2:])
            for k in POOLS}


def attend_query(q, rows, B_K, B_V):
    """Output [H, d_h] of one query over a request's rows."""
    H, G = q.shape[0], rows["S_K"].shape[1]
    out = np.zeros(q.shape)
    for h in range(H):
        g = group_of(h, H, G)
        if len(rows["S_K"]):
            out[h] = attend(q[h], expand_head(rows["S_K"][:, g], rows["R_K"][:, h], B_K[h]),
                            expand_head(rows["S_V"][:, g], rows["R_V"][:, h], B_V[h]))
    return out
