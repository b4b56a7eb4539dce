"""Inputs, float64 references and error bounds for the tests of the block-scaled
cache.

Codes and exponents of a write are defined to the bit and compared so.  The bound
of an attention output follows the kernels' arithmetic.  The tensor-core decode
takes q and p = q B_K[h] as three E4M3 terms and the weights as two, each term the
nearest E4M3 value of what the ones before leave.  E4M3's half step is 2^-4 of a
value's power of two, or 2^-10 below 2^-6, and terms are scaled so that the
largest of the first is 2^7.8 at least: three terms are off by at most 2^-14 of
the value or 2^-26 of the row's largest, two by 2^-9 or 2^-21 of the largest.

    |s_j - s_j*| <= E = max_j (2^-14 + n 2^-23) (|q|.|S_K| + |p|.|R_K|) + 2^-26 (max|q| sum|S_K| + max|p| sum|R_K|)
                        + d_h 2^-23 |R_K|.(|q| |B_K|)            (/ sqrt(d_h); n = d_h + r products; p a sum of d_h)
    weights a_j = e_j / sum e: relative error <= 2 E + 2^-9 + 2^-21 (exp, sum)
    |got - ref| <= 2^-8 |ref| + (2 E + 2^-9 + 2^-21 + (rows + r + 32) 2^-23) A + 2^-21 F
        A = sum_j a_j (|S_V[j]| + |R_V[j]| |B_V|^T)
        F = max_j (a_j 2^eS_j) sum_j |S_V code| + max_j (a_j 2^eR_j) sum_j |R_V code| |B_V|^T
A sum over the tensor core is taken as additions that may truncate (2^-23 each).
The tiled prefill rounds its weights to bf16 (2^-8 for the 2^-9) and p to 2^-16.
"""
import numpy as np
import torch

import lrkv_inputs as I
import oracle.scaled as S
from gpu_util import dev
from oracle.fp8 import e4m3_decode
from oracle.grouped import group_of

POOLS = S.POOLS


def random_cache(rng, pages, page_size, H, d_h, r, block, G=1, loud=3):
    """A cache of random codes; heads and blocks differ in magnitude."""
    codes, exps = {}, {}
    for k in POOLS:
        heads, width = (G, d_h) if k[0] == "S" else (H, r)
        c = rng.integers(0, 256, (pages, page_size, heads, width)).astype(np.uint8)
        v = np.clip(rng.standard_normal(c.shape) * 96, -448, 448)
        codes[k] = S.e4m3_encode(v)
        e = rng.integers(-1, 2, (pages, page_size // block, heads)) + rng.integers(-loud, loud + 1, heads) - 7
        exps[k] = (e + 127).astype(np.uint8)
    return S.Cache(codes, exps)


def to_device(cache):
    """The oracle's cache as an api.ScaledCache."""
    import rank_kv_attention_gb300 as L
    t = {k: dev(cache.codes[k][:, :, 0] if k[0] == "S" and cache.codes[k].shape[2] == 1 else cache.codes[k], "fp8")
         for k in POOLS}
    e = {k: torch.from_numpy(cache.exps[k].copy()).cuda() for k in POOLS}
    return L.ScaledCache(*[t[k] for k in POOLS], *[e[k] for k in POOLS])


def to_host(dc, like):
    """The device cache's bytes, shaped like the oracle's cache `like`."""
    codes = {k: getattr(dc, k).cpu().view(torch.uint8).numpy().reshape(like.codes[k].shape) for k in POOLS}
    return S.Cache(codes, {k: getattr(dc, "E_" + k).cpu().numpy() for k in POOLS})


def assert_same(got, want):
    """Equal caches; the two NaN codes are the same."""
    for k in POOLS:
        assert np.array_equal(got.exps[k], want.exps[k]), f"E_{k}: {np.argwhere(got.exps[k] != want.exps[k])[:5]}"
        a, b = (np.where((c & 0x7f) == 0x7f, 0x7f, c) for c in (got.codes[k], want.codes[k]))
        assert np.array_equal(a, b), f"{k}: {np.argwhere(a != b)[:5]} of {np.count_nonzero(a != b)}"


def table_of(rng, lens, page_size, pages, width=None):
    """Page table of requests with these lengths, -1 past their last page."""
    need = [-(-n // page_size) for n in lens]
    ids = rng.permutation(pages)[:sum(need)]
    assert sum(need) <= pages
    t = np.full((len(lens), width or max(1, max(need))), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k], at = ids[at:at + k], at + k
    return t


def bf16(rng, shape, std=1.0):
    """(bits, float64 values) of bf16 normals."""
    bits = I.f32_to_bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))
    return bits, I.bf16_bits_to_f64(bits)


def reference(q, cache, B_K, B_V, pages, n, tiled=False):
    """(ref, bound) [H, d_h] of one query over a request's first n rows."""
    rows = S.history(cache, pages, n)
    ref = S.attend_query(q, rows, B_K, B_V)
    H, d_h = q.shape
    r, G = rows["R_K"].shape[2], rows["S_K"].shape[1]
    bound = np.zeros_like(ref)
    ps = cache.page_size
    at = [(int(pages[j // ps]), j % ps) for j in range(n) if 0 <= int(pages[j // ps]) < len(cache.codes["R_K"])]
    if not at:
        return ref, bound
    pg, sl = np.array(at).T
    eS, eR = (S.exp_of(cache.exps[k][pg, sl // cache.block]).astype(np.float64) for k in ("S_V", "R_V"))
    cS, cR = (np.abs(e4m3_decode(cache.codes[k][pg, sl])) for k in ("S_V", "R_V"))
    u_q, u_w = (2.0 ** -16, 2.0 ** -8) if tiled else (2.0 ** -14, 2.0 ** -9)
    for h in range(H):
        g = group_of(h, H, G)
        sk, sv, rk, rv = rows["S_K"][:, g], rows["S_V"][:, g], rows["R_K"][:, h], rows["R_V"][:, h]
        p = q[h] @ B_K[h]
        s = (sk @ q[h] + rk @ p) / np.sqrt(d_h)
        mass = np.abs(sk) @ np.abs(q[h]) + np.abs(rk) @ np.abs(p)
        floor = np.abs(q[h]).max() * np.abs(sk).sum(1) + np.abs(p).max() * np.abs(rk).sum(1)
        p_err = d_h * 2.0 ** -23 * (np.abs(rk) @ (np.abs(q[h]) @ np.abs(B_K[h])))
        E = np.max((u_q + (d_h + r) * 2.0 ** -23) * mass + 2.0 ** -26 * floor + p_err) / np.sqrt(d_h)
        a = np.exp(s - s.max())
        a /= a.sum()
        absB = np.abs(B_V[h]).T
        A = a @ np.abs(sv) + (a @ np.abs(rv)) @ absB
        F = np.max(a * 2.0 ** eS[:, g]) * cS[:, g].sum(0) + (np.max(a * 2.0 ** eR[:, h]) * cR[:, h].sum(0)) @ absB
        bound[h] = (2.0 ** -8 * np.abs(ref[h]) + (2 * E + u_w + 2.0 ** -21 + (n + r + 32) * 2.0 ** -23) * A
                    + 2.0 ** -21 * F)
    return ref, bound


def check(got, ref, bound, what="", norm=2.0 ** -7):
    """Every element within its bound, and, unless norm is None, the whole within `norm` of its size: the worst case above
    grows with the number of rows, but errors of rows are independent and add up as the values, of either sign, do, so the
    whole is off by about the half steps of the output (2^-8) and of the weights (2^-9)."""
    if norm is not None:
        off, size = np.linalg.norm(got - ref), np.linalg.norm(ref)
        assert off <= norm * size, f"{what}: {off / size:.2e} of its size off"
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (f"{what}: {np.count_nonzero(bad)} of {bad.size} outside the bound, worst "
                           f"{np.max(np.abs(got - ref) / np.maximum(bound, 1e-300)):.2f} of it")
