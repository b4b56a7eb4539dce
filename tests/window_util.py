"""Inputs, float64 references and error bounds for the windowed attention
tests.

The bound of one output element follows the arithmetic that the kernels do,
with half a step of each type (bf16 2^-8, fp16 2^-11, fp32 2^-24) counted once
per rounding; a tensor-core sum of n products is taken as n additions that may
truncate (2^-23 each):

    |s_j - s_j*| <= E = max_j ((d_h + r) 2^-23 (|q|.|S_K| + |p|.|R_K|) + u_p |p|.|R_K|) c
        c = N / sqrt(d_h): p enters the score product with relative error u_p
    weights a_j = e_j / sum e: relative error <= 2 E + u_w + 2^-21 (exp, sum),
        u_w the rounding of the weight that enters the value product
    out: |got - ref| <= u_out |ref| + (2 E + u_w + 2^-21 + (rows + r + 32) 2^-23) A,
        A = sum_j a_j (|S_V[j]| + |R_V[j]| |B_V|^T)

u_p, u_w: bf16 caches carry p and (decode) the weights as bf16 high and low
halves, 2^-16; 8-bit caches as f16, 2^-11; fp32 caches as fp32, 2^-23; the
tiled prefill rounds its weights to bf16, 2^-8.
"""
import numpy as np

import lrkv_inputs as I
import oracle.window as W
from gpu_util import dev, pools_f64
from oracle.grouped import group_of

U_OUT = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -8, "f32": 2.0 ** -24}
U_P = {"bf16": 2.0 ** -16, "fp8": 2.0 ** -11, "f32": 2.0 ** -23}


def reference(q, pools, B_K, B_V, pages, t, page_size, window, sinks, dtype, N_K=None, u_w=None):
    """(ref, bound) [H, d_h] of one query at position t of a request."""
    ref = W.attend_query(q, *pools, B_K, B_V, pages, t, page_size, window, sinks, N_K)
    u_w = U_P[dtype] if u_w is None else u_w
    seen = W.visible(t, window, sinks)
    sk, sv, rk, rv = (W.pool_rows(p, pages, seen, page_size) for p in pools)
    if sk.ndim == 2:
        sk, sv = sk[:, None], sv[:, None]
    nk = None if N_K is None else W.pool_rows(N_K, pages, seen, page_size)
    H, d_h = q.shape
    r, G = rk.shape[2], sk.shape[1]
    bound = np.empty_like(ref)
    for h in range(H):
        g = group_of(h, H, G)
        p = q[h] @ B_K[h]
        c = (np.abs(nk[:, h]) if nk is not None else 1.0) / np.sqrt(d_h)
        s = (sk[:, g] @ q[h] + rk[:, h] @ p) * (nk[:, h] if nk is not None else 1.0) / np.sqrt(d_h)
        priv = np.abs(rk[:, h]) @ np.abs(p)
        # p itself is a sum of d_h products
        p_err = d_h * 2.0 ** -23 * (np.abs(rk[:, h]) @ (np.abs(q[h]) @ np.abs(B_K[h])))
        E = np.max(((d_h + r) * 2.0 ** -23 * (np.abs(sk[:, g]) @ np.abs(q[h]) + priv) + U_P[dtype] * priv + p_err) * c)
        a = np.exp(s - s.max())
        a /= a.sum()
        A = a @ np.abs(sv[:, g]) + (a @ np.abs(rv[:, h])) @ np.abs(B_V[h]).T
        bound[h] = U_OUT[dtype] * np.abs(ref[h]) + (2 * E + u_w + 2.0 ** -21 + (len(seen) + r + 32) * 2.0 ** -23) * A
    return ref, bound


def check(got, ref, bound, what=""):
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (f"{what}: {np.count_nonzero(bad)} of {bad.size} outside the bound, worst "
                           f"{np.max(np.abs(got - ref) / bound):.2f} of it")


def blank_unseen(case, window, sinks, page_garbage=-1):
    """Give the rows no decode query sees a NaN canary and pages that hold only such rows the id `page_garbage`.

    The page table keeps one column past the longest request."""
    canary = {"bf16": I.BF16_NAN_BITS, "fp8": I.FP8_NAN_CODE}.get(case.dtype, I.F32_NAN_CANARY)
    ps = case.page_size
    for b, L in enumerate(case.seq_lens):
        seen = set(W.visible(int(L) - 1, window, sinks))
        for j in range(int(L)):
            if j not in seen:
                for p in (case.S_K, case.S_V, case.R_K, case.R_V):
                    p[case.page_table[b, j // ps], j % ps] = canary
        for p in range(-(-int(L) // ps)):
            if not any(j in seen for j in range(p * ps, min(int(L), (p + 1) * ps))):
                case.page_table[b, p] = page_garbage


def decode_reference(case, window, sinks, N_K=None, pairs=None):
    """(ref, bound) [B, H, d_h] of a DecodeCase (zero where a request has no row)."""
    f = lambda a: I.to_f64(a, case.act_dtype)
    pools = pools_f64(case)
    q, B_K, B_V = f(case.q), f(case.B_K), f(case.B_V)
    ref, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b, L in enumerate(case.seq_lens):
        if L >= 1:
            ref[b], bound[b] = reference(q[b], pools, B_K, B_V, case.page_table[b], int(L) - 1, case.page_size,
                                         window, sinks, case.dtype, N_K)
    return ref, bound


def plan_on_device(seq_lens, new_rows, table, free, num_pages, page_size, max_rows, window, sinks, status=None, **kw):
    """api.page_plan of host inputs; returns (PagePlan, page table tensor)."""
    import torch

    import rank_kv_attention_gb300 as L
    free_pages = np.full(num_pages, -1, np.int32)
    free_pages[:len(free)] = free
    pt = dev(np.asarray(table), "i32")
    out = torch.full((num_pages,), -7, dtype=torch.int32, device="cuda")
    plan = L.page_plan(dev(np.asarray(seq_lens), "i32"), dev(np.asarray(new_rows), "i32"), pt, dev(free_pages, "i32"),
                       dev(np.array([len(free)]), "i32"), page_size, max_rows, free_out=out, window=window,
                       sinks=sinks, status=status, **kw)
    return plan, pt
