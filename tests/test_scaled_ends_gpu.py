"""The block-scaled cache on the GPU at the ends of what its calls allow."""
import numpy as np
import pytest
import torch

import lrkv_inputs as I
import oracle.scaled as S
from gpu_util import dev, host
from scaled_util import bf16, check, random_cache, reference, table_of, to_device, to_host
from test_scaled_gpu import (BAD_ROW, BAD_SEQLEN, check_decode, close_caches, decode_case, poison_past_the_end, projected,
                             run_decode, status, weights)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Decode: scales of the values at the ends of their range
# ---------------------------------------------------------------------------
LOW, HIGH = (10, 28), (237, 247)   # stored bytes: 2^-117 .. 2^-100, 2^110 .. 2^119
ENDS = [(16, 128, 48, 64, 64, 1), (32, 128, 32, 64, 16, 1), (4, 128, 64, 32, 32, 1), (24, 128, 56, 64, 64, 1),
        (8, 64, 16, 32, 16, 1), (12, 128, 72, 64, 64, 1), (16, 128, 32, 64, 64, 2), (2, 256, 256, 16, 16, 1)]


def set_ends(rng, cache, which):
    """Scales of the values; codes small enough that sums of a row's parts stay finite."""
    for k in ("S_V", "R_V"):
        codes, exps = cache.codes[k], cache.exps[k]
        codes[...] = S.e4m3_encode(np.clip(rng.standard_normal(codes.shape) * 16, -48, 48))
        low, high = rng.integers(*LOW, exps.shape), rng.integers(*HIGH, exps.shape)
        if which == "lowest":
            exps[...] = LOW[0]
        elif which == "highest":
            exps[...] = HIGH[1] - 1
        elif which == "low":
            exps[...] = low
        elif which == "high":
            exps[...] = high
        elif which == "heads":                     # loud and quiet heads next to each other
            exps[...] = np.where(rng.random((1, 1, exps.shape[2])) < 0.5, low, high)
        else:                                      # loud and quiet blocks of one head
            exps[...] = np.where(rng.random(exps.shape) < 0.5, low, high)
    for k in ("S_K", "R_K"):                       # tiles whose largest scores differ by some octaves
        cache.exps[k][:] = (127 - 7 + rng.integers(-3, 3, cache.exps[k].shape)).astype(np.uint8)


@pytest.mark.parametrize("which", ["lowest", "highest", "low", "high", "heads", "blocks"])
@pytest.mark.parametrize("H,d_h,r,ps,block,G", ENDS)
def test_decode_of_values_at_the_ends_of_the_range(H, d_h, r, ps, block, G, which):
    """Values of 2^-117 to 2^127: what a weight is worth does not depend on how loud its value is.  (Requests on shared
    pages, rows enough that a part of one has several tiles.)"""
    rng = np.random.default_rng(H + r)
    lens, many = [1500, 129, 64, 1, 700], 17
    cache, table, q, B_K, B_V = decode_case(rng, lens, H, d_h, r, ps, block, G)
    set_ends(rng, cache, which)
    poison_past_the_end(cache, table, lens)
    q, lens = bf16(rng, (len(lens) * many, H, d_h)), lens * many
    case = cache, np.tile(table, (many, 1)), q, B_K, B_V
    check_decode(run_decode(*case, lens), *case, lens, which=[0, 1, 2, 3, 4, 30, 44, 84], norm=None)


@pytest.mark.parametrize("H,d_h,r", [(16, 128, 48), (8, 64, 16)])
def test_decode_of_a_quiet_tile_behind_a_louder_score(H, d_h, r):
    """Two tiles of the least scale, equal scores in each, half an octave to two apart: both count.  (Requests on shared
    pages, enough that a part has both of its tiles.)"""
    rng = np.random.default_rng(60)
    B, n, many = 8, 256, 40
    cache, table, q, B_K, B_V = decode_case(rng, [n] * B, H, d_h, r, 64, 64)
    set_ends(rng, cache, "lowest")
    for k in ("S_K", "R_K"):
        cache.codes[k][:] = 0
    one = S.e4m3_encode(np.array(1.0))
    x = np.zeros((B, H, d_h), np.float32)
    for b in range(B):                             # scores in octaves: 2 and 2^e
        x[b, :, 0] = 2 * np.sqrt(d_h) * np.log(2.0)
        for j in range(n):
            page, slot = table[b, j // 64], j % 64
            cache.codes["S_K"][page, slot, 0, 0] = one
            cache.exps["S_K"][page, 0] = 127 + (0 if j < 128 else (-1, -2, -3, 0, -20, 1, -1, -1)[b])
    bits = I.f32_to_bf16_bits(x)
    q = np.tile(bits, (many, 1, 1)), np.tile(I.bf16_bits_to_f64(bits), (many, 1, 1))
    case, lens = (cache, np.tile(table, (many, 1)), q, B_K, B_V), [n] * (B * many)
    check_decode(run_decode(*case, lens), *case, lens, which=[*range(B), *range(100, 100 + B), B * many - 1], norm=None)


@pytest.mark.parametrize("H,d_h,r", [(16, 128, 48), (8, 64, 16)])
def test_decode_of_the_loudest_rows_that_agree(H, d_h, r):
    """Many rows of the same largest value: their mean is that value, however many they are."""
    rng = np.random.default_rng(61)
    lens = [4096, 1000]
    cache, table, q, B_K, B_V = decode_case(rng, lens, H, d_h, r, 64, 64)
    cache.codes["S_V"][:], cache.exps["S_V"][:] = 0x7e, 246        # 448 * 2^119
    cache.codes["R_V"][:], cache.exps["R_V"][:] = 0, 10
    check_decode(run_decode(cache, table, q, B_K, B_V, lens), cache, table, q, B_K, B_V, lens)


@pytest.mark.parametrize("which", ["one", "two"])
@pytest.mark.parametrize("H,d_h,r,G", [(16, 128, 48, 1), (32, 128, 32, 1), (8, 64, 16, 1), (12, 128, 72, 1), (16, 128, 32, 2)])
def test_decode_of_scores_larger_than_any_scale(H, d_h, r, G, which):
    """One row of each request (or two that agree) scores 2^12 to 2^100, all others nothing: the output is its value (their
    mean), whose scale must not drown in the score.  The weights are exactly 0 and 1 (or 1/2), so what is left of the bound
    is their rounding, the sums' and the output's."""
    rng = np.random.default_rng(69)
    powers, n, many = [12, 17, 22, 24, 26, 30, 60, 100], 300, 30
    B = len(powers)
    cache, table, q, B_K, B_V = decode_case(rng, [n] * B, H, d_h, r, 64, 16, G)
    set_ends(rng, cache, "blocks")
    cache.exps["R_V"][:] = rng.integers(120, 135, cache.exps["R_V"].shape)
    cache.exps["S_V"][:] = rng.integers(115, 140, cache.exps["S_V"].shape)
    for k in ("S_K", "R_K"):
        cache.codes[k][:] = 0
    x = np.zeros((B, H, d_h), np.float32)
    x[:, :, 0] = 1.5                               # (no power of two: the score has digits below its first)
    rows = [rng.choice(n, 2, replace=False) for _ in range(B)]
    want, size = np.zeros((B, H, d_h)), np.zeros((B, H, d_h))
    for b in range(B):
        picked = rows[b][:1] if which == "one" else rows[b]
        for j in picked:
            page, slot = table[b, j // 64], j % 64
            cache.codes["S_K"][page, slot, :, 0] = S.e4m3_encode(np.array(1.125))
            cache.exps["S_K"][page, slot // 16] = 127 + powers[b]
        for j in picked:
            page, slot = table[b, j // 64], j % 64
            for h in range(H):
                sv, rv = cache.row("S_V", page, slot)[h * G // H], cache.row("R_V", page, slot)[h]
                want[b, h] += (sv + B_V[1][h] @ rv) / len(picked)
                size[b, h] += (np.abs(sv) + np.abs(B_V[1][h]) @ np.abs(rv)) / len(picked)
    bits = I.f32_to_bf16_bits(x)
    q = np.tile(bits, (many, 1, 1)), np.tile(I.bf16_bits_to_f64(bits), (many, 1, 1))
    out = host(run_decode(cache, np.tile(table, (many, 1)), q, B_K, B_V, [n] * (B * many)), "bf16").reshape(many, B, H, d_h)
    for got in (out[0], out[many // 2], out[-1]):
        check(got, want, 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -21 + (r + 32) * 2.0 ** -23) * size)


# ---------------------------------------------------------------------------
# Decode: which kernel a shape takes
# ---------------------------------------------------------------------------
def on_tensor_cores(H, d_h, r, G=1, ps=64):
    """Whether a shape's decode keeps an operand image, of 4 rows of 128 bytes a head at least, for every request."""
    import rank_kv_attention_gb300 as L
    c = L.ScaledCache.empty(1, ps, H, d_h, r, block=16, groups=G)
    each = (L.decode_scaled_workspace_bytes(c, 40000, 4096) - L.decode_scaled_workspace_bytes(c, 30000, 4096)) / 10000
    return each >= 4 * H * (d_h + r + 2) + 512 * H


def test_shapes_that_decode_on_tensor_cores():
    """d_h = 128, one shared basis, 4 heads up to 32 in steps of 4, r up to 64: all of them but those whose operands do not
    fit, 24 heads of r = 64, 28 of r from 48 on and 32 of r from 48 on."""
    for H in range(4, 33, 4):
        for r in range(8, 65, 8):
            assert on_tensor_cores(H, 128, r) == (r <= {24: 56, 28: 40, 32: 40}.get(H, 64)), (H, r)
    for other in ((18, 128, 56), (36, 128, 8), (16, 128, 72), (16, 64, 48), (16, 128, 48, 2), (2, 128, 8)):
        assert not on_tensor_cores(*other), other


@pytest.mark.parametrize("H,r,ps,block", [(24, 56, 64, 64), (24, 48, 32, 16), (24, 64, 64, 64), (28, 40, 64, 32), (28, 8, 16, 16),
                                          (32, 40, 64, 64), (32, 48, 64, 64), (20, 64, 64, 16), (18, 56, 64, 64)])
def test_decode_of_many_heads(H, r, ps, block):
    """Shapes on both sides of what fits."""
    rng = np.random.default_rng(H * 100 + r)
    lens = [1, 17, 64, 129, 300, 1000, 2300]
    case = decode_case(rng, lens, H, 128, r, ps, block)
    poison_past_the_end(case[0], case[1], lens)
    st = status()
    check_decode(run_decode(*case, lens, status=st), *case, lens)
    assert int(st) == 0


# ---------------------------------------------------------------------------
# Prefill: rows past max_ctx
# ---------------------------------------------------------------------------
def prefill(rng, H, d_h, r, ps, start, rows_of, max_ctx, table=None, pages=None, d=64, x=None, q=None, change=None):
    """A call on an output of threes and a workspace of NaN: (output, the cache after it, status, cu_rows, (q, B_K, B_V), table,
    (the cache before it, weights, x))."""
    import rank_kv_attention_gb300 as L
    B, lens = len(start), np.add(start, rows_of)
    cu, n = np.concatenate([[0], np.cumsum(rows_of)]), int(sum(rows_of))
    if table is None:
        pages = int(sum(-(-v // ps) for v in lens)) + 1
        table = table_of(rng, lens, ps, pages)
    cache = random_cache(rng, pages, ps, H, d_h, r, 16, loud=1)
    if change:
        change(cache, table)
    w, x, q = weights(rng, d, H, d_h, r, 1), x or bf16(rng, (n, d)), q or bf16(rng, (n, H, d_h))
    B_K, B_V = bf16(rng, (H, d_h, r), r ** -0.5), bf16(rng, (H, d_h, r), r ** -0.5)
    dc, st = to_device(cache), status()
    out = torch.full((n, H, d_h), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((L.prefill_scaled_workspace_bytes(dc, B, n, max_ctx),), 0xff, dtype=torch.uint8, device="cuda")
    L.prefill_scaled(dev(x[0], "bf16"), dev(q[0], "bf16"), dev(cu, "i32"), dev(np.asarray(start), "i32"), max_ctx,
                     *[dev(w[m][0], "bf16") for m in w], dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), dc, dev(table, "i32"), out=out,
                     ws=ws, status=st)
    held = to_host(dc, cache)
    return host(out, "bf16"), held, int(st), cu, (q[1], B_K[1], B_V[1]), table, (cache, w, x)


PAST = [([0], [60], 50), ([0], [64], 64), ([0], [300], 200), ([64], [128], 64), ([64], [128], 100), ([64], [128], 192),
        ([130], [40], 150), ([130], [40], 130), ([700], [20], 705), ([700], [300], 960), ([0, 64, 300], [30, 90, 20], 140),
        ([0, 200, 10], [10, 20, 30], 215)]


PAST_SHAPES = [(16, 128, 48, 64, 64), (16, 128, 48, 64, 72), (8, 128, 16, 128, 64), (4, 32, 8, 32, 64)]


@pytest.mark.parametrize("start,rows_of,max_ctx", PAST)
@pytest.mark.parametrize("H,d_h,r,ps,d", PAST_SHAPES)
def test_prefill_flags_rows_past_max_ctx(H, d_h, r, ps, d, start, rows_of, max_ctx):
    """Rows from max_ctx on are written and flagged, behind a history or not; rows before it alone are not.  (d = 72: the
    append that stages its rows, whatever their number.)"""
    rng = np.random.default_rng(sum(start) + max_ctx)
    _, held, st, cu, _, table, (cache, w, x) = prefill(rng, H, d_h, r, ps, start, rows_of, max_ctx, d=d)
    assert st == (BAD_SEQLEN if max(np.add(start, rows_of)) > max_ctx else 0)
    S.write(cache, projected(x[1], w), cu, start, table)
    close_caches(held, cache, None, cu, start, table, d)


@pytest.mark.parametrize("start,rows_of,max_ctx", PAST)
@pytest.mark.parametrize("H,d_h,r,ps,d", PAST_SHAPES)
def test_prefill_past_max_ctx(H, d_h, r, ps, d, start, rows_of, max_ctx):
    """Rows up to max_ctx are attended as ever, whatever the workspace held; the outputs of those from it on are zero or as
    they were."""
    rng = np.random.default_rng(sum(start) + max_ctx)
    got, held, _, cu, (q, B_K, B_V), table, _ = prefill(rng, H, d_h, r, ps, start, rows_of, max_ctx, d=d)
    for b in range(len(start)):
        fit = min(max(0, max_ctx - start[b]), rows_of[b])
        for i in sorted({0, fit // 2, fit - 1} & set(range(fit))):
            ref, bound = reference(q[cu[b] + i], held, B_K, B_V, table[b], start[b] + i + 1, d_h == 128)
            check(got[cu[b] + i], ref, bound, f"request {b} row {i}")
        rest = got[cu[b] + fit:cu[b + 1]]
        assert ((rest == 0) | (rest == 3)).all()


@pytest.mark.parametrize("rows,d", [(20, 64), (40, 64), (20, 72)])
def test_prefill_past_max_ctx_in_a_pool_smaller_than_its_requests(rows, d):
    """Requests behind one shared page, values laid out once a page of the pool."""
    rng = np.random.default_rng(rows + d)
    H, r, ps, B, start, max_ctx = 8, 16, 64, 3, [64] * 3, 70
    table = np.array([[0, 1 + b] for b in range(B)], np.int32)
    got, held, st, cu, (q, B_K, B_V), _, _ = prefill(rng, H, 128, r, ps, start, [rows] * B, max_ctx, table, pages=4, d=d)
    assert st == BAD_SEQLEN
    for b in range(B):
        for i in (0, max_ctx - 65):
            ref, bound = reference(q[cu[b] + i], held, B_K, B_V, table[b], 65 + i, True)
            check(got[cu[b] + i], ref, bound, f"request {b} row {i}")
        rest = got[cu[b] + max_ctx - 64:cu[b + 1]]
        assert ((rest == 0) | (rest == 3)).all()


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 32, 8, 32)])
def test_prefill_at_the_end_of_the_table(H, d_h, r, ps):
    """max_ctx is the table's end: rows past it have no place, which is another flag."""
    rng = np.random.default_rng(62)
    table = np.arange(4, dtype=np.int32)[None]
    got, held, st, cu, (q, B_K, B_V), _, _ = prefill(rng, H, d_h, r, ps, [4 * ps - 30], [70], 4 * ps, table, pages=4)
    assert st == BAD_ROW
    for i in (0, 29):
        ref, bound = reference(q[i], held, B_K, B_V, table[0], 4 * ps - 30 + i + 1, d_h == 128)
        check(got[i], ref, bound, f"row {i}")
    assert not got[30:].any()


# ---------------------------------------------------------------------------
# Prefill: what is not finite; many requests; the least values
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (32, 128, 16, 64), (4, 32, 8, 32)])
@pytest.mark.parametrize("start,rows", [(0, 40), (10, 150), (900, 100), (0, 900)])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_prefill_of_a_query_that_is_not_finite(H, d_h, r, ps, start, rows, value):
    """It gives NaN in its row and head, as a decode does; the other rows and heads are right."""
    rng = np.random.default_rng(63 + rows)
    bits, q = bf16(rng, (rows, H, d_h))
    for i, h in ((0, 1), (rows // 2, 2), (rows - 1, 0)):
        bits[i, h, 7], q[i, h, 7] = (I.BF16_NAN_BITS if np.isnan(value) else 0x7f80), value
    got, held, st, _, (_, B_K, B_V), table, _ = prefill(rng, H, d_h, r, ps, [start], [rows], start + rows, q=(bits, q))
    assert st == 0
    for i, h in ((0, 1), (rows // 2, 2), (rows - 1, 0)):
        assert np.isnan(got[i, h]).all(), (i, h)
        got[i, h] = q[i, h] = 0
    assert np.isfinite(got).all()
    for i, h in ((0, 1), (rows // 2, 2), (rows - 1, 0), (rows // 3, 0)):
        ref, bound = reference(q[i], held, B_K, B_V, table[0], start + i + 1, d_h == 128)
        if i != rows // 3:
            ref[h] = 0                             # (the row put to zero above)
        check(got[i], ref, bound, f"row {i}", norm=None)


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 32, 8, 32)])
@pytest.mark.parametrize("pool", ["S_K", "S_V"])
def test_prefill_behind_a_row_that_is_not_finite(H, d_h, r, ps, pool):
    """A NaN code of a row that all queries see makes their outputs NaN, and no other request's."""
    rng = np.random.default_rng(64)

    def change(cache, table):
        cache.codes[pool][table[0, 1], 3, 0, :] = 0x7f
    got, held, st, cu, (q, B_K, B_V), table, _ = prefill(rng, H, d_h, r, ps, [100, 40], [30, 50], 130, change=change)
    assert st == 0 and np.isnan(got[:30]).all()
    for i in (30, 79):
        ref, bound = reference(q[i], held, B_K, B_V, table[1], 40 + i - 30 + 1, d_h == 128)
        check(got[i], ref, bound, f"row {i}")


def test_prefill_of_more_requests_than_a_grid_holds():
    """70,000 requests, most without rows."""
    rng = np.random.default_rng(65)
    H, r, ps, B = 4, 16, 64, 70000
    live = np.sort(rng.choice(B, 30, replace=False))
    live[-1] = B - 1
    rows_of, start = np.zeros(B, int), np.zeros(B, int)
    rows_of[live], start[live] = rng.integers(1, 70, 30), rng.integers(0, 60, 30)
    table = np.full((B, 2), -1, np.int32)
    table[live] = rng.permutation(61)[:60].reshape(30, 2)
    got, held, st, cu, (q, B_K, B_V), _, _ = prefill(rng, H, 128, r, ps, list(start), list(rows_of), 128, table, pages=61)
    assert st == 0
    for b in live:
        for i in {0, rows_of[b] - 1}:
            ref, bound = reference(q[cu[b] + i], held, B_K, B_V, table[b], int(start[b] + i) + 1, True)
            check(got[cu[b] + i], ref, bound, f"request {b} row {i}")


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 32, 8, 32)])
@pytest.mark.parametrize("which", ["lowest", "low"])
def test_prefill_behind_the_smallest_values(H, d_h, r, ps, which):
    """One new row of zeros behind a history of the least scales."""
    rng = np.random.default_rng(66)
    x = np.zeros((1, 64), np.uint16), np.zeros((1, 64))
    got, held, st, _, (q, B_K, B_V), table, _ = prefill(rng, H, d_h, r, ps, [400], [1], 401, x=x,
                                                        change=lambda c, t: set_ends(rng, c, which))
    ref, bound = reference(q[0], held, B_K, B_V, table[0], 401, d_h == 128)
    check(got[0], ref, bound, norm=None)
    assert st == 0 and ref.any()


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 32, 8, 32)])
@pytest.mark.parametrize("byte", [10, 207])
def test_prefill_behind_rows_that_agree(H, d_h, r, ps, byte):
    """A history of the same largest values, as quiet as the cache holds them, or 448 * 2^80: with 1500 rows below the 2^100
    to which the tiled kernel's sums are finite.  Their mean is that value."""
    rng = np.random.default_rng(68)

    def change(cache, table):
        cache.codes["S_V"][:], cache.exps["S_V"][:] = 0x7e, byte
        cache.codes["R_V"][:], cache.exps["R_V"][:] = 0, 10
    x = np.zeros((1, 64), np.uint16), np.zeros((1, 64))
    got, held, st, _, (q, B_K, B_V), table, _ = prefill(rng, H, d_h, r, ps, [1500], [1], 1501, x=x, change=change)
    ref, bound = reference(q[0], held, B_K, B_V, table[0], 1501, d_h == 128)
    check(got[0], ref, bound)
    assert st == 0


# ---------------------------------------------------------------------------
# Calls one after another
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 32, 8, 32)])
def test_calls_in_a_row_share_a_workspace(H, d_h, r, ps):
    """Prefills with either append, appends and decodes on one stream and one workspace, none waited for: the same to the
    bit as each with its own, waited for."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(67)
    d, B, width = 64, 3, 2048 // ps
    cache, table = random_cache(rng, B * width, ps, H, d_h, r, 16, loud=1), rng.permutation(B * width).astype(np.int32)
    dt = dev(table.reshape(B, width), "i32")
    w = [dev(a, "bf16") for a, _ in weights(rng, d, H, d_h, r, 1).values()]
    Bs = [dev(bf16(rng, (H, d_h, r), r ** -0.5)[0], "bf16") for _ in range(2)]
    steps, at = [], np.zeros(B, int)
    for rows_of in ([300, 1, 200], [10, 20, 9], [1, 1, 1], [0, 700, 40], [1, 1, 1], [30, 0, 0], [1, 1, 1], [600, 500, 400]):
        n = sum(rows_of)
        steps.append((dev(bf16(rng, (n, d))[0], "bf16"), dev(bf16(rng, (n, H, d_h))[0], "bf16"),
                      dev(np.concatenate([[0], np.cumsum(rows_of)]), "i32"), dev(at, "i32"), dev(at + rows_of, "i32"),
                      max(rows_of) == 1))
        at = at + rows_of
    size = max(L.prefill_scaled_workspace_bytes(to_device(cache), B, s[0].shape[0], 2048) for s in steps)
    size = max(size, L.decode_scaled_workspace_bytes(to_device(cache), B, 2048))

    def run(ws_of, after):
        dc, outs = to_device(cache), []
        torch.cuda.synchronize()
        for x, q, cu, start, lens, single in steps:
            if single:
                L.append_scaled(x, cu, start, *w, dc, dt, ws=ws_of())
                after()
                outs.append(L.decode_scaled(q, dc, *Bs, lens, dt, 2048, ws=ws_of()))
            else:
                outs.append(L.prefill_scaled(x, q, cu, start, 2048, *w, *Bs, dc, dt, ws=ws_of()))
            after()
        torch.cuda.synchronize()
        return dc, outs
    one = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    a, outs = run(lambda: one, lambda: None)
    b, alone = run(lambda: torch.full((size,), 0x7f, dtype=torch.uint8, device="cuda"), torch.cuda.synchronize)
    for x, y in zip(outs, alone):
        assert torch.isfinite(x).all() and torch.equal(x, y)
    for k in ("S_K", "S_V", "R_K", "R_V", "E_S_K", "E_S_V", "E_R_K", "E_R_V"):
        assert torch.equal(getattr(a, k).view(torch.uint8), getattr(b, k).view(torch.uint8)), k
