"""lrkv_decode_window, lrkv_prefill_window and lrkv_page_plan (through the C
ABI) against the float64 / integer definitions of oracle/window.py, with the
error bounds of window_util."""
import numpy as np
import pytest
import torch

import lrkv_inputs as I
import oracle
import oracle.window as W
from gpu_util import DevDecode, dev, host
from window_util import blank_unseen, check, decode_reference, plan_on_device, reference

pytestmark = pytest.mark.gpu

LENS = [1, 17, 300, 64, 65, 129, 700]


def run_decode(d, window, sinks, **kw):
    import rank_kv_attention_gb300 as L
    return L.decode_window(d.q, d.cache, d.B_K, d.B_V, d.seq_lens, d.page_table, d.max_seq_len, window, sinks, **kw)


def decode_case(lens, H, d_h, r, dtype="bf16", seed=0, **kw):
    return I.make_decode_case(len(lens), H, d_h, r, lens, dtype=dtype, seed=seed, shuffle=True, spare_pages=3, **kw)


# ---------------------------------------------------------------------------
# Decode
# ---------------------------------------------------------------------------
SHAPES = [(16, 128, 48, "bf16"), (16, 128, 56, "bf16"), (32, 128, 32, "bf16"), (16, 128, 32, "bf16"),
          (16, 128, 64, "bf16"), (16, 128, 16, "bf16"), (32, 128, 16, "bf16"), (16, 128, 48, "fp8"),
          (16, 128, 56, "fp8"), (32, 128, 32, "fp8"), (16, 128, 64, "fp8"),
          (8, 64, 24, "bf16"), (4, 128, 40, "bf16"), (4, 16, 4, "f32"), (6, 32, 8, "f32"), (8, 64, 24, "fp8")]


@pytest.mark.parametrize("H,d_h,r,dtype", SHAPES)
@pytest.mark.parametrize("window,sinks", [(100, 5), (64, 0)])
def test_decode_shapes(H, d_h, r, dtype, window, sinks):
    case = decode_case(LENS, H, d_h, r, dtype, seed=H + r)
    blank_unseen(case, window, sinks)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = host(run_decode(DevDecode(case), window, sinks, status=status), case.act_dtype)
    check(got, *decode_reference(case, window, sinks), f"{H} {d_h} {r} {dtype}")
    assert int(status.item()) == 0


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 16, 17, 64, 100, 2 ** 31 - 1])
def test_decode_window_edges(window, sinks):
    """Windows and sinks at, below and above tiles, pages and lengths; unseen rows hold NaN."""
    lens = [1, 15, 16, 17, 64, 65, 128, 129, 257, 400]
    case = decode_case(lens, 16, 128, 48, seed=3)
    blank_unseen(case, window, sinks, page_garbage=10 ** 6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = host(run_decode(DevDecode(case), window, sinks, status=status), "bf16")
    check(got, *decode_reference(case, window, sinks), f"window {window} sinks {sinks}")
    assert int(status.item()) == 0


@pytest.mark.parametrize("page_size,dtype", [(16, "bf16"), (32, "bf16"), (128, "bf16"), (1024, "bf16"), (32, "fp8"),
                                             (48, "fp8"), (16, "f32")])
def test_decode_page_sizes(page_size, dtype):
    H, d_h, r = (6, 32, 8) if dtype == "f32" else (16, 128, 48)
    case = decode_case([5, 33, 200, 16, 1100], H, d_h, r, dtype, seed=page_size, page_size=page_size)
    blank_unseen(case, 90, 20)
    got = host(run_decode(DevDecode(case), 90, 20), case.act_dtype)
    check(got, *decode_reference(case, 90, 20), f"page {page_size} {dtype}")


@pytest.mark.parametrize("B,lo,hi,window,sinks", [(1, 3000, 3000, 2500, 4), (3, 900, 5000, 3000, 100), (1, 9000, 9000, 64, 8),
                                                  (40, 1, 700, 300, 4), (170, 1, 200, 77, 3), (333, 20, 90, 33, 1)])
def test_decode_batches(B, lo, hi, window, sinks):
    """Few requests with long windows to many requests with short ones."""
    lens = np.random.default_rng(B).integers(lo, hi + 1, size=B)
    case = decode_case(lens, 16, 128, 48, seed=B)
    blank_unseen(case, window, sinks)
    got = host(run_decode(DevDecode(case), window, sinks), "bf16")
    check(got, *decode_reference(case, window, sinks), f"B={B}")


@pytest.mark.parametrize("H,r,groups", [(16, 48, 2), (16, 32, 2), (16, 48, 4), (8, 24, 2)])
def test_decode_groups(H, r, groups):
    case = decode_case([1, 40, 300, 513], H, 128, r, seed=groups, groups=groups)
    blank_unseen(case, 130, 9)
    got = host(run_decode(DevDecode(case), 130, 9), "bf16")
    check(got, *decode_reference(case, 130, 9), f"groups {groups}")


@pytest.mark.parametrize("H,d_h,r,dtype", [(16, 128, 48, "bf16"), (16, 128, 48, "fp8"), (4, 16, 4, "f32"), (8, 64, 24, "bf16")])
def test_decode_key_norms(H, d_h, r, dtype):
    """Scores are multiplied by the stored reciprocal norms of the visible rows."""
    case = decode_case([1, 40, 300, 513], H, d_h, r, dtype, seed=11)
    blank_unseen(case, 130, 9)
    d = DevDecode(case)
    adt = case.act_dtype
    N = np.random.default_rng(5).uniform(0.5, 1.5, size=case.R_K.shape[:3]).astype(np.float32)
    N = I.f32_to_bf16_bits(N) if adt == "bf16" else N
    d.cache.N_K, d.cache.norm_eps = dev(N, adt), 1e-6
    check(host(run_decode(d, 130, 9), adt), *decode_reference(case, 130, 9, N_K=I.to_f64(N, adt)), dtype)


def test_decode_whole_history_is_lrkv_decode():
    """A window that covers everything attends what lrkv_decode attends: both lie within the bound."""
    case = decode_case([1, 100, 777, 2048], 16, 128, 48, seed=21)
    d = DevDecode(case)
    ref, bound = decode_reference(case, 10 ** 6, 0)
    check(host(run_decode(d, 10 ** 6, 0), "bf16"), ref, bound, "window")
    check(host(d.run(), "bf16"), ref, bound, "decode")


@pytest.mark.parametrize("H,d_h,r,dtype", [(16, 128, 48, "bf16"), (16, 128, 48, "fp8"), (4, 16, 4, "f32")])
def test_decode_bad_metadata_is_flagged_not_read(H, d_h, r, dtype):
    import rank_kv_attention_gb300 as L
    case = decode_case([40, 400, 300, 9, 60], H, d_h, r, dtype, seed=9)
    window, sinks = 100, 4
    d = DevDecode(case)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d.seq_lens[0] = 0
    d.seq_lens[3] = case.page_table.shape[1] * 64 + 1
    d.page_table[2, 3] = 10 ** 6          # rows 200 .. 255 of the visible 200 .. 299
    d.page_table[4, 0] = -1               # its only page: nothing is left
    got = host(run_decode(d, window, sinks, status=status), case.act_dtype)
    assert int(status.item()) == (L.LRKV_STATUS_BAD_SEQLEN | L.LRKV_STATUS_BAD_PAGE)
    assert np.all(got[0] == 0) and np.all(got[3] == 0) and np.all(got[4] == 0)
    ref, bound = decode_reference(case, window, sinks)
    check(got[1], ref[1], bound[1], "the request beside them")
    assert np.all(np.isfinite(got[2]))


def test_decode_huge_scores_and_infinities_in_unseen_rows():
    """Scores of +-1e4 (one row takes all the weight) and infinities where nothing is seen."""
    case = decode_case([500, 77], 16, 128, 48, seed=13)
    case.q[:] = I.f32_to_bf16_bits(I.bf16_bits_to_f32(case.q) * np.float32(1000))
    blank_unseen(case, 64, 3)
    inf = np.uint16(0x7F80)
    for b, L in enumerate(case.seq_lens):
        for j in range(3, L - 64):
            for p in (case.S_K, case.S_V, case.R_K, case.R_V):
                if case.page_table[b, j // 64] >= 0:
                    p[case.page_table[b, j // 64], j % 64] = inf
    got = host(run_decode(DevDecode(case), 64, 3), "bf16")
    check(got, *decode_reference(case, 64, 3))


@pytest.mark.parametrize("H,d_h,r,dtype", [(16, 128, 48, "bf16"), (16, 128, 48, "fp8"), (4, 16, 4, "f32"), (8, 64, 24, "bf16")])
@pytest.mark.parametrize("row", [0, 3, 201, 230, 299])
def test_decode_nan_in_a_visible_row_is_not_hidden(H, d_h, r, dtype, row):
    """A NaN key of a row that a query sees makes that request's outputs NaN, and no other's."""
    canary = {"bf16": I.BF16_NAN_BITS, "fp8": I.FP8_NAN_CODE}.get(dtype, I.F32_NAN_CANARY)
    case = decode_case([300, 300, 8], H, d_h, r, dtype, seed=31)
    clean = host(run_decode(DevDecode(case), 99, 4), case.act_dtype)
    case.S_K[case.page_table[1, row // 64], row % 64] = canary
    got = host(run_decode(DevDecode(case), 99, 4), case.act_dtype)
    assert np.isnan(got[1]).all()
    np.testing.assert_array_equal(got[[0, 2]], clean[[0, 2]])


def test_decode_stale_workspace_repeats_bit_for_bit():
    import rank_kv_attention_gb300 as L
    for lens, window, shape in (([700, 5, 2500], 600, (16, 128, 48, "bf16")), ([9000], 8000, (16, 128, 48, "bf16")),
                                ([30, 900, 77], 200, (6, 32, 8, "f32"))):
        H, d_h, r, dtype = shape
        case = decode_case(lens, H, d_h, r, dtype, seed=8)
        d = DevDecode(case)
        ws = L.workspace(L.decode_window_workspace_bytes(len(lens), H, d_h, r, d.max_seq_len, window, 4, d.cache.dtype) + 256)
        outs = []
        for fill in (0xFF, 0x7F, 0x00):
            ws.fill_(fill)
            outs.append(run_decode(d, window, 4, ws=ws).clone())
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        check(host(outs[0], dtype), *decode_reference(case, window, 4))


def test_decode_streams_at_once_and_graph_replay():
    """Calls on four streams at once, then one captured and replayed with new queries and lengths."""
    import rank_kv_attention_gb300 as L
    cases = [decode_case(np.random.default_rng(s).integers(1, 3000, size=24), 16, 128, 48, seed=s) for s in range(4)]
    ds = [DevDecode(c) for c in cases]
    alone = [run_decode(d, 1024, 4).clone() for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    outs = []
    for _ in range(5):
        outs = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                outs.append(run_decode(d, 1024, 4))
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert torch.equal(a, o)
    # an explicit stream argument
    o = run_decode(ds[0], 1024, 4, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(o, alone[0])
    d = ds[1]
    out, ws = torch.empty_like(d.q), L.workspace(L.decode_window_workspace_bytes(24, 16, 128, 48, d.max_seq_len, 1024, 4))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_decode(d, 1024, 4, out=out, ws=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, alone[1])
    d.q.copy_(d.q.flip(0).clone())
    d.seq_lens.copy_(torch.clamp(d.seq_lens - 1, min=1))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, run_decode(d, 1024, 4))


@pytest.mark.parametrize("H,r,dtype", [(16, 48, "bf16"), (32, 32, "bf16"), (16, 56, "bf16"), (16, 64, "fp8")])
@pytest.mark.parametrize("B", [1, 2, 5])
def test_decode_split_requests(H, r, dtype, B):
    """Few requests with windows long enough that each is split over clusters, one of them short and one empty."""
    lens = [6000, 40, 0, 4097, 5999][:B]
    case = decode_case(lens, H, 128, r, dtype, seed=B)
    blank_unseen(case, 4000, 30)
    got = host(run_decode(DevDecode(case), 4000, 30), case.act_dtype)
    check(got, *decode_reference(case, 4000, 30), f"B={B}")


@pytest.mark.parametrize("H,r,dtype", [(16, 48, "bf16"), (32, 32, "bf16"), (16, 56, "bf16"), (16, 64, "fp8")])
@pytest.mark.parametrize("lens,window,sinks", [([3000], 1000, 4), ([6000, 40], 4000, 30), ([1500, 0, 1400, 1501, 17], 1024, 0),
                                               ([2100] * 7 + [5], 2048, 4), ([1100] * 16, 1024, 4)])
def test_decode_split_with_a_workspace(H, r, dtype, lens, window, sinks):
    """The layout that a caller's workspace allows, beside the one without: both within the bound; one byte less is refused."""
    import rank_kv_attention_gb300 as L
    case = decode_case(lens, H, 128, r, dtype, seed=len(lens))
    blank_unseen(case, window, sinks)
    d, (ref, bound) = DevDecode(case), decode_reference(case, window, sinks)
    need = L.decode_window_workspace_bytes(len(lens), H, 128, r, d.max_seq_len, window, sinks, d.cache.dtype)
    assert need > 0 or len(lens) > 5
    check(host(run_decode(d, window, sinks), case.act_dtype), ref, bound, "without")
    if need:
        ws = L.workspace(need).fill_(0xFF)
        got = run_decode(d, window, sinks, ws=ws)
        check(host(got, case.act_dtype), ref, bound, "with")
        assert torch.equal(got, run_decode(d, window, sinks, ws=ws))
        with pytest.raises(L.LrkvError):
            run_decode(d, window, sinks, ws=L.workspace(need - 256)[:need - 256])


# ---------------------------------------------------------------------------
# Prefill
# ---------------------------------------------------------------------------
def prefill_inputs(rows, starts, d, H, d_h, r, dtype, window, sinks, seed, page_size=64, groups=1, unseen=-1):
    """A cache whose history rows that the chunk can see are filled; other rows hold NaN, pages without a
    visible row have the id `unseen`."""
    from rank_kv_attention_gb300.api import PagedCache
    rng = np.random.default_rng(seed)
    adt = I.act_dtype(dtype)
    w = I.make_weights(d, H, d_h, r, adt, seed=seed, groups=groups)
    ends = [s + n for s, n in zip(starts, rows)]
    pt, num_pages = I.make_page_table(ends, page_size, True, rng, 2)
    pools = list(I.empty_pools(num_pages, page_size, H, d_h, r, dtype, canary=True, groups=groups))
    for b, (s, n) in enumerate(zip(starts, rows)):
        for p in range(-(-ends[b] // page_size)):
            live = [j for j in range(p * page_size, min(ends[b], (p + 1) * page_size))
                    if n and (j > s - window or j < sinks)]
            for j in live:
                if j < s:
                    for pool in pools:
                        x = rng.standard_normal(pool.shape[2:]).astype(np.float32)
                        pool[pt[b, p], j % page_size] = (I.f32_to_bf16_bits(x) if dtype == "bf16" else
                                                         I.f32_to_e4m3_codes(x / I.FP8_SCALE) if dtype == "fp8" else x)
            if not live:
                pt[b, p] = unseen
    n = sum(rows)
    enc = I.f32_to_bf16_bits if adt == "bf16" else (lambda a: a)
    X = enc(rng.standard_normal((n, d)).astype(np.float32))
    Q = enc(rng.standard_normal((n, H, d_h)).astype(np.float32))
    scale = (I.FP8_SCALE,) * 4 if dtype == "fp8" else (1.0,) * 4
    cache = PagedCache(*[dev(p, dtype) for p in pools], scale)
    return w, pt, cache, X, Q


def run_prefill(w, pt, cache, X, Q, rows, starts, window, sinks, adt, **kw):
    import rank_kv_attention_gb300 as L
    cu = np.concatenate([[0], np.cumsum(rows)])
    max_ctx = max(1, max(s + n for s, n in zip(starts, rows)))
    return L.prefill_window(dev(X, adt), dev(Q, adt), dev(cu, "i32"), dev(np.array(starts), "i32"), max_ctx,
                            dev(w.W_S_K, adt), dev(w.W_S_V, adt), dev(w.U_K, adt), dev(w.U_V, adt), dev(w.B_K, adt),
                            dev(w.B_V, adt), cache, dev(pt, "i32"), window, sinks, **kw)


def cache_f64(cache, dtype):
    if dtype == "fp8":
        return [oracle.fp8.dequantize(p.view(torch.uint8).cpu().numpy(), s)
                for p, s in zip((cache.S_K, cache.S_V, cache.R_K, cache.R_V), cache.scale)]
    return [host(p, dtype) for p in (cache.S_K, cache.S_V, cache.R_K, cache.R_V)]


def check_prefill(out, cache, w, pt, X, Q, rows, starts, window, sinks, dtype, tiled, page_size=64, sample=None, N_K=None):
    adt = I.act_dtype(dtype)
    f = lambda a: I.to_f64(a, adt)
    pools = cache_f64(cache, dtype)
    got, q, cu = host(out, adt), f(Q), np.concatenate([[0], np.cumsum(rows)])
    d = X.shape[1]
    proj = oracle.grouped.project_grouped(f(X), f(w.W_S_K), f(w.W_S_V), f(w.U_K), f(w.U_V), pools[0].shape[2] if pools[0].ndim == 4 else 1)
    mass = oracle.grouped.project_grouped(np.abs(f(X)), *(np.abs(f(a)) for a in (w.W_S_K, w.W_S_V, w.U_K, w.U_V)),
                                          pools[0].shape[2] if pools[0].ndim == 4 else 1)
    u = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -4, "f32": 2.0 ** -24}[dtype]
    for b, (s, n) in enumerate(zip(starts, rows)):
        for i in (range(n) if sample is None else [k for k in sample if k < n]):
            t = s + i
            # the appended row: half a step of the cache's type (8-bit: or of its smallest step) and the sum's error
            for pool, x, m in zip(pools, proj, mass):
                have = pool[pt[b, t // page_size], t % page_size]
                want = x[cu[b] + i].reshape(have.shape)
                tiny = 2.0 ** -10 * I.FP8_SCALE if dtype == "fp8" else 0.0
                tol = u * np.abs(want) + tiny + (1 + u) * d * 2.0 ** -23 * m[cu[b] + i].reshape(have.shape)
                assert np.all(np.abs(have - want) <= tol), f"row {t} of request {b}"
            ref, bound = reference(q[cu[b] + i], pools, f(w.B_K), f(w.B_V), pt[b], t, page_size, window, sinks, dtype,
                                   N_K=N_K, u_w=2.0 ** -8 if tiled else None)
            check(got[cu[b] + i], ref, bound, f"request {b} position {t}")


@pytest.mark.parametrize("H,d_h,r,dtype", [(16, 128, 48, "bf16"), (4, 128, 64, "bf16"), (3, 128, 8, "bf16"), (2, 128, 40, "bf16"),
                                           (8, 64, 24, "bf16"), (16, 128, 48, "fp8"), (4, 32, 8, "f32")])
@pytest.mark.parametrize("window,sinks", [(50, 5), (130, 0)])
def test_prefill_shapes(H, d_h, r, dtype, window, sinks):
    rows, starts = [33, 1, 150], [70, 300, 0]
    args = prefill_inputs(rows, starts, 96, H, d_h, r, dtype, window, sinks, seed=H)
    w, pt, cache, X, Q = args
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(w, pt, cache, X, Q, rows, starts, window, sinks, I.act_dtype(dtype), status=status)
    tiled = dtype == "bf16" and d_h == 128
    check_prefill(out, cache, w, pt, X, Q, rows, starts, window, sinks, dtype, tiled)
    assert int(status.item()) == 0


@pytest.mark.parametrize("window", [1, 63, 64, 65, 127, 128, 129, 200, 4000, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 64, 130, 300, 2 ** 31 - 1])
def test_prefill_window_edges(window, sinks):
    """Window and sinks around the 64-row slices and 128-row tiles of keys and queries; unseen rows hold NaN,
    unseen pages a foreign id."""
    rows, starts = [130, 2, 129, 260], [0, 513, 390, 127]
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, 2, 128, 16, "bf16", window, sinks, seed=5, unseen=10 ** 6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(w, pt, cache, X, Q, rows, starts, window, sinks, "bf16", status=status)
    check_prefill(out, cache, w, pt, X, Q, rows, starts, window, sinks, "bf16", True,
                  sample=[0, 1, 2, 62, 63, 64, 65, 126, 127, 128, 129, 191, 192, 255, 256, 259])
    assert int(status.item()) == 0


@pytest.mark.parametrize("page_size", [16, 64, 128, 192])
def test_prefill_page_sizes(page_size):
    rows, starts = [100, 140], [210, 0]
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, 2, 128, 24, "bf16", 90, 7, seed=page_size, page_size=page_size)
    out = run_prefill(w, pt, cache, X, Q, rows, starts, 90, 7, "bf16")
    check_prefill(out, cache, w, pt, X, Q, rows, starts, 90, 7, "bf16", page_size % 64 == 0, page_size=page_size)


def test_prefill_groups_and_norms():
    rows, starts = [40, 20], [0, 90]
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, 4, 64, 8, "bf16", 30, 3, seed=3, groups=2)
    out = run_prefill(w, pt, cache, X, Q, rows, starts, 30, 3, "bf16")
    check_prefill(out, cache, w, pt, X, Q, rows, starts, 30, 3, "bf16", False)
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, 16, 128, 48, "bf16", 30, 3, seed=4)
    cache.N_K = torch.rand(*cache.R_K.shape[:3], device="cuda").add_(0.5).to(torch.bfloat16)
    cache.norm_eps = 1e-6
    out = run_prefill(w, pt, cache, X, Q, rows, starts, 30, 3, "bf16")
    check_prefill(out, cache, w, pt, X, Q, rows, starts, 30, 3, "bf16", False, N_K=host(cache.N_K, "bf16"))


def test_prefill_one_row_over_a_long_window():
    """A single row per request through the per-row path, on an 8-bit cache and on one with key norms."""
    for dtype in ("fp8", "bf16"):
        w, pt, cache, X, Q = prefill_inputs([1], [5000], 64, 16, 128, 48, dtype, 4500, 3, seed=11)
        N = None
        if dtype == "bf16":
            cache.N_K = torch.rand(*cache.R_K.shape[:3], device="cuda").add_(0.5).to(torch.bfloat16)
            cache.norm_eps = 1e-6
        out = run_prefill(w, pt, cache, X, Q, [1], [5000], 4500, 3, "bf16")
        N = host(cache.N_K, "bf16") if dtype == "bf16" else None
        check_prefill(out, cache, w, pt, X, Q, [1], [5000], 4500, 3, dtype, False, N_K=N)


def test_prefill_empty_requests_and_no_rows():
    rows, starts = [0, 30, 0, 5], [10, 0, 0, 64]
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, 2, 128, 16, "bf16", 20, 2, seed=6)
    out = run_prefill(w, pt, cache, X, Q, rows, starts, 20, 2, "bf16")
    check_prefill(out, cache, w, pt, X, Q, rows, starts, 20, 2, "bf16", True)
    import rank_kv_attention_gb300 as L
    z = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    o = L.prefill_window(z(0, 64), z(0, 2, 128), dev(np.zeros(2), "i32"), dev(np.zeros(1), "i32"), 1, dev(w.W_S_K, "bf16"),
                         dev(w.W_S_V, "bf16"), dev(w.U_K, "bf16"), dev(w.U_V, "bf16"), dev(w.B_K, "bf16"), dev(w.B_V, "bf16"),
                         cache, dev(pt[:1], "i32"), 5)
    assert o.shape == (0, 2, 128)


@pytest.mark.parametrize("n", [20, 130, 300])
def test_prefill_chunks_back_to_back(n):
    """Chunks of two prompts enqueued without a pause (each one's history is what the one before appends), eagerly and
    from a graph, give what the same chunks give one at a time."""
    from rank_kv_attention_gb300.api import PagedCache
    window, sinks, chunks, d = 150, 10, 5, 2048
    rows, ends = [n, n - 7], [chunks * n, chunks * (n - 7)]
    w, pt, cache, X, Q = prefill_inputs(ends, [0, 0], d, 16, 128, 48, "bf16", 10 ** 6, 0, seed=n)
    ws = [dev(a, "bf16") for a in (w.W_S_K, w.W_S_V, w.U_K, w.U_V, w.B_K, w.B_V)]
    Xd, Qd, table = dev(X, "bf16"), dev(Q, "bf16"), dev(pt, "i32")
    cu = dev(np.cumsum([0] + rows), "i32")
    take = [torch.cat([torch.arange(b * ends[0] + k * m, b * ends[0] + (k + 1) * m) for b, m in enumerate(rows)]).cuda()
            for k in range(chunks)]
    parts = [(Xd[i].contiguous(), Qd[i].contiguous(), dev(np.array([k * m for m in rows]), "i32")) for k, i in enumerate(take)]

    def run(c, pause):
        import rank_kv_attention_gb300 as L
        outs = []
        for x, q, start in parts:
            outs.append(L.prefill_window(x, q, cu, start, max(ends), *ws, c, table, window, sinks))
            if pause:
                torch.cuda.synchronize()
        return torch.cat(outs)

    fresh = lambda: PagedCache(*[p.clone() for p in (cache.S_K, cache.S_V, cache.R_K, cache.R_V)])
    want = run(fresh(), True)
    assert torch.isfinite(want.float()).all()
    for _ in range(5):
        assert torch.equal(run(fresh(), False), want)
    c, g = fresh(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(c, False)
    for _ in range(3):
        for p, q in zip((c.S_K, c.S_V, c.R_K, c.R_V), (cache.S_K, cache.S_V, cache.R_K, cache.R_V)):
            p.copy_(q)
        g.replay()
        assert torch.equal(got, want)


@pytest.mark.parametrize("n", [40, 100, 700])
def test_prefill_rows_of_no_request_are_flagged(n):
    """Rows past cu_rows[B] and rows past the page table are skipped and flagged, whichever append runs."""
    import rank_kv_attention_gb300 as L
    rows, starts = [n, n], [0, 64]
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, 2, 128, 16, "bf16", 50, 2, seed=n)
    want = run_prefill(w, pt, cache, X, Q, rows, starts, 50, 2, "bf16")
    call = lambda cu, start, status: L.prefill_window(
        dev(X, "bf16"), dev(Q, "bf16"), dev(np.array(cu), "i32"), dev(np.array(start), "i32"), n + 64, dev(w.W_S_K, "bf16"),
        dev(w.W_S_V, "bf16"), dev(w.U_K, "bf16"), dev(w.U_V, "bf16"), dev(w.B_K, "bf16"), dev(w.B_V, "bf16"), cache,
        dev(pt, "i32"), 50, 2, status=status)
    for cu, start in (((0, n, n + n // 2), (0, 64)), ((0, n, 2 * n), (0, pt.shape[1] * 64 - 5))):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = call(cu, start, status)
        assert int(status.item()) & L._abi.LRKV_STATUS_BAD_ROW
        assert torch.equal(got[:n], want[:n])


def test_prefill_bad_page_is_flagged():
    """A page that rows of the window lie on is missing: flagged, the rows that do not need it still match."""
    import rank_kv_attention_gb300 as L
    rows, starts = [64, 64], [256, 256]
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, 2, 128, 16, "bf16", 100, 4, seed=8)
    pt[0, 3] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(w, pt, cache, X, Q, rows, starts, 100, 4, "bf16", status=status)
    assert int(status.item()) == L.LRKV_STATUS_BAD_PAGE
    assert torch.isfinite(out.float()).all()
    f = lambda a: I.to_f64(a, "bf16")
    pools = cache_f64(cache, "bf16")
    for i in (0, 63):
        ref, bound = reference(f(Q)[64 + i], pools, f(w.B_K), f(w.B_V), pt[1], 256 + i, 64, 100, 4, "bf16", u_w=2.0 ** -8)
        check(host(out, "bf16")[64 + i], ref, bound)


# ---------------------------------------------------------------------------
# Page plan
# ---------------------------------------------------------------------------
def live_table(lens, page_size, max_pages, window, sinks, rng, spare):
    """A table that holds the pages of a windowed cache (others -1), the free ids, and the pool's size."""
    table = np.full((len(lens), max_pages), -1, np.int32)
    cells = []
    for b, L in enumerate(lens):
        for p in range(-(-int(L) // page_size)):
            if not window or p * page_size < sinks or (p + 1) * page_size > L - window + 1:
                cells.append((b, p))
    ids = rng.permutation(len(cells) + spare)
    for (b, p), i in zip(cells, ids):
        table[b, p] = i
    return table, [int(i) for i in ids[len(cells):]], len(cells) + spare


def check_plan(plan, table, want, max_rows):
    n = want["cu_rows"][-1]
    assert plan.seq_lens.tolist() == want["seq_lens"]
    assert plan.cu_rows.tolist() == want["cu_rows"]
    for got, key in ((plan.positions, "positions"), (plan.seq_ids, "seq_ids"), (plan.slots, "slots")):
        assert got.tolist() == want[key] + [-1] * (max_rows - n), key
    assert np.array_equal(table.cpu().numpy(), want["page_table"])
    k = int(plan.n_free.item())
    assert k == len(want["free"])
    free = plan.free_pages.tolist()
    assert free[:k] == want["free"] and all(x == -7 for x in free[k:])


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 9), (100, 0), (100, 5), (1, 0), (64, 64), (333, 130)])
@pytest.mark.parametrize("B,page_size,longest,most", [(1, 16, 0, 1), (1, 64, 900, 700), (7, 16, 300, 1), (64, 64, 1500, 1), (65, 32, 700, 300),
                                                      (2500, 16, 90, 20)])
def test_plan(B, page_size, longest, most, window, sinks):
    rng = np.random.default_rng(B + window)
    lens = rng.integers(0, longest + 1, size=B)
    new = rng.integers(0, most + 1, size=B)
    new[rng.random(B) < 0.15] = -1
    new[rng.random(B) < 0.15] = 0
    max_pages = -(-(longest + most) // page_size) + 1
    table, free, num = live_table(lens, page_size, max_pages, window, sinks, rng, 4 + int(np.maximum(new, 0).sum()) // page_size + B)
    max_rows = int(np.maximum(new, 0).sum()) + 6
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = W.page_plan(lens, new, table, free, page_size, num, window, sinks, max_rows)
    plan, pt = plan_on_device(lens, new, table, free, num, page_size, max_rows, window, sinks, status)
    check_plan(plan, pt, want, max_rows)
    assert not want["refused"] and not want["invalid"] and int(status.item()) == 0


@pytest.mark.parametrize("B", [5, 40, 2100])
@pytest.mark.parametrize("short_rows,short_pages", [(0, 3), (11, 0), (9, 2), (10 ** 9, 0)])
def test_plan_refuses_what_does_not_fit(B, short_rows, short_pages):
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(B)
    lens, new = rng.integers(0, 200, size=B), rng.integers(0, 60, size=B)
    new[B // 2] = -1
    lens[0], new[1] = -3, -2                  # and two invalid requests
    ps = 16
    need = sum(-(-(int(a) + int(n)) // ps) - -(-int(a) // ps) for a, n in zip(lens[2:], new[2:]) if n > 0)
    table, free, num = live_table(np.maximum(lens, 0), ps, 17, 64, 4, rng, max(0, need - short_pages))
    max_rows = max(0, int(np.maximum(new[2:], 0).sum()) - short_rows)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = W.page_plan(lens, new, table, free, ps, num, 64, 4, max_rows)
    plan, pt = plan_on_device(lens, new, table, free, num, ps, max_rows, 64, 4, status)
    check_plan(plan, pt, want, max_rows)
    assert want["refused"] and int(status.item()) == (L.LRKV_STATUS_NO_PAGES | L.LRKV_STATUS_BAD_SEQLEN)


def test_plan_bad_ids_become_minus_one():
    import rank_kv_attention_gb300 as L
    table = np.array([[5, 99, -1, -1], [2, -1, -1, -1]], np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan, pt = plan_on_device([20, 16], [-1, 17], table, [0, 1, 77], 8, 16, 20, 0, 0, status)
    # request 1 gains ids 77 (none) and 1; request 0 returns 5 and 99 (none)
    assert pt.cpu().tolist() == [[5, 99, -1, -1], [2, -1, 1, -1]]
    assert plan.free_pages.tolist()[:3] == [0, 5, -1] and int(plan.n_free.item()) == 3
    assert plan.slots.tolist() == [-1] * 16 + [16] + [-1] * 3
    assert int(status.item()) == L.LRKV_STATUS_BAD_PAGE
    # a count of free pages past the pool
    status.zero_()
    free = dev(np.arange(8), "i32")
    p = L.page_plan(dev([3], "i32"), dev([1], "i32"), dev([[0]], "i32"), free, dev([9], "i32"), 16, 1, status=status)
    assert int(p.n_free.item()) == 8 and int(status.item()) == L.LRKV_STATUS_BAD_PAGE


# ---------------------------------------------------------------------------
# All of them as a server would run them
# ---------------------------------------------------------------------------
def far(cache, extra):
    """The same cache at the end of pools that are `extra` pages longer."""
    from rank_kv_attention_gb300.api import PagedCache

    def grow(p):
        q = torch.empty((extra + p.shape[0], *p.shape[1:]), dtype=p.dtype, device="cuda")
        q[extra:].view(torch.uint8).copy_(p.view(torch.uint8))
        return q
    return PagedCache(*[grow(p) for p in (cache.S_K, cache.S_V, cache.R_K, cache.R_V)], cache.scale)


@pytest.mark.parametrize("H,d_h,r,dtype", [(16, 128, 48, "bf16"), (16, 128, 48, "fp8"), (8, 64, 16, "f32")])
def test_offsets_past_32_bits(H, d_h, r, dtype):
    """Pages whose private rows start past 2^31 elements: decode, append and prefill as in a small pool, bit for bit."""
    extra = 2 ** 31 // (64 * H * r) + 1
    d = DevDecode(decode_case([1, 300, 65, 700], H, d_h, r, dtype, seed=H))
    want = run_decode(d, 200, 5)
    d.cache, d.page_table = far(d.cache, extra), d.page_table + extra
    assert torch.equal(run_decode(d, 200, 5), want)
    del d
    rows, starts, adt = [90, 33], [130, 0], I.act_dtype(dtype)
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, H, d_h, r, dtype, 120, 3, seed=2)
    big = far(cache, extra)
    want = run_prefill(w, pt, cache, X, Q, rows, starts, 120, 3, adt)
    got = run_prefill(w, np.where(pt >= 0, pt + extra, pt), big, X, Q, rows, starts, 120, 3, adt)
    assert torch.equal(got, want)
    for p, q in zip((cache.S_K, cache.S_V, cache.R_K, cache.R_V), (big.S_K, big.S_V, big.R_K, big.R_V)):
        assert torch.equal(q[extra:].view(torch.uint8), p.view(torch.uint8))


def test_binding_refuses_sizes_past_32_bits():
    """A size that would wrap into a valid one is refused."""
    import rank_kv_attention_gb300 as L
    d = DevDecode(decode_case([5, 9], 16, 128, 48))
    for window, sinks, longest in ((2 ** 32 + 5, 0, 9), (5, 2 ** 32, 9), (5, 0, 2 ** 32 + 9)):
        with pytest.raises(ValueError):
            L.decode_window(d.q, d.cache, d.B_K, d.B_V, d.seq_lens, d.page_table, longest, window, sinks)
    w, pt, cache, X, Q = prefill_inputs([70], [0], 64, 16, 128, 48, "bf16", 50, 2, seed=1)
    for window, sinks in ((2 ** 32 + 5, 0), (5, 2 ** 32 + 1)):
        with pytest.raises(ValueError):
            run_prefill(w, pt, cache, X, Q, [70], [0], window, sinks, "bf16")
    with pytest.raises(ValueError):
        plan_on_device([3], [1], [[0, 1]], [2], 3, 64, 4, window=2 ** 32 + 64, sinks=0)
    with pytest.raises(ValueError):
        plan_on_device([3], [1], [[0, 1]], [2], 3, 2 ** 32 + 64, 4, window=64, sinks=0)


def test_serving_run_with_a_bounded_pool():
    """Prompts in chunks, then single tokens, requests that end and new ones in their place: plan, prefill and
    decode on a pool that holds only the windows' pages, one graph-captured decode step among them.  Each output
    matches the definition over the rows that were ever written (kept here on the host)."""
    import rank_kv_attention_gb300 as L
    from rank_kv_attention_gb300.api import PagedCache
    H, d_h, r, d, ps, window, sinks, B = 16, 128, 16, 64, 16, 40, 5, 3
    rng = np.random.default_rng(77)
    w = I.make_weights(d, H, d_h, r, "bf16", seed=1)
    per = -(-sinks // ps) + window // ps + 2 + 3      # a request's pages at most: sinks, window, a chunk of 40 rows
    num = B * per
    cache = PagedCache(*[dev(p, "bf16") for p in I.empty_pools(num, ps, H, d_h, r, "bf16")])
    table = torch.full((B, 40), -1, dtype=torch.int32, device="cuda")
    lens = [torch.zeros(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")]
    free = [torch.arange(num, dtype=torch.int32, device="cuda"), torch.empty(num, dtype=torch.int32, device="cuda")]
    n_free = torch.tensor([num], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    W4 = [dev(a, "bf16") for a in (w.W_S_K, w.W_S_V, w.U_K, w.U_V)]
    bases = [dev(w.B_K, "bf16"), dev(w.B_V, "bf16")]
    f = lambda a: I.to_f64(a, "bf16")
    kept = [[] for _ in range(B)]                     # every row of each request, as the cache stored it
    steps = [[40, 33, 0], [40, 7, 20], [40, 1, 1], [1, 1, 40]] + [[1, 1, 1]] * 30 + [[-1, 1, 1], [25, -1, 1], [1, 30, 1]] + [[1, 1, 1]] * 12
    for k, new in enumerate(steps):
        n = sum(max(0, x) for x in new)
        plan = L.page_plan(lens[0], dev(np.array(new), "i32"), table, free[0], n_free, ps, n, free_out=free[1], window=window, sinks=sinks, status=status)
        X = I.f32_to_bf16_bits(rng.standard_normal((n, d)).astype(np.float32))
        Q = I.f32_to_bf16_bits(rng.standard_normal((n, H, d_h)).astype(np.float32))
        if new == [1, 1, 1]:
            L.append(dev(X, "bf16"), plan.positions, plan.seq_ids, *W4, cache, table, status=status)
            out = L.decode_window(dev(Q, "bf16"), cache, *bases, plan.seq_lens, table, 640, window, sinks, status=status)
        else:
            out = L.prefill_window(dev(X, "bf16"), dev(Q, "bf16"), plan.cu_rows, lens[0], 640, *W4, *bases, cache, table, window, sinks, status=status)
        assert int(status.item()) == 0, k
        flat = [p.reshape(num * ps, *p.shape[2:]) for p in cache_f64(cache, "bf16")]
        got, slots, ids = host(out, "bf16"), plan.slots.tolist(), plan.seq_ids.tolist()
        for b in range(B):
            if new[b] == -1:
                kept[b] = []
        for i in range(n):
            kept[ids[i]].append([x[slots[i]] for x in flat])
        at = [len(x) - max(0, m) for x, m in zip(kept, new)]
        for i in range(n):
            b = ids[i]
            rows = [np.stack([x[c] for x in kept[b]])[:, None] for c in range(4)]  # one row per page
            ref, bound = reference(f(Q)[i], rows, f(w.B_K), f(w.B_V), range(len(kept[b])), at[b], 1, window, sinks, "bf16", u_w=2.0 ** -8)
            check(got[i], ref, bound, f"step {k} request {b} position {at[b]}")
            at[b] += 1
        lens[0] = plan.seq_lens
        free.reverse()
        n_free = plan.n_free
        live = [int(x) for b in range(B) for p, x in enumerate(table[b].tolist())
                if p * ps < len(kept[b]) and (p * ps < sinks or (p + 1) * ps > len(kept[b]) - window + 1)]
        spare = free[0].tolist()[:int(n_free.item())]
        assert sorted(live + spare) == list(range(num)), f"step {k}: a page is lost or held twice"
    assert max(len(x) for x in kept) > 70


def test_serving_step_in_a_graph():
    """Plan, append and decode of single tokens captured once and replayed, against the same calls made one by one."""
    import rank_kv_attention_gb300 as L
    from rank_kv_attention_gb300.api import PagedCache
    H, d_h, r, d, ps, window, sinks, B = 16, 128, 48, 64, 16, 48, 4, 5
    num, gen = B * 8 + 6, torch.Generator(device="cuda").manual_seed(3)
    w = I.make_weights(d, H, d_h, r, "bf16", seed=2)
    W4 = [dev(a, "bf16") for a in (w.W_S_K, w.W_S_V, w.U_K, w.U_V)]
    bases = [dev(w.B_K, "bf16"), dev(w.B_V, "bf16")]
    steps, ends = 70, {20: 1, 41: 3, 42: 0}

    def start():
        return dict(lens=torch.zeros(B, dtype=torch.int32, device="cuda"), new=torch.ones(B, dtype=torch.int32, device="cuda"),
                    table=torch.full((B, 64), -1, dtype=torch.int32, device="cuda"), free=torch.arange(num, dtype=torch.int32, device="cuda"),
                    out_free=torch.empty(num, dtype=torch.int32, device="cuda"), n=torch.tensor([num], dtype=torch.int32, device="cuda"),
                    X=torch.empty(B, d, dtype=torch.bfloat16, device="cuda"), q=torch.empty(B, H, d_h, dtype=torch.bfloat16, device="cuda"),
                    cache=PagedCache(*[dev(p, "bf16") for p in I.empty_pools(num, ps, H, d_h, r, "bf16")]))

    def step(s):
        p = L.page_plan(s["lens"], s["new"], s["table"], s["free"], s["n"], ps, B, free_out=s["out_free"], window=window, sinks=sinks)
        L.append(s["X"], p.positions, p.seq_ids, *W4, s["cache"], s["table"])
        out = L.decode_window(s["q"], s["cache"], *bases, p.seq_lens, s["table"], 1024, window, sinks)
        s["lens"].copy_(p.seq_lens)
        s["n"].copy_(p.n_free)
        s["free"].copy_(s["out_free"])
        return out

    a, b = start(), start()
    step(a)                                             # (a step before the capture; undone)
    a = start()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step(a)
    a.update({k: a[k] for k in a})
    for k in ("lens", "new", "table", "free", "n"):
        a[k].copy_(start()[k])
    for k in range(steps):
        x, q = (torch.randn(t.shape, device="cuda", generator=gen).to(torch.bfloat16) for t in (a["X"], a["q"]))
        for s in (a, b):
            s["X"].copy_(x), s["q"].copy_(q), s["new"].fill_(1)
            if k in ends:
                s["new"][ends[k]] = -1
        g.replay()
        want = step(b)
        live = b["new"] > 0
        assert torch.equal(captured[live], want[live]), k
        assert torch.equal(a["lens"], b["lens"]) and torch.equal(a["table"], b["table"]) and torch.equal(a["n"], b["n"]), k
    assert int(b["lens"].max()) == steps
