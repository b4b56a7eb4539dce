"""The windowed operators in the calls that a server makes around the ordinary
ones.  References and bounds are those of window_util."""
import ctypes

import numpy as np
import pytest
import torch

import lrkv_inputs as I
from gpu_util import DevDecode, dev, host
from test_window_gpu import check_prefill, decode_case, prefill_inputs, run_decode, run_prefill
from window_util import check, decode_reference

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# One workspace for a batch that shrinks
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H,r,dtype", [(16, 48, torch.bfloat16), (32, 32, torch.bfloat16), (16, 64, torch.float8_e4m3fn)])
def test_workspace_bytes_never_fall_as_a_call_grows(H, r, dtype):
    import rank_kv_attention_gb300 as L
    need = lambda B, longest, window, sinks: L.decode_window_workspace_bytes(B, H, 128, r, longest, window, sinks, dtype)
    grid = [(B, n, w, s) for B in (1, 2, 3, 4, 8, 12, 16, 24, 48, 64, 200) for n in (1, 40, 700, 2100, 60000)
            for w in (1, 30, 600, 2048, 50000) for s in (0, 4, 300)]
    sizes = {c: need(*c) for c in grid}
    for a, x in sizes.items():
        for b, y in sizes.items():
            if all(p <= q for p, q in zip(a, b)):
                assert x <= y, (a, x, b, y)


@pytest.mark.parametrize("H,r,dtype", [(16, 48, "bf16"), (16, 64, "fp8")])
def test_a_workspace_for_the_largest_batch_serves_the_smaller_ones(H, r, dtype):
    import rank_kv_attention_gb300 as L
    lens = [2100, 5, 2099, 700] * 6
    case = decode_case(lens, H, 128, r, dtype, seed=4)
    d = DevDecode(case)
    # the largest of each size: 24 requests need no more states than 4 or 16 do
    ws = L.workspace(L.decode_window_workspace_bytes(24, H, 128, r, 2100, 2048, 4, d.cache.dtype))
    for window, sinks in ((2048, 4), (300, 0)):
        ref, bound = decode_reference(case, window, sinks)
        for B in (24, 16, 12, 8, 5, 4, 2, 1):
            ws.fill_(0xFF)
            longest = max(lens[:B])
            got = L.decode_window(d.q[:B], d.cache, d.B_K, d.B_V, d.seq_lens[:B], d.page_table[:B], longest, window, sinks, ws=ws)
            check(host(got, case.act_dtype), ref[:B], bound[:B], f"B={B} window={window}")


# ---------------------------------------------------------------------------
# Streams of the caller's
# ---------------------------------------------------------------------------
def stream_calls(kind):
    """A call on fixed inputs that gives the same outputs each time: call(stream=...) -> tensors."""
    import rank_kv_attention_gb300 as L
    if kind.startswith("decode"):
        lens, window = ([9000], 8000) if kind == "decode split" else ([300, 5, 2000, 1100], 1024)
        d = DevDecode(decode_case(lens, 16, 128, 48, seed=1))
        return lambda **kw: [run_decode(d, window, 4, **kw)]
    if kind.startswith("prefill"):
        dtype, rows, starts = ("fp8" if kind == "prefill per row" else "bf16"), [100, 30], [70, 200]
        w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, 16, 128, 48, dtype, 90, 3, seed=6)
        args = [dev(a, "bf16") for a in (X, Q)], [dev(np.array(a), "i32") for a in ([0, 100, 130], starts)]
        weights = [dev(a, "bf16") for a in (w.W_S_K, w.W_S_V, w.U_K, w.U_V, w.B_K, w.B_V)]
        table = dev(pt, "i32")
        return lambda **kw: [L.prefill_window(*args[0], *args[1], 230, *weights, cache, table, 90, 3, **kw)]
    lens, new = [dev(np.array(a), "i32") for a in ([500, 64, 7], [300, -1, 1])]
    table = dev(np.arange(3 * 16).reshape(3, 16), "i32")
    free, n_free = torch.arange(48, 100, dtype=torch.int32, device="cuda"), dev(np.array([52]), "i32")
    pages = torch.cat([free, torch.full((48,), -1, dtype=torch.int32, device="cuda")])

    def call(**kw):
        p = L.page_plan(lens, new, table, pages, n_free, 64, 400, window=200, sinks=4, **kw)
        return [p.seq_lens, p.cu_rows, p.positions, p.seq_ids, p.slots, p.n_free, p.free_pages[:48]]
    return call


@pytest.mark.parametrize("kind", ["decode", "decode split", "prefill", "prefill per row", "plan"])
def test_outputs_on_another_stream(kind):
    """A call on a stream of its own while memory just freed on the current stream has work queued on it, and outputs read
    on the current stream and freed before that read has run: neither disturbs a result."""
    call, side, here = stream_calls(kind), torch.cuda.Stream(), torch.cuda.current_stream()
    want = [t.clone() for t in call()]
    same = lambda got: all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    for _ in range(3):
        freed = [torch.empty_like(t) for t in want] + [torch.empty(1 << k, dtype=torch.uint8, device="cuda") for k in range(9, 24)]
        torch.cuda._sleep(50_000_000)
        for t in freed:
            t.view(torch.uint8).fill_(0xEE)
        del freed, t
        got = call(stream=side)
        torch.cuda.synchronize()
        assert same(got)
        got = call(stream=side)
        here.wait_stream(side)
        torch.cuda._sleep(50_000_000)
        kept = [t.clone() for t in got]
        shapes = [(t.shape, t.dtype) for t in got]
        del got
        with torch.cuda.stream(side):
            over = [torch.empty(s, dtype=d, device="cuda").view(torch.uint8).fill_(0xEE) for s, d in shapes for _ in range(3)]
        torch.cuda.synchronize()
        assert same(kept)
        del kept, over


@pytest.mark.parametrize("kind", ["prefill", "prefill per row", "plan", "decode split"])
def test_calls_at_once_on_several_streams(kind):
    calls = [stream_calls(kind) for _ in range(4)]
    want = [t.clone() for t in calls[0]()]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = []
        for call, s in zip(calls, sides):
            with torch.cuda.stream(s):
                got.append(call())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


# ---------------------------------------------------------------------------
# The benchmark's profile
# ---------------------------------------------------------------------------
def test_profile_counts_a_split_call_once():
    """A call that first asks for a workspace is one launch of the attention kernel, not two."""
    import rank_kv_attention_gb300 as L
    lib = L.lib()

    def launches():
        ms, n = ctypes.c_double(), ctypes.c_int32()
        assert lib.lrkv_profile_read(0, ctypes.byref(ms), ctypes.byref(n)) == L.LRKV_OK
        return n.value, ms.value

    d = DevDecode(decode_case([9000], 16, 128, 48))
    desc = d.cache.desc()
    out = torch.empty_like(d.q)
    bare = lambda: lib.lrkv_decode_window(
        d.q.data_ptr(), ctypes.byref(desc), d.B_K.data_ptr(), d.B_V.data_ptr(), d.seq_lens.data_ptr(), d.page_table.data_ptr(),
        1, d.page_table.shape[1], 9000, 8000, 4, out.data_ptr(), None, 0, None, torch.cuda.current_stream().cuda_stream)
    assert bare() == L.LRKV_E_WORKSPACE
    assert lib.lrkv_profile_enable(1) == L.LRKV_OK
    try:
        assert bare() == L.LRKV_E_WORKSPACE and launches() == (0, 0.0)
        run_decode(d, 8000, 4)
        n, ms = launches()
        assert n == 1 and ms > 0
    finally:
        lib.lrkv_profile_enable(0)


# ---------------------------------------------------------------------------
# Contexts far longer than the window
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H,d_h,r,dtype,n", [(2, 128, 16, "bf16", 8300), (2, 64, 8, "fp8", 8300), (2, 32, 4, "f32", 8300),
                                             (2, 128, 16, "bf16", 61)])
def test_prefill_on_a_long_context(H, d_h, r, dtype, n):
    """New rows at positions about 2^17: rows times context pass 2^30 where n is 8300, rows times visible rows stay small.
    All but the last pages of the table are -1."""
    start, window, sinks = 131000, 90, 3
    w, pt, cache, X, Q = prefill_inputs([n], [start], 64, H, d_h, r, dtype, window, sinks, seed=n)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(w, pt, cache, X, Q, [n], [start], window, sinks, I.act_dtype(dtype), status=status)
    tiled = dtype == "bf16" and d_h == 128
    check_prefill(out, cache, w, pt, X, Q, [n], [start], window, sinks, dtype, tiled,
                  sample=[0, 1, 60, 63, 64, 88, 89, 90, 127, 128, 4000, 8191, 8192, 8299])
    assert int(status.item()) == 0


# ---------------------------------------------------------------------------
# A prefix that requests of one call share
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,starts,d", [([128, 40, 30], [0, 128, 64], 2048), ([64, 100, 400], [256, 320, 320], 2048),
                                           ([30, 20, 1], [34, 64, 64], 2048)])
def test_prefill_shares_a_prefix_within_the_call(rows, starts, d):
    """The histories of two requests are whole pages of another's new rows, in calls so small that the append leaves SMs
    idle.  The cache holds NaN until the append has written it."""
    window, sinks, ps = 200, 5, 64
    w, pt, cache, X, Q = prefill_inputs(rows, starts, d, 16, 128, 48, "bf16", 10 ** 6, 0, seed=len(rows) + rows[0])
    for b in (1, 2):
        pt[b, :starts[b] // ps] = pt[0, :starts[b] // ps]
    pools = (cache.S_K, cache.S_V, cache.R_K, cache.R_V)
    before = [p.clone() for p in pools]
    for _ in range(5):
        for p, x in zip(pools, before):
            p.copy_(x)
        out = run_prefill(w, pt, cache, X, Q, rows, starts, window, sinks, "bf16")
        check_prefill(out, cache, w, pt, X, Q, rows, starts, window, sinks, "bf16", True, sample=[0, 1, 19, 29, 39, 63, 99, 399])


# ---------------------------------------------------------------------------
# NaN queries
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 40, 130, 300])
def test_prefill_nan_queries_reach_the_output(n):
    """A query with a NaN has no answer: its row is NaN in the heads it touches, as in the single-token form; other rows
    and heads are unchanged."""
    import rank_kv_attention_gb300 as L
    rows, starts, window, sinks, H = [n, 3], [200, 0], 90, 4, 2
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, H, 128, 16, "bf16", window, sinks, seed=n)
    clean = run_prefill(w, pt, cache, X, Q, rows, starts, window, sinks, "bf16")
    hit = sorted({0, n // 2, n - 1, n + 1})
    for i in hit:
        Q[i, 1, 7] = I.BF16_NAN_BITS
    got = run_prefill(w, pt, cache, X, Q, rows, starts, window, sinks, "bf16")
    want = clean.clone()
    want[hit, 1] = float("nan")
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    # the same query as a single token
    last = torch.tensor([starts[0] + n], dtype=torch.int32, device="cuda")
    one = L.decode_window(dev(Q[n - 1:n], "bf16"), cache, dev(w.B_K, "bf16"), dev(w.B_V, "bf16"), last, dev(pt[:1], "i32"),
                          int(last), window, sinks)
    assert torch.equal(torch.isnan(one[0]), torch.isnan(got[n - 1]))


# ---------------------------------------------------------------------------
# Many requests
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H,d_h,r,dtype", [(16, 128, 32, "bf16"), (16, 128, 32, "fp8"), (3, 32, 8, "f32")])
def test_decode_of_many_requests(H, d_h, r, dtype):
    """Far more requests than the GPU holds clusters, some empty, some of one row."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 150, size=1100)
    lens[::7] = 1
    window, sinks = 70, 3
    case = decode_case(lens, H, d_h, r, dtype, seed=2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = host(run_decode(DevDecode(case), window, sinks, status=status), case.act_dtype)
    check(got, *decode_reference(case, window, sinks))
    import rank_kv_attention_gb300 as L
    assert int(status.item()) == L.LRKV_STATUS_BAD_SEQLEN  # (the empty ones)


@pytest.mark.parametrize("dtype,most", [("bf16", 300), ("bf16", 1300), ("fp8", 90)])
def test_prefill_of_a_mixed_step(dtype, most):
    """One prompt's chunk beside single tokens, each request on a history of its own."""
    rng = np.random.default_rng(most)
    rows, starts = [1] * 60, [int(x) for x in rng.integers(0, 500, size=60)]
    rows[23], rows[41] = most, 5
    window, sinks = 130, 4
    w, pt, cache, X, Q = prefill_inputs(rows, starts, 64, 4, 128, 16, dtype, window, sinks, seed=most)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_prefill(w, pt, cache, X, Q, rows, starts, window, sinks, "bf16", status=status)
    check_prefill(out, cache, w, pt, X, Q, rows, starts, window, sinks, dtype, dtype == "bf16",
                  sample=[0, 1, 4, 63, 64, 127, 128, 129, 255, 299, 1023, 1299])
    assert int(status.item()) == 0
