"""The block-scaled cache on the GPU against its float64 definitions (bounds: scaled_util.py)."""
import numpy as np
import pytest
import torch

import lrkv_inputs as I
import oracle
import oracle.scaled as S
from gpu_util import dev, host, host_bits
from scaled_util import (POOLS, assert_same, bf16, check, random_cache, reference, table_of, to_device, to_host)

pytestmark = pytest.mark.gpu
BAD_PAGE, BAD_SEQLEN, BAD_ROW = 1, 2, 4


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def shape_of(k, H, d_h, r, G):
    return (G, d_h) if k[0] == "S" else (H, r)


def values(rng, n, H, d_h, r, G, dtype):
    """name -> (device rows, their float64 values): heads and rows differ in magnitude, some rows are zero."""
    out = {}
    for k in POOLS:
        heads, width = shape_of(k, H, d_h, r, G)
        x = rng.standard_normal((n, heads, width)) * np.exp(2 * rng.standard_normal((n, heads, 1)))
        x[rng.random(n) < 0.1] = 0
        if dtype == "bf16":
            bits = I.f32_to_bf16_bits(x.astype(np.float32))
            out[k] = dev(bits, "bf16"), I.bf16_bits_to_f64(bits)
        else:
            out[k] = dev(x, "f32"), x.astype(np.float32).astype(np.float64)
    return out


def write(dc, rows, cu, start, table, **kw):
    import rank_kv_attention_gb300 as L
    L.write_scaled(*[rows[k][0].reshape(rows[k][0].shape[0], -1) for k in POOLS], dev(np.asarray(cu), "i32"),
                   dev(np.asarray(start), "i32"), dc, dev(table, "i32"), **kw)


def oracle_write(cache, rows, cu, start, table):
    S.write(cache, {k: rows[k][1] for k in POOLS}, cu, start, table)


LAYOUTS = [(16, 128, 48, 1, 64, 64), (16, 128, 56, 1, 64, 16), (4, 64, 16, 1, 32, 32), (2, 16, 8, 1, 16, 16),
           (6, 32, 40, 2, 48, 16), (3, 256, 256, 1, 48, 48), (8, 128, 64, 4, 128, 64), (32, 128, 32, 1, 128, 128),
           (1, 16, 16, 1, 1024, 1024), (20, 128, 8, 1, 64, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,d_h,r,G,ps,block", LAYOUTS)
def test_write_and_read(H, d_h, r, G, ps, block, dtype):
    """Chunks of several calls, from inside blocks, of no, one and many rows: codes and exponents to the bit, every other
    byte as it was; read back exactly in both types."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(H * 1000 + r)
    chunks = [[3, 0, 1, 2 * block + 5], [block, 1, 0, 1], [1, ps + 3, block - 1, 7]]
    lens = np.sum(chunks, 0)
    pages = int(sum(-(-n // ps) for n in lens)) + 2
    table = table_of(rng, lens, ps, pages)
    cache = random_cache(rng, pages, ps, H, d_h, r, block, G)
    dc, at = to_device(cache), np.zeros(4, np.int64)
    for rows_of in chunks:
        cu = np.concatenate([[0], np.cumsum(rows_of)])
        x = values(rng, int(cu[-1]), H, d_h, r, G, dtype)
        st = status()
        write(dc, x, cu, at, table, status=st)
        oracle_write(cache, x, cu, at, table)
        assert int(st) == 0
        assert_same(to_host(dc, cache), cache)
        at += rows_of
    cu = np.concatenate([[0], np.cumsum(lens)])
    for dt, kind in ((torch.bfloat16, "bf16"), (torch.float32, "f32")):
        got = L.read_scaled(dev(cu, "i32"), dev(np.zeros(4), "i32"), int(cu[-1]), dc, dev(table, "i32"), dtype=dt)
        for k, t in zip(POOLS, got):
            want = S.read(cache, k, cu, [0] * 4, table, np.zeros((int(cu[-1]),) + shape_of(k, H, d_h, r, G)))
            assert np.array_equal(host(t, kind).reshape(want.shape), want), k


def test_write_the_whole_range_of_magnitudes():
    """fp32 values from subnormals to the largest, infinities, NaN, negative zero; exponents at both ends."""
    rng = np.random.default_rng(5)
    H, d_h, r, ps = 4, 16, 8, 16
    cache = random_cache(rng, 40, ps, H, d_h, r, 16)
    dc, n = to_device(cache), 40 * ps
    rows = {}
    for k in POOLS:
        heads, width = shape_of(k, H, d_h, r, 1)
        e = np.repeat(rng.integers(-149, 128, (40, heads, 1)), ps, 0)
        with np.errstate(over="ignore"):
            x = (rng.standard_normal((n, heads, width)) * 2.0 ** e).astype(np.float32)
        x[rng.random(x.shape) < 0.02] = np.inf
        x[rng.random(x.shape) < 0.02] = -np.inf
        x[rng.random(x.shape) < 0.02] = np.nan
        x[rng.random(x.shape) < 0.02] = -0.0
        x[16:32] = np.nan                                        # a block without a finite value
        x[32:48] = 3.4e38                                        # beyond 448 * 2^119: saturates
        rows[k] = dev(x, "f32"), x.astype(np.float64)
    table = rng.permutation(40).astype(np.int32)[None]
    write(dc, rows, [0, n], [0], table)
    oracle_write(cache, rows, [0, n], [0], table)
    assert_same(to_host(dc, cache), cache)


@pytest.mark.parametrize("byte", [0, 9, 10, 246, 247, 255])
def test_scale_bytes_outside_the_range(byte):
    """They read as the nearest in it, and count so where a block grows."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(byte)
    cache = random_cache(rng, 2, 16, 2, 16, 8, 16)
    for k in POOLS:
        cache.exps[k][:] = byte
    dc, table = to_device(cache), np.array([[1, 0]], np.int32)
    got = L.read_scaled(dev(np.array([0, 20]), "i32"), dev(np.zeros(1), "i32"), 20, dc, dev(table, "i32"), dtype=torch.float32)
    for k, t in zip(POOLS, got):
        want = S.read(cache, k, [0, 20], [0], table, np.zeros((20,) + shape_of(k, 2, 16, 8, 1)))
        assert np.array_equal(host(t, "f32").reshape(want.shape), want)
    x = values(rng, 3, 2, 16, 8, 1, "f32")
    write(dc, x, [0, 3], [5], table)
    oracle_write(cache, x, [0, 3], [5], table)
    assert_same(to_host(dc, cache), cache)


def test_rows_that_have_no_place():
    """Negative positions, rows past the table, pages outside the pool, rows of no request: skipped and flagged (rows of no
    request are not), everything else written; reading leaves those rows of the output alone."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(6)
    H, d_h, r, ps, block = 4, 32, 8, 32, 16
    cache = random_cache(rng, 9, ps, H, d_h, r, block)
    table = np.array([[0, 1, -1], [2, 3, 4], [5, 9, 6], [7, 8, -5]], np.int32)
    cu, start = np.array([3, 23, 50, 110, 140]), np.array([-7, 80, 10, 30])   # rows 0-2 and 140-144 belong to nobody
    x = values(rng, 145, H, d_h, r, 1, "bf16")
    dc, st = to_device(cache), status()
    write(dc, x, cu, start, table, status=st)
    oracle_write(cache, x, cu, start, table)
    assert_same(to_host(dc, cache), cache)
    assert int(st) == BAD_ROW | BAD_PAGE
    out, st = L.ScaledRows(*[torch.full((145,) + shape_of(k, H, d_h, r, 1), 7.0, device="cuda") for k in POOLS]), status()
    L.read_scaled(dev(cu, "i32"), dev(start, "i32"), 145, dc, dev(table, "i32"), out=out, status=st)
    for k, t in zip(POOLS, out):
        want = S.read(cache, k, cu, start, table, np.full((145,) + shape_of(k, H, d_h, r, 1), 7.0))
        assert np.array_equal(host(t, "f32"), want)
    assert int(st) == BAD_ROW | BAD_PAGE
    # positions whose distance to the table does not fit in 32 bits
    st = status()
    write(dc, values(rng, 8, H, d_h, r, 1, "bf16"), [0, 4, 8], [2 ** 31 - 2, -2 ** 31], table[:2], status=st)
    assert int(st) == BAD_ROW
    assert_same(to_host(dc, cache), cache)


def test_requests_without_order_do_no_harm():
    """cu_rows that fall or run past n: no row is read or written outside the call's."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(7)
    H, d_h, r, ps = 4, 32, 8, 32
    cache = random_cache(rng, 12, ps, H, d_h, r, 16)
    dc, table = to_device(cache), np.arange(12, dtype=np.int32).reshape(4, 3)
    x = values(rng, 30, H, d_h, r, 1, "bf16")
    for cu in ([0, 20, 10, 25, 90], [-50, 4, 3, 2, 1], [40, 50, 60, 70, 80], [2 ** 31 - 1, -2 ** 31, 7, 8, 2 ** 31 - 1]):
        write(dc, x, cu, [0, 0, 0, 0], table)
        L.read_scaled(dev(np.array(cu), "i32"), dev(np.zeros(4), "i32"), 30, dc, dev(table, "i32"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("B", [1, 31, 32, 33, 1100])
def test_write_finds_its_requests(B):
    """Many requests, most with one row, some with none or several."""
    rng = np.random.default_rng(B)
    H, d_h, r, ps, block = 2, 16, 8, 32, 16
    n_of = rng.choice([0, 1, 1, 1, 2, 40], B)
    n_of[-1] = 1
    start = rng.integers(0, 40, B)
    table = table_of(rng, n_of + start, ps, int(sum(-(-n // ps) for n in n_of + start)), width=3)
    cache = random_cache(rng, int(table.max()) + 1, ps, H, d_h, r, block)
    cu = np.concatenate([[0], np.cumsum(n_of)])
    x = values(rng, int(cu[-1]), H, d_h, r, 1, "bf16")
    dc, st = to_device(cache), status()
    write(dc, x, cu, start, table, status=st)
    oracle_write(cache, x, cu, start, table)
    assert int(st) == 0
    assert_same(to_host(dc, cache), cache)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_and_read_rows_with_a_stride(dtype):
    """The slices of one projection's output; the columns between them stay."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(8)
    H, d_h, r, ps, n = 4, 32, 24, 32, 50
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    y = torch.randn(n, 2 * d_h + 2 * H * r + 48, device="cuda").to(dt)
    edges = [0, d_h, d_h + 16, 2 * d_h + 16, 2 * d_h + 32, 2 * d_h + 32 + H * r, 2 * d_h + 48 + H * r]
    cut = lambda t: [t[:, :d_h], t[:, edges[2]:edges[3]], t[:, edges[4]:edges[5]].unflatten(1, (H, r)),  # noqa: E731
                     t[:, edges[6]:].unflatten(1, (H, r))]
    cache = random_cache(rng, 4, ps, H, d_h, r, 16)
    dc, table, cu = to_device(cache), np.array([[2, 0], [3, 1]], np.int32), [0, 20, 50]
    dcu, dst, dtab = dev(np.array(cu), "i32"), dev(np.array([0, 1]), "i32"), dev(table, "i32")
    L.write_scaled(*cut(y), dcu, dst, dc, dtab)
    S.write(cache, {k: host(t.contiguous(), dtype).reshape((n,) + shape_of(k, H, d_h, r, 1)) for k, t in zip(POOLS, cut(y))},
            cu, [0, 1], table)
    assert_same(to_host(dc, cache), cache)
    z = y.clone()
    L.read_scaled(dcu, dst, n, dc, dtab, out=cut(z))
    for k, t in zip(POOLS, cut(z)):
        want = S.read(cache, k, cu, [0, 1], table, np.zeros((n,) + shape_of(k, H, d_h, r, 1)))
        assert np.array_equal(host(t.contiguous(), dtype).reshape(want.shape), want)
    for t in cut(z):
        t.zero_()
    for t in cut(y):
        t.zero_()
    assert torch.equal(y, z)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def decode_case(rng, lens, H, d_h, r, ps, block, G=1, loud=2, spare=2):
    lens = np.asarray(lens)
    pages = int(sum(-(-n // ps) for n in lens)) + spare
    cache = random_cache(rng, pages, ps, H, d_h, r, block, G, loud)
    table = table_of(rng, lens, ps, pages)
    q, B_K, B_V = (bf16(rng, (len(lens), H, d_h)), bf16(rng, (H, d_h, r), r ** -0.5), bf16(rng, (H, d_h, r), r ** -0.5))
    return cache, table, q, B_K, B_V


def poison_past_the_end(cache, table, lens):
    """NaN codes and the largest scales wherever no request has a row."""
    seen = {k: np.zeros(cache.codes[k].shape[:2], bool) for k in POOLS}
    for k in POOLS:
        for b, n in enumerate(lens):
            for j in range(n):
                seen[k][table[b, j // cache.page_size], j % cache.page_size] = True
        cache.codes[k][~seen[k]] = 0x7f
        blocks = seen[k].reshape(seen[k].shape[0], -1, cache.block).any(2)
        cache.exps[k][~blocks] = 255


def run_decode(cache, table, q, B_K, B_V, lens, longest=None, **kw):
    import rank_kv_attention_gb300 as L
    lens = np.asarray(lens)
    return L.decode_scaled(dev(q[0], "bf16"), to_device(cache), dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), dev(lens, "i32"),
                           dev(table, "i32"), int(longest or max(1, lens.max())), **kw)


def check_decode(out, cache, table, q, B_K, B_V, lens, which=None, **kw):
    got = host(out, "bf16")
    for b in range(len(lens)) if which is None else which:
        ref, bound = reference(q[1][b], cache, B_K[1], B_V[1], table[b], int(lens[b]))
        check(got[b], ref, bound, f"request {b} of {lens[b]} rows", **kw)


DECODE = [  # tensor-core shapes
    (16, 128, 48, 64, 64, 1), (16, 128, 56, 64, 16, 1), (32, 128, 32, 64, 64, 1), (16, 128, 64, 128, 32, 1),
    (16, 128, 48, 32, 32, 1), (16, 128, 32, 16, 16, 1), (4, 128, 16, 64, 64, 1), (8, 128, 40, 48, 48, 1),
    (12, 128, 24, 64, 32, 1), (20, 128, 48, 64, 64, 1), (28, 128, 56, 64, 64, 1), (16, 128, 8, 64, 64, 1),
    # others
    (8, 64, 16, 32, 16, 1), (6, 32, 40, 64, 64, 1), (12, 128, 72, 64, 64, 1), (2, 256, 256, 16, 16, 1),
    (16, 128, 32, 64, 64, 2), (8, 128, 48, 64, 32, 4), (40, 128, 16, 64, 64, 1), (3, 16, 16, 16, 16, 3)]


@pytest.mark.parametrize("H,d_h,r,ps,block,G", DECODE)
def test_decode(H, d_h, r, ps, block, G):
    """Ragged lengths around every tile edge; NaN codes and scales wherever no row is."""
    rng = np.random.default_rng(H * 100 + r)
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 191, 193, 300, 511, 700]
    case = decode_case(rng, lens, H, d_h, r, ps, block, G)
    poison_past_the_end(case[0], case[1], lens)
    st = status()
    out = run_decode(*case, lens, status=st)
    assert int(st) == 0
    check_decode(out, *case, lens)


@pytest.mark.parametrize("H,r,block", [(16, 48, 64), (32, 32, 16), (8, 16, 32)])
@pytest.mark.parametrize("lens", [[1], [64], [1500], [5000], [9000, 1], [3000, 4000, 128]])
def test_decode_of_few_requests(H, r, block, lens):
    rng = np.random.default_rng(sum(lens) + H)
    case = decode_case(rng, lens, H, 128, r, 64, block)
    poison_past_the_end(case[0], case[1], lens)
    check_decode(run_decode(*case, lens), *case, lens)


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 128, 8, 64), (4, 32, 8, 16)])
def test_decode_of_many_requests(H, d_h, r, ps):
    """More requests than SMs, most of a few rows: several requests a CTA."""
    rng = np.random.default_rng(9)
    lens = rng.integers(1, 200, 700)
    lens[::7] = 1
    case = decode_case(rng, lens, H, d_h, r, ps, 16)
    out = run_decode(*case, lens)
    check_decode(out, *case, lens, which=range(0, 700, 23))
    # every request alone gives the same to rounding
    pick = [3, 7, 350, 699]
    sub = (case[0], case[1][pick], (case[2][0][pick], case[2][1][pick]), case[3], case[4])
    check_decode(run_decode(*sub, lens[pick]), *sub, lens[pick])


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (8, 128, 16, 16), (4, 32, 8, 16)])
def test_decode_of_invalid_requests(H, d_h, r, ps):
    """Lengths of zero, negative or past the table give zeros; rows on a bad page are not attended; the others are right."""
    rng = np.random.default_rng(10)
    good = np.array([200, 70, 130, 64, 5, 90, 100])
    case = decode_case(rng, good, H, d_h, r, ps, 16)
    cache, table = case[0], case[1]
    poison_past_the_end(cache, table, good)
    lens = good.copy()
    lens[0], lens[3], lens[5] = 0, -9, table.shape[1] * ps + 1
    table = table.copy()
    table[1, 0] = -1                              # its first page
    table[2, 64 // ps] = len(cache.codes["R_K"])  # one in the middle
    table[6, :] = 2 ** 31 - 1                     # all of them
    case = (cache, table) + case[2:]
    st = status()
    out = run_decode(*case, lens, longest=int(good.max()), status=st)
    assert int(st) == BAD_SEQLEN | BAD_PAGE
    got = host(out, "bf16")
    for b in (0, 3, 5, 6):
        assert not got[b].any()
    check_decode(out, *case, lens, which=[1, 2, 4])


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 32, 8, 16)])
def test_decode_past_max_seq_len(H, d_h, r, ps):
    """A length may exceed max_seq_len: it sizes a launch, no more."""
    rng = np.random.default_rng(11)
    lens = np.array([700, 3, 1300])
    case = decode_case(rng, lens, H, d_h, r, ps, 16)
    check_decode(run_decode(*case, lens, longest=1), *case, lens)


@pytest.mark.parametrize("H,d_h,r", [(16, 128, 48), (4, 32, 8)])
def test_decode_of_loud_blocks(H, d_h, r):
    """Scales many octaves apart from block to block: softmax weights of almost nothing times values of almost everything."""
    rng = np.random.default_rng(12)
    lens = [500, 260, 64, 129]
    cache, table, q, B_K, B_V = decode_case(rng, lens, H, d_h, r, 64, 16)
    for k in ("S_V", "R_V"):
        cache.exps[k][:] = (127 - 7 + rng.integers(-30, 31, cache.exps[k].shape)).astype(np.uint8)
    for k in ("S_K", "R_K"):
        cache.exps[k][:] = (127 - 7 + rng.integers(-8, 4, cache.exps[k].shape)).astype(np.uint8)
    check_decode(run_decode(cache, table, q, B_K, B_V, lens), cache, table, q, B_K, B_V, lens, norm=None)


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -60, 2.0 ** 40])
def test_decode_of_quiet_and_loud_queries(scale):
    """The scores keep their size where the keys make up for it; a zero query attends evenly."""
    rng = np.random.default_rng(13)
    H, r, lens = 16, 48, [300, 65]
    cache, table, q, B_K, B_V = decode_case(rng, lens, H, 128, r, 64, 32)
    bits = I.f32_to_bf16_bits((q[1] * scale).astype(np.float32))
    q = bits, I.bf16_bits_to_f64(bits)
    if scale:
        for k in ("S_K", "R_K"):
            cache.exps[k] -= np.uint8(int(np.log2(scale)) % 256)
    check_decode(run_decode(cache, table, q, B_K, B_V, lens), cache, table, q, B_K, B_V, lens)


@pytest.mark.parametrize("H,d_h,r", [(16, 128, 48), (4, 32, 8)])
def test_a_nan_query_gives_nan(H, d_h, r):
    rng = np.random.default_rng(14)
    lens = [100, 100, 1]
    cache, table, q, B_K, B_V = decode_case(rng, lens, H, d_h, r, 64, 64)
    bits = q[0].copy()
    bits[1, 2, 5] = I.BF16_NAN_BITS
    out = host(run_decode(cache, table, (bits, q[1]), B_K, B_V, lens), "bf16")
    assert np.isnan(out[1, 2]).all() and np.isfinite(np.delete(out[1], 2, 0)).all()
    for b in (0, 2):
        ref, bound = reference(q[1][b], cache, B_K[1], B_V[1], table[b], lens[b])
        check(out[b], ref, bound)


def test_decode_is_the_same_every_time():
    rng = np.random.default_rng(15)
    lens = rng.integers(1, 3000, 40)
    case = decode_case(rng, lens, 16, 128, 48, 64, 32)
    ws = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    first = run_decode(*case, lens, ws=ws)
    for _ in range(3):
        assert torch.equal(run_decode(*case, lens, ws=ws), first)


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 16, 8, 16)])
def test_a_pool_past_2_31_bytes(H, d_h, r, ps):
    """The last pages of a cache of more than 2^31 bytes a pool."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(16)
    pages = (5 << 29) // (ps * H * r)
    dc = L.ScaledCache.empty(pages, ps, H, d_h, r, block=ps)
    small = random_cache(rng, 4, ps, H, d_h, r, ps)
    src, ids = to_device(small), [pages - 1, 0, pages - 3, pages // 2]
    for k in POOLS:
        for name in (k, "E_" + k):
            to, fr = getattr(dc, name).view(torch.uint8), getattr(src, name).view(torch.uint8)
            for i, p in enumerate(ids):
                to[p].copy_(fr[i])
    lens = np.array([3 * ps - 5, ps - 2])
    table = np.array([[0, 1, 2], [3, -1, -1]], np.int32)
    far = np.array([[ids[0], ids[1], ids[2]], [ids[3], -1, -1]], np.int32)
    q, B_K, B_V = bf16(rng, (2, H, d_h)), bf16(rng, (H, d_h, r), r ** -0.5), bf16(rng, (H, d_h, r), r ** -0.5)
    x = values(rng, 3, H, d_h, r, 1, "bf16")
    write(dc, x, [0, 2, 3], lens - [2, 1], far)
    oracle_write(small, x, [0, 2, 3], lens - [2, 1], table)
    out = L.decode_scaled(dev(q[0], "bf16"), dc, dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), dev(lens, "i32"), dev(far, "i32"),
                          int(lens.max()))
    check_decode(out, small, table, q, B_K, B_V, lens)
    got = L.read_scaled(dev(np.array([0, lens[0]]), "i32"), dev(np.zeros(1), "i32"), int(lens[0]), dc, dev(far[:1], "i32"),
                        dtype=torch.float32)
    for k, t in zip(POOLS, got):
        want = S.read(small, k, [0, int(lens[0])], [0], table[:1], np.zeros((int(lens[0]),) + shape_of(k, H, d_h, r, 1)))
        assert np.array_equal(host(t, "f32").reshape(want.shape), want)


# ---------------------------------------------------------------------------
# Append and prefill
# ---------------------------------------------------------------------------
def weights(rng, d, H, d_h, r, G):
    out = {}
    for k, w in zip(POOLS, ("W_S_K", "W_S_V", "U_K", "U_V")):
        heads, width = shape_of(k, H, d_h, r, G)
        std = np.exp2(rng.integers(-3, 3, (heads, 1, 1))) * 0.75 * d ** -0.5
        bits, v = bf16(rng, (heads, width, d))
        bits = I.f32_to_bf16_bits((v * std).astype(np.float32))
        out[w] = (bits.reshape(G * d_h, d) if k[0] == "S" else bits), I.bf16_bits_to_f64(bits)
    return out


def projected(x, w):
    return {k: np.einsum("nd,hwd->nhw", x, w[m][1]) for k, m in zip(POOLS, ("W_S_K", "W_S_V", "U_K", "U_V"))}


def close_caches(got, want, rows, cu, start, table, d):
    """A cache written from rows in fp32 against the one from the exact rows: a value that lies on the border of two codes,
    or a maximum on the border of two scales, may go either way.  Codes of new rows: within half a step of the fp32 row,
    whose error a sum of d products bounds; exponents as needed by the fp32 row's bounds."""
    for k in POOLS:
        g, w = got.exps[k].astype(int), want.exps[k].astype(int)
        assert np.mean(g != w) <= 1e-3 and np.abs(g - w).max() <= 1, k
        vg = np.stack([got.row(k, p, s) for p in range(g.shape[0]) for s in range(got.page_size)])
        vw = np.stack([want.row(k, p, s) for p in range(g.shape[0]) for s in range(got.page_size)])
        big = np.maximum(np.abs(vg), np.abs(vw))
        step = np.repeat(2.0 ** (np.maximum(g, w) - 127.0), got.block, 1).reshape(-1, g.shape[2])[..., None]
        differ = vg != vw
        assert np.mean(differ) <= 1e-3, (k, np.mean(differ))
        assert np.all(np.abs(vg - vw) <= np.maximum(2.0 ** -3 * big, 2.0 ** -9 * step)), k


PROJ = [(16, 128, 48, 1, 64, 64, 256), (8, 128, 16, 1, 64, 16, 64), (4, 64, 16, 1, 32, 32, 96), (6, 32, 40, 2, 48, 16, 72),
        (32, 128, 32, 1, 64, 32, 128), (12, 128, 72, 1, 64, 64, 64), (16, 128, 64, 1, 128, 64, 192)]


@pytest.mark.parametrize("rows_of", [[1, 1, 1], [0, 17, 40], [150, 1, 230]])
@pytest.mark.parametrize("H,d_h,r,G,ps,block,d", PROJ)
def test_append(H, d_h, r, G, ps, block, d, rows_of):
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(d + sum(rows_of))
    start = np.array([ps - 1, 0, block + 3])
    lens = start + rows_of
    pages = int(sum(-(-n // ps) for n in lens)) + 1
    cache, table = random_cache(rng, pages, ps, H, d_h, r, block, G), table_of(rng, lens, ps, pages)
    cu, n = np.concatenate([[0], np.cumsum(rows_of)]), int(sum(rows_of))
    w, x = weights(rng, d, H, d_h, r, G), bf16(rng, (n, d))
    dc, st = to_device(cache), status()
    L.append_scaled(dev(x[0], "bf16"), dev(cu, "i32"), dev(start, "i32"), *[dev(w[m][0], "bf16") for m in w], dc,
                    dev(table, "i32"), status=st)
    assert int(st) == 0
    S.write(cache, projected(x[1], w), cu, start, table)
    close_caches(to_host(dc, cache), cache, None, cu, start, table, d)


@pytest.mark.parametrize("H,d_h,r,G,ps,block,d", [PROJ[0], PROJ[4], PROJ[1], (8, 128, 64, 4, 128, 64, 128)])
def test_append_and_prefill_of_many_short_requests(H, d_h, r, G, ps, block, d):
    """More requests than row tiles pay for: none, one and a few rows each."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(H + r)
    B = 70
    rows_of, start = rng.integers(0, 5, B), rng.integers(0, 100, B)
    lens = rows_of + start
    pages = int(sum(-(-n // ps) for n in lens)) + 1
    table = table_of(rng, lens, ps, pages, width=-(-104 // ps))
    cu, n = np.concatenate([[0], np.cumsum(rows_of)]), int(rows_of.sum())
    before = random_cache(rng, pages, ps, H, d_h, r, block, G, loud=1)
    w, x, q = weights(rng, d, H, d_h, r, G), bf16(rng, (n, d)), bf16(rng, (n, H, d_h))
    B_K, B_V = bf16(rng, (H, d_h, r), r ** -0.5), bf16(rng, (H, d_h, r), r ** -0.5)
    dc, other, st = to_device(before), to_device(before), status()
    args = [dev(cu, "i32"), dev(start, "i32")]
    L.append_scaled(dev(x[0], "bf16"), *args, *[dev(w[m][0], "bf16") for m in w], dc, dev(table, "i32"), status=st)
    out = L.prefill_scaled(dev(x[0], "bf16"), dev(q[0], "bf16"), *args, 104, *[dev(w[m][0], "bf16") for m in w],
                           dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), other, dev(table, "i32"), status=st)
    assert int(st) == 0
    held, want = to_host(dc, before), before.copy()
    S.write(want, projected(x[1], w), cu, start, table)
    close_caches(held, want, None, cu, start, table, d)
    assert_same(to_host(other, before), held)
    got = host(out, "bf16")
    for b in range(0, B, 7):
        for i in {cu[b], cu[b + 1] - 1} if rows_of[b] else ():
            ref, bound = reference(q[1][i], held, B_K[1], B_V[1], table[b], int(start[b] + i - cu[b] + 1), G == 1)
            check(got[i], ref, bound, f"request {b}")


@pytest.mark.parametrize("rows_of,start", [([1, 1, 1], [5, 0, 200]), ([130, 0, 200], [0, 9, 77]), ([3, 300, 64], [190, 0, 64])])
@pytest.mark.parametrize("H,d_h,r,G,ps,block,d", PROJ)
def test_prefill(H, d_h, r, G, ps, block, d, rows_of, start):
    """The outputs over what the cache holds after the call; rows of no request stay."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(d + sum(rows_of) + H)
    lens = np.array(start) + rows_of
    pages = int(sum(-(-n // ps) for n in lens)) + 1
    cache, table = random_cache(rng, pages, ps, H, d_h, r, block, G, loud=1), table_of(rng, lens, ps, pages)
    poison_past_the_end(cache, table, start)
    cu, n = np.concatenate([[2], 2 + np.cumsum(rows_of)]), int(sum(rows_of)) + 5
    w, x = weights(rng, d, H, d_h, r, G), bf16(rng, (n, d))
    q, B_K, B_V = bf16(rng, (n, H, d_h)), bf16(rng, (H, d_h, r), r ** -0.5), bf16(rng, (H, d_h, r), r ** -0.5)
    dc, st = to_device(cache), status()
    out = torch.full((n, H, d_h), 3.0, dtype=torch.bfloat16, device="cuda")
    L.prefill_scaled(dev(x[0], "bf16"), dev(q[0], "bf16"), dev(cu, "i32"), dev(np.array(start), "i32"), int(lens.max()),
                     *[dev(w[m][0], "bf16") for m in w], dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), dc, dev(table, "i32"),
                     out=out, status=st)
    assert int(st) == 0
    held = to_host(dc, cache)
    S.write(cache, projected(x[1], w), cu, start, table)
    poison = cache.copy()
    for c in (held, poison):     # (rows no request has hold NaN)
        for k in POOLS:
            c.codes[k] = np.where((c.codes[k] & 0x7f) == 0x7f, 0, c.codes[k])
    close_caches(held, poison, None, cu, start, table, d)
    got = host(out, "bf16")
    assert (got[:2] == 3).all() and (got[cu[-1]:] == 3).all()
    tiled = d_h == 128 and G == 1 and r <= 64 and ps % 64 == 0
    for b in range(3):
        for i in sorted({cu[b], (cu[b] + cu[b + 1]) // 2, cu[b + 1] - 1} & set(range(cu[b], cu[b + 1]))):
            ref, bound = reference(q[1][i], held, B_K[1], B_V[1], table[b], start[b] + i - cu[b] + 1, tiled)
            check(got[i], ref, bound, f"request {b} row {i - cu[b]}")


def test_prefill_in_a_pool_smaller_than_its_requests():
    """Requests that share all but their last pages: the values are laid out once a page of the pool."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(20)
    H, d_h, r, ps, d, B = 8, 128, 16, 64, 64, 12
    cache = random_cache(rng, 4 + B, ps, H, d_h, r, 32, loud=1)
    table = np.array([[0, 1, 2, 3, 4 + b] for b in range(B)], np.int32)
    start, cu = np.full(B, 4 * ps), np.arange(B + 1) * 20
    w, x, q = weights(rng, d, H, d_h, r, 1), bf16(rng, (20 * B, d)), bf16(rng, (20 * B, H, d_h))
    B_K, B_V = bf16(rng, (H, d_h, r), r ** -0.5), bf16(rng, (H, d_h, r), r ** -0.5)
    dc = to_device(cache)
    out = L.prefill_scaled(dev(x[0], "bf16"), dev(q[0], "bf16"), dev(cu, "i32"), dev(start, "i32"), 4 * ps + 20,
                           *[dev(w[m][0], "bf16") for m in w], dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), dc, dev(table, "i32"))
    held, got = to_host(dc, cache), host(out, "bf16")
    for b in (0, 5, 11):
        for i in (0, 19):
            ref, bound = reference(q[1][20 * b + i], held, B_K[1], B_V[1], table[b], 4 * ps + i + 1, True)
            check(got[20 * b + i], ref, bound)


@pytest.mark.parametrize("start,rows", [(0, 100), (100, 70), (130, 300), (255, 66)])
@pytest.mark.parametrize("wide", [False, True])
def test_prefill_of_one_request(start, rows, wide):
    """wide: a table beyond the pool, whose pages the values then follow.  The loud new rows make the block that they share
    with the history grow."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(start + rows)
    H, r, ps, d, block = 8, 24, 64, 64, 64
    pages = -(-(start + rows) // ps)
    cache = random_cache(rng, pages, ps, H, 128, r, block, loud=1)
    table = np.full((1, 3 * pages if wide else pages), -1, np.int32)
    table[0, :pages] = rng.permutation(pages)
    w, x, q = weights(rng, d, H, 128, r, 1), bf16(rng, (rows, d), 8.0), bf16(rng, (rows, H, 128))
    B_K, B_V = bf16(rng, (H, 128, r), r ** -0.5), bf16(rng, (H, 128, r), r ** -0.5)
    dc, st = to_device(cache), status()
    out = L.prefill_scaled(dev(x[0], "bf16"), dev(q[0], "bf16"), dev(np.array([0, rows]), "i32"), dev(np.array([start]), "i32"),
                           table.shape[1] * ps, *[dev(w[m][0], "bf16") for m in w], dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), dc,
                           dev(table, "i32"), status=st)
    assert int(st) == 0
    held, got = to_host(dc, cache), host(out, "bf16")
    S.write(cache, projected(x[1], w), [0, rows], [start], table)
    close_caches(held, cache, None, [0, rows], [start], table, d)
    for i in sorted({0, 1, rows // 2, rows - 1}):
        ref, bound = reference(q[1][i], held, B_K[1], B_V[1], table[0], start + i + 1, True)
        check(got[i], ref, bound, f"row {i}")


@pytest.mark.parametrize("H,d_h,r,ps", [(8, 128, 16, 64), (4, 32, 8, 16)])
def test_prefill_on_bad_pages(H, d_h, r, ps):
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(21)
    d, start, rows_of = 64, [130, 64], [70, 20]
    lens = np.add(start, rows_of)
    cache, table = random_cache(rng, 40, ps, H, d_h, r, 16, loud=1), table_of(rng, lens, ps, 40)
    table[0, 64 // ps], table[1, 64 // ps] = -1, 40
    cu = [0, 70, 90]
    w, x, q = weights(rng, d, H, d_h, r, 1), bf16(rng, (90, d)), bf16(rng, (90, H, d_h))
    B_K, B_V = bf16(rng, (H, d_h, r), r ** -0.5), bf16(rng, (H, d_h, r), r ** -0.5)
    dc, st = to_device(cache), status()
    out = L.prefill_scaled(dev(x[0], "bf16"), dev(q[0], "bf16"), dev(np.array(cu), "i32"), dev(np.array(start), "i32"),
                           int(lens.max()), *[dev(w[m][0], "bf16") for m in w], dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), dc,
                           dev(table, "i32"), status=st)
    assert int(st) == BAD_PAGE
    held, got = to_host(dc, cache), host(out, "bf16")
    for b, i in ((0, 0), (0, 69), (1, 0), (1, 19)):
        ref, bound = reference(q[1][cu[b] + i], held, B_K[1], B_V[1], table[b], start[b] + i + 1, d_h == 128)
        check(got[cu[b] + i], ref, bound)


SPLIT = [(16, 48, 64, 32, [700], [300]), (16, 48, 64, 64, [511], [1]), (16, 64, 128, 64, [300, 512], [128, 100]),
         (32, 32, 64, 64, [1400], [256]), (4, 16, 64, 16, [-40], [900]), (4, 56, 64, 64, [384, 385, 1000], [1, 130, 257]),
         (8, 8, 192, 48, [900], [127]), (16, 40, 64, 64, [3001], [512]), (16, 48, 64, 64, [3001], [100]),
         (4, 48, 64, 64, [100, 513, 1300, 900], [20, 3, 128, 129]), (32, 16, 64, 32, [1000], [5])]


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("H,r,ps,block,start,rows_of", SPLIT)
def test_prefill_of_few_query_tiles(H, r, ps, block, start, rows_of, bad):
    """Chunks behind long histories, whose query tiles leave SMs idle: CTAs share a tile's keys.  bad: pages missing near both
    ends."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(H * r + sum(rows_of) + bad)
    B, d = len(start), 64
    lens = np.add(start, rows_of)
    pages = int(sum(-(-n // ps) for n in lens)) + 1
    cache, table = random_cache(rng, pages, ps, H, 128, r, block, loud=1), table_of(rng, lens, ps, pages)
    poison_past_the_end(cache, table, start)
    for b in range(B) if bad else ():
        table[b, 1], table[b, (lens[b] - 1) // ps - 1] = -1, pages
    cu, n = np.concatenate([[0], np.cumsum(rows_of)]), int(sum(rows_of))
    w, x, q = weights(rng, d, H, 128, r, 1), bf16(rng, (n, d)), bf16(rng, (n, H, 128))
    B_K, B_V = bf16(rng, (H, 128, r), r ** -0.5), bf16(rng, (H, 128, r), r ** -0.5)
    dc, st = to_device(cache), status()
    args = [dev(x[0], "bf16"), dev(q[0], "bf16"), dev(cu, "i32"), dev(np.array(start), "i32"), int(lens.max()),
            *[dev(w[m][0], "bf16") for m in w], dev(B_K[0], "bf16"), dev(B_V[0], "bf16")]
    out, again = torch.zeros(2, n, H, 128, dtype=torch.bfloat16, device="cuda")
    L.prefill_scaled(*args, dc, dev(table, "i32"), out=out, status=st)
    # (rows that are counted from a negative position may be more than max_ctx)
    tiled = -(-int(lens.max()) // 128) * 128
    assert int(st) == (BAD_PAGE if bad else 0) | (BAD_ROW if min(start) < 0 else 0) | (BAD_SEQLEN if max(rows_of) > tiled else 0)
    L.prefill_scaled(*args, to_device(cache), dev(table, "i32"), out=again)
    same = torch.equal(again, out)
    assert same
    held, got = to_host(dc, cache), host(out, "bf16")
    for b in range(B):
        for i in sorted({max(0, -start[b]), rows_of[b] // 2, max(0, rows_of[b] - 129), min(tiled, rows_of[b]) - 1}):
            ref, bound = reference(q[1][cu[b] + i], held, B_K[1], B_V[1], table[b], start[b] + i + 1, True)
            check(got[cu[b] + i], ref, bound, f"request {b} row {i}")
        assert not got[cu[b]:cu[b] + max(0, -start[b])].any()


# ---------------------------------------------------------------------------
# Used together
# ---------------------------------------------------------------------------
class Server:
    """Requests served from a block-scaled cache as a program does it: page plan, prefill or append, decode."""

    def __init__(self, rng, H=16, d_h=128, r=48, ps=64, block=32, d=128, pages=40, B=3, max_pages=12):
        import rank_kv_attention_gb300 as L
        self.L, self.H, self.d_h, self.r, self.ps, self.d, self.B = L, H, d_h, r, ps, d, B
        self.w = weights(rng, d, H, d_h, r, 1)
        self.dw = [dev(self.w[m][0], "bf16") for m in self.w]
        self.B_K, self.B_V = bf16(rng, (H, d_h, r), r ** -0.5), bf16(rng, (H, d_h, r), r ** -0.5)
        self.dB = dev(self.B_K[0], "bf16"), dev(self.B_V[0], "bf16")
        self.oracle = random_cache(rng, pages, ps, H, d_h, r, block)
        self.cache = to_device(self.oracle)
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free, self.n_free = dev(rng.permutation(pages), "i32"), dev(np.array([pages]), "i32")
        self.lens = dev(np.zeros(B), "i32")

    def plan(self, new, rows):
        p = self.L.page_plan(self.lens, dev(np.asarray(new), "i32"), self.table, self.free, self.n_free, self.ps, rows)
        before = self.lens
        self.lens, self.free, self.n_free = p.seq_lens, p.free_pages, p.n_free
        return p, before


def test_a_request_served_from_its_prompt_on():
    """Two prompt chunks, then single tokens: every output over what the cache then holds, and the cache as the oracle's."""
    rng = np.random.default_rng(30)
    s = Server(rng)
    for new in ([70, 1, 200], [33, 64, 0], [1, 1, 1], [1, 0, 1], [1, 1, 1]):
        n, single = sum(new), max(new) == 1
        x, q = bf16(rng, (n, s.d)), bf16(rng, (n, s.H, s.d_h))
        p, before = s.plan(new, n)
        start, cu = before.cpu().numpy(), np.concatenate([[0], np.cumsum(new)])
        if single:
            s.L.append_scaled(dev(x[0], "bf16"), p.cu_rows, before, *s.dw, s.cache, s.table)
            live = [b for b in range(s.B) if new[b]]
            out = s.L.decode_scaled(dev(q[0], "bf16"), s.cache, *s.dB, s.lens[live], s.table[live].contiguous(), 700)
        else:
            out = s.L.prefill_scaled(dev(x[0], "bf16"), dev(q[0], "bf16"), p.cu_rows, before, 512, *s.dw, *s.dB, s.cache,
                                     s.table)
        table = s.table.cpu().numpy()
        S.write(s.oracle, projected(x[1], s.w), cu, start, table)
        held, got = to_host(s.cache, s.oracle), host(out, "bf16")
        close_caches(held, s.oracle, None, cu, start, table, s.d)
        s.oracle = held
        for b in range(s.B):
            for i in {cu[b], cu[b + 1] - 1} if new[b] else ():
                ref, bound = reference(q[1][i], held, s.B_K[1], s.B_V[1], table[b], int(start[b]) + int(i - cu[b]) + 1, not single)
                check(got[i], ref, bound, f"{new} request {b}")


def test_a_step_captured_in_a_graph():
    """Append and decode in one graph, replayed on new rows, queries and lengths; a second graph of its own beside it."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(31)
    s = Server(rng, pages=30, max_pages=8)
    s.plan([100, 64, 250], 414)
    start = s.lens.clone()
    cu = dev(np.arange(4), "i32")
    graphs = []
    for k in range(2):
        x, q = torch.zeros(3, s.d, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 16, 128, dtype=torch.bfloat16, device="cuda")
        at, lens = start.clone(), start + 1
        wa = L.api.workspace(L.append_scaled_workspace_bytes(s.cache, 3))
        wd = L.api.workspace(L.decode_scaled_workspace_bytes(s.cache, 3, 512))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())

        def step():
            L.append_scaled(x, cu, at, *s.dw, s.cache, s.table, ws=wa)
            return L.decode_scaled(q, s.cache, *s.dB, lens, s.table, 512, ws=wd)
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, x, q, at, lens, out))
    table = s.table.cpu().numpy()
    for i in range(6):
        g, x, q, at, lens, out = graphs[i % 2]
        xb, qb = bf16(rng, (3, s.d)), bf16(rng, (3, 16, 128))
        x.copy_(dev(xb[0], "bf16"))
        q.copy_(dev(qb[0], "bf16"))
        at.copy_(start + i)
        lens.copy_(start + i + 1)
        g.replay()
        held, got = to_host(s.cache, s.oracle), host(out, "bf16")
        for b in range(3):
            n = int(start[b]) + i + 1
            ref, bound = reference(qb[1][b], held, s.B_K[1], s.B_V[1], table[b], n)
            check(got[b], ref, bound)


def test_calls_on_two_streams():
    """Two decodes and a read at once, each on a stream and with a workspace of its own."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(32)
    lens = [900, 64, 2000, 1]
    cases = [decode_case(rng, lens, 16, 128, 48, 64, 64), decode_case(rng, lens, 32, 128, 32, 64, 16)]
    args = [(dev(q[0], "bf16"), to_device(c), dev(k[0], "bf16"), dev(v[0], "bf16"), dev(np.array(lens), "i32"), dev(t, "i32"), 2000)
            for c, t, q, k, v in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for k in (0, 1):
            outs[k].append(L.decode_scaled(*args[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k, case in enumerate(cases):
        check_decode(outs[k][0], *case, lens)
        assert all(torch.equal(o, outs[k][0]) for o in outs[k])


def test_written_rows_attend_like_a_bf16_cache_of_their_values():
    """decode_scaled over codes and decode over the values it reads back: the same attention."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(33)
    lens = np.array([700, 130])
    cache, table, q, B_K, B_V = decode_case(rng, lens, 16, 128, 48, 64, 32)
    dc, cu = to_device(cache), np.array([0, 700, 830])
    rows = L.read_scaled(dev(cu, "i32"), dev(np.zeros(2), "i32"), 830, dc, dev(table, "i32"))
    pools = [torch.zeros(20, 64, *t.shape[1:], dtype=torch.bfloat16, device="cuda") for t in rows]
    wide = np.array([[b * 11 + k for k in range(11)] if b == 0 else [11 + k if k < 3 else -1 for k in range(11)] for b in range(2)])
    for b in range(2):
        for j in range(lens[b]):
            for p, t in zip(pools, rows):
                p[int(wide[b, j // 64]), j % 64] = t[cu[b] + j]
    want = host(L.decode(dev(q[0], "bf16"), L.PagedCache(*pools), dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), dev(lens, "i32"),
                         dev(wide, "i32"), 700), "bf16")
    out = run_decode(cache, table, q, B_K, B_V, lens)
    check_decode(out, cache, table, q, B_K, B_V, lens)
    for b in range(2):
        _, bound = reference(q[1][b], cache, B_K[1], B_V[1], table[b], int(lens[b]))
        assert np.all(np.abs(host(out, "bf16")[b] - want[b]) <= 2 * bound)


# ---------------------------------------------------------------------------
# Ends of the ranges
# ---------------------------------------------------------------------------
MORE = [(8, 128, 64, 4, 128, 64, 128), (16, 128, 8, 1, 64, 64, 64), (4, 128, 40, 2, 128, 128, 64), (6, 128, 128, 1, 64, 16, 64),
        (4, 128, 16, 1, 256, 256, 64), (8, 128, 24, 1, 64, 32, 72)]


@pytest.mark.parametrize("rows_of", [[1, 0, 2], [70, 1, 200]])
@pytest.mark.parametrize("H,d_h,r,G,ps,block,d", MORE)
def test_append_and_prefill_of_more_shapes(H, d_h, r, G, ps, block, d, rows_of):
    """Groups of wide heads, narrow and wide private rows, blocks of a page, widths that the projection on tensor cores
    does not take."""
    test_append(H, d_h, r, G, ps, block, d, rows_of)
    test_prefill(H, d_h, r, G, ps, block, d, rows_of, [ps - 3, 0, block + 3])


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 32, 8, 32)])
def test_append_and_prefill_of_rows_that_have_no_place(H, d_h, r, ps):
    """Negative positions, rows past the table, pages outside the pool: skipped and flagged; the other rows are written and
    attended as ever."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(40)
    d, B, width = 64, 4, 4
    cache = random_cache(rng, 14, ps, H, d_h, r, 16, loud=1)
    table = np.array([[0, 1, 2, -1], [3, 4, 5, 6], [7, 14, 8, 9], [10, 11, -5, 12]], np.int32)
    cu, start = np.array([2, 72, 152, 222, 292]), np.array([-9, width * ps - 30, 20, 30])
    n = 300
    w, x, q = weights(rng, d, H, d_h, r, 1), bf16(rng, (n, d)), bf16(rng, (n, H, d_h))
    B_K, B_V = bf16(rng, (H, d_h, r), r ** -0.5), bf16(rng, (H, d_h, r), r ** -0.5)
    args = (dev(cu, "i32"), dev(start, "i32"))
    before = cache.copy()
    for prefill in (False, True):
        dc, st = to_device(before), status()
        if prefill:
            out = L.prefill_scaled(dev(x[0], "bf16"), dev(q[0], "bf16"), *args, width * ps, *[dev(w[m][0], "bf16") for m in w],
                                   dev(B_K[0], "bf16"), dev(B_V[0], "bf16"), dc, dev(table, "i32"), status=st)
        else:
            L.append_scaled(dev(x[0], "bf16"), *args, *[dev(w[m][0], "bf16") for m in w], dc, dev(table, "i32"), status=st)
        assert int(st) == BAD_ROW | BAD_PAGE
        want = before.copy()
        S.write(want, projected(x[1], w), cu, start, table)
        held = to_host(dc, cache)
        close_caches(held, want, None, cu, start, table, d)
    got = host(out, "bf16")
    for b, i in ((0, 9), (0, 69), (1, 0), (1, 29), (2, 69), (3, 69)):
        ref, bound = reference(q[1][cu[b] + i], held, B_K[1], B_V[1], table[b], int(start[b]) + i + 1, d_h == 128)
        check(got[cu[b] + i], ref, bound, f"request {b} row {i}")


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 32, 8, 32)])
def test_a_prefill_past_max_ctx_is_flagged(H, d_h, r, ps):
    """Rows from max_ctx on (of the tiled kernel: query tiles) are written, not attended, and flagged."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(48)
    d, n = 64, 300
    cache = random_cache(rng, 12, ps, H, d_h, r, 16, loud=1)
    dc, table, st = to_device(cache), np.arange(12, dtype=np.int32)[None], status()
    w, x, q = weights(rng, d, H, d_h, r, 1), bf16(rng, (n, d)), bf16(rng, (n, H, d_h))
    B = dev(bf16(rng, (H, d_h, r), r ** -0.5)[0], "bf16")
    L.prefill_scaled(dev(x[0], "bf16"), dev(q[0], "bf16"), dev(np.array([0, n]), "i32"), dev(np.zeros(1), "i32"), 128,
                     *[dev(w[m][0], "bf16") for m in w], B, B, dc, dev(table, "i32"), status=st)
    assert int(st) & BAD_SEQLEN
    S.write(cache, projected(x[1], w), [0, n], [0], table)
    close_caches(to_host(dc, cache), cache, None, [0, n], [0], table, d)


@pytest.mark.parametrize("H,d_h,r,ps", [(16, 128, 48, 64), (4, 32, 8, 32)])
def test_append_and_prefill_without_order_do_no_harm(H, d_h, r, ps):
    """cu_rows that fall or run past n: no row is read or written outside the call's, and the next call is right."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(41)
    d, n = 64, 150
    cache = random_cache(rng, 16, ps, H, d_h, r, 16, loud=1)
    dc, table = to_device(cache), np.arange(16, dtype=np.int32).reshape(4, 4)
    w, x, q = weights(rng, d, H, d_h, r, 1), bf16(rng, (n, d)), bf16(rng, (n, H, d_h))
    dw, B = [dev(w[m][0], "bf16") for m in w], dev(bf16(rng, (H, d_h, r), r ** -0.5)[0], "bf16")
    dx, dq, dt, zero = dev(x[0], "bf16"), dev(q[0], "bf16"), dev(table, "i32"), dev(np.zeros(4), "i32")
    for cu in ([0, 90, 40, 100, 900], [-50, 4, 3, 2, 1], [400, 500, 600, 700, 800], [2 ** 31 - 1, -2 ** 31, 7, 80, 2 ** 31 - 1],
               [0, 0, 0, 0, 0]):
        dcu = dev(np.array(cu), "i32")
        L.append_scaled(dx, dcu, zero, *dw, dc, dt)
        L.prefill_scaled(dx, dq, dcu, zero, 4 * ps, *dw, B, B, dc, dt)
        L.prefill_scaled(dx, dq, dcu, zero, 20, *dw, B, B, dc, dt)          # (rows past max_ctx)
    torch.cuda.synchronize()
    cache, cu = to_host(dc, cache), [0, 40, 90, 100, 150]
    L.append_scaled(dx, dev(np.array(cu), "i32"), zero, *dw, dc, dt)
    S.write(cache, projected(x[1], w), cu, [0] * 4, table)
    close_caches(to_host(dc, cache), cache, None, cu, [0] * 4, table, d)


@pytest.mark.parametrize("d,rows", [(64, 100), (72, 20)])
def test_append_of_values_that_are_not_finite(d, rows):
    """A row of X with an infinity or a NaN: NaN or infinite sums become NaN codes, the block's other rows decide its scale."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(42)
    H, d_h, r, ps = 16, 128, 48, 64
    cache = random_cache(rng, 3, ps, H, d_h, r, 32)
    dc, table = to_device(cache), np.array([[1, 0, 2]], np.int32)
    w, (bits, x) = weights(rng, d, H, d_h, r, 1), bf16(rng, (rows, d))
    for i, v, b in ((3, np.nan, I.BF16_NAN_BITS), (7, np.inf, 0x7f80), (rows - 1, -np.inf, 0xff80)):
        x[i, i % d], bits[i, i % d] = v, b
    L.append_scaled(dev(bits, "bf16"), dev(np.array([0, rows]), "i32"), dev(np.array([5]), "i32"),
                    *[dev(w[m][0], "bf16") for m in w], dc, dev(table, "i32"))
    with np.errstate(invalid="ignore"):
        y = projected(x, w)
    for k in POOLS:
        assert not np.isfinite(y[k][[3, 7, rows - 1]]).any()
    S.write(cache, y, [0, rows], [5], table)
    held = to_host(dc, cache)
    for c in (held, cache):      # (NaN codes in the same places, then compared as zeros)
        for k in POOLS:
            nan = (c.codes[k] & 0x7f) == 0x7f
            for i in (3, 7, rows - 1):
                assert nan[table[0, (5 + i) // ps], (5 + i) % ps].all()
            assert nan.sum() == 3 * nan[0, 0].size
            c.codes[k] = np.where(nan, 0, c.codes[k])
    close_caches(held, cache, None, [0, rows], [5], table, d)


@pytest.mark.parametrize("H,d_h,r", [(16, 128, 48), (4, 32, 8)])
def test_decode_of_the_largest_queries(H, d_h, r):
    """Elements at the end of bf16's range against the smallest keys: scores of ordinary size."""
    rng = np.random.default_rng(43)
    lens = [200, 64]
    cache, table, q, B_K, B_V = decode_case(rng, lens, H, d_h, r, 64, 32)
    for k in ("S_K", "R_K"):
        cache.codes[k] = (rng.integers(0, 8, cache.codes[k].shape) | (rng.integers(0, 2, cache.codes[k].shape) << 7)).astype(np.uint8)
        cache.exps[k][:] = 10
    x = np.zeros((2, H, d_h), np.float32)
    x[:, :, 5], x[:, :, 9] = 3.38e38, -3e38
    bits = I.f32_to_bf16_bits(x)
    bk = B_K[1].copy()
    bk[:, [5, 9]] = np.clip(bk[:, [5, 9]], -0.45, 0.45)    # (p stays finite)
    bkb = I.f32_to_bf16_bits(bk.astype(np.float32))
    q, B_K = (bits, I.bf16_bits_to_f64(bits)), (bkb, I.bf16_bits_to_f64(bkb))
    check_decode(run_decode(cache, table, q, B_K, B_V, lens), cache, table, q, B_K, B_V, lens)


def test_decode_reads_a_page_twice_and_shares_pages():
    """A table that names a page twice, and requests on the same pages: read as often as named."""
    rng = np.random.default_rng(44)
    lens = [250, 128, 70]
    cache, table, q, B_K, B_V = decode_case(rng, lens, 16, 128, 48, 64, 16)
    table[0, 2], table[1], table[2, 0] = table[0, 0], table[0], table[0, 3]
    check_decode(run_decode(cache, table, q, B_K, B_V, lens), cache, table, q, B_K, B_V, lens)


@pytest.mark.parametrize("H,r", [(16, 48), (32, 16)])
def test_decode_of_thousands_of_requests(H, r):
    """More requests than a launch's threads, of one row or none."""
    rng = np.random.default_rng(45)
    B, cache = 5000, random_cache(rng, 8, 64, H, 128, r, 64)
    lens = rng.choice([0, 1, 1, 2, 64], B)
    lens[:300], lens[-1] = 0, 64
    table = rng.integers(0, 8, (B, 1)).astype(np.int32)
    q, B_K, B_V = bf16(rng, (B, H, 128)), bf16(rng, (H, 128, r), r ** -0.5), bf16(rng, (H, 128, r), r ** -0.5)
    st = status()
    out = run_decode(cache, table, q, B_K, B_V, lens, status=st)
    assert int(st) == BAD_SEQLEN
    assert not host(out, "bf16")[lens == 0].any()
    which = [b for b in list(range(300, B, 211)) + [B - 1] if lens[b]]
    check_decode(out, cache, table, q, B_K, B_V, lens, which=which)


def test_a_prefill_captured_in_a_graph_and_on_a_stream():
    """One graph of a prefill, replayed for other rows, counts and positions, with rows to spare; the same calls on a
    stream of their own give the same."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(46)
    s = Server(rng, pages=40, max_pages=8)
    table = np.array([rng.permutation(40)[:24].reshape(3, 8)], np.int32)[0]
    dt, n = dev(table, "i32"), 160
    x, q = (torch.zeros(n, k, dtype=torch.bfloat16, device="cuda") for k in (s.d, 16 * 128))
    q = q.view(n, 16, 128)
    cu, at = dev(np.array([0, 0, 0, 0]), "i32"), dev(np.zeros(3), "i32")
    ws = L.api.workspace(L.prefill_scaled_workspace_bytes(s.cache, 3, n, 512))
    out, side = torch.empty(n, 16, 128, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream()

    def call(cache, **kw):
        return L.prefill_scaled(x, q, cu, at, 512, *s.dw, *s.dB, cache, dt, **kw)
    with torch.cuda.stream(side):
        call(s.cache, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(s.cache, out=out, ws=ws)
    for counts, start in (([100, 1, 30], [0, 63, 200]), ([0, 160, 0], [9, 300, 9]), ([50, 50, 50], [100, 0, 230])):
        xb, qb = bf16(rng, (n, s.d)), bf16(rng, (n, 16, 128))
        x.copy_(dev(xb[0], "bf16"))
        q.copy_(dev(qb[0], "bf16"))
        cu.copy_(dev(np.concatenate([[0], np.cumsum(counts)]), "i32"))
        at.copy_(dev(np.array(start), "i32"))
        other = to_device(to_host(s.cache, s.oracle))
        torch.cuda.synchronize()
        g.replay()
        alone = call(other, stream=side)
        torch.cuda.synchronize()
        rows = sum(counts)
        assert torch.equal(out[:rows], alone[:rows])
        held = to_host(s.cache, s.oracle)
        assert_same(to_host(other, s.oracle), held)
        got, c = host(out, "bf16"), np.concatenate([[0], np.cumsum(counts)])
        for b in range(3):
            for i in {0, counts[b] - 1} if counts[b] else ():
                ref, bound = reference(qb[1][c[b] + i], held, s.B_K[1], s.B_V[1], table[b], start[b] + i + 1, True)
                check(got[c[b] + i], ref, bound)


def test_writes_and_reads_on_other_streams():
    """Rows written on one stream and read on another after it, beside an append into a second cache."""
    import rank_kv_attention_gb300 as L
    rng = np.random.default_rng(47)
    H, d_h, r, ps, d, n = 16, 128, 48, 64, 64, 300
    caches = [random_cache(rng, 6, ps, H, d_h, r, 32) for _ in range(2)]
    dcs, table, w = [to_device(c) for c in caches], np.arange(6, dtype=np.int32)[None], weights(rng, d, H, d_h, r, 1)
    rows, x = values(rng, n, H, d_h, r, 1, "bf16"), bf16(rng, (n, d))
    dw, cu, at, dt, dx = [dev(w[m][0], "bf16") for m in w], dev(np.array([0, n]), "i32"), dev(np.zeros(1), "i32"), dev(table, "i32"), \
        dev(x[0], "bf16")
    a, b, c = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()
    for _ in range(5):
        L.append_scaled(dx, cu, at, *dw, dcs[1], dt, stream=b)
        L.write_scaled(*[rows[k][0].reshape(n, -1) for k in POOLS], cu, at, dcs[0], dt, stream=a)
    c.wait_stream(a)
    got = L.read_scaled(cu, at, n, dcs[0], dt, dtype=torch.float32, stream=c)
    torch.cuda.synchronize()
    S.write(caches[0], {k: rows[k][1] for k in POOLS}, [0, n], [0], table)
    S.write(caches[1], projected(x[1], w), [0, n], [0], table)
    assert_same(to_host(dcs[0], caches[0]), caches[0])
    close_caches(to_host(dcs[1], caches[1]), caches[1], None, [0, n], [0], table, d)
    for k, t in zip(POOLS, got):
        want = S.read(caches[0], k, [0, n], [0], table, np.zeros((n,) + shape_of(k, H, d_h, r, 1)))
        assert np.array_equal(host(t, "f32").reshape(want.shape), want)
