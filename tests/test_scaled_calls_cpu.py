"""What the block-scaled cache's functions refuse, on host tensors and fake
addresses, and where the buffers of a call come from.  No call here touches a GPU."""
import ctypes

import pytest
import torch

from rank_kv_attention_gb300 import _abi, api
from test_window_calls_cpu import Library, Stream

H, D_H, R, PAGE, BLOCK, B, MAX_PAGES, N, D = 4, 128, 16, 64, 32, 2, 3, 7, 64
F8, BF, U8, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.uint8, torch.int32


@pytest.fixture
def lib(monkeypatch):
    fake = Library()
    monkeypatch.setattr(_abi, "lib", lambda: fake)
    monkeypatch.setattr(api, "_device_of", lambda t, name: -1)  # (what host tensors answer)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 5, raising=False)
    return fake


def z(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt)


def cache(G=1, **kw):
    sh = (5, PAGE, D_H) if G == 1 else (5, PAGE, G, D_H)
    t = dict(S_K=z(*sh, dt=F8), S_V=z(*sh, dt=F8), R_K=z(5, PAGE, H, R, dt=F8), R_V=z(5, PAGE, H, R, dt=F8),
             E_S_K=z(5, PAGE // BLOCK, G, dt=U8), E_S_V=z(5, PAGE // BLOCK, G, dt=U8),
             E_R_K=z(5, PAGE // BLOCK, H, dt=U8), E_R_V=z(5, PAGE // BLOCK, H, dt=U8))
    return api.ScaledCache(**{**t, **kw})


def rows(dt=BF, n=N):
    return [z(n, D_H, dt=dt), z(n, D_H, dt=dt), z(n, H, R, dt=dt), z(n, H, R, dt=dt)]


def at(**kw):
    t = dict(cu_rows=z(B + 1, dt=I32), start_pos=z(B, dt=I32), page_table=z(B, MAX_PAGES, dt=I32))
    return {**t, **kw}


def write(x=None, c=None, places=None, **kw):
    p = places or at()
    api.write_scaled(*(x or rows()), p["cu_rows"], p["start_pos"], c or cache(), p["page_table"], **kw)


def read(n=N, c=None, places=None, **kw):
    p = places or at()
    return api.read_scaled(p["cu_rows"], p["start_pos"], n, c or cache(), p["page_table"], **kw)


WEIGHTS = dict(W_S_K=(D_H, D), W_S_V=(D_H, D), U_K=(H, R, D), U_V=(H, R, D))


def append(c=None, places=None, X=None, stream=None, ws=None, **w):
    p, t = places or at(), {**{k: z(*s) for k, s in WEIGHTS.items()}, **w}
    api.append_scaled(z(N, D) if X is None else X, p["cu_rows"], p["start_pos"], t["W_S_K"], t["W_S_V"], t["U_K"], t["U_V"],
                      c or cache(), p["page_table"], ws=ws, stream=stream)


def decode(c=None, longest=100, stream=None, ws=None, **t):
    a = {**dict(q=z(B, H, D_H), B_K=z(H, D_H, R), B_V=z(H, D_H, R), seq_lens=z(B, dt=I32),
                page_table=z(B, MAX_PAGES, dt=I32)), **t}
    return api.decode_scaled(a["q"], c or cache(), a["B_K"], a["B_V"], a["seq_lens"], a["page_table"], longest, ws=ws,
                             stream=stream)


def prefill(c=None, places=None, longest=100, stream=None, ws=None, **t):
    p = places or at()
    a = {**dict(X=z(N, D), Q=z(N, H, D_H), B_K=z(H, D_H, R), B_V=z(H, D_H, R), **{k: z(*s) for k, s in WEIGHTS.items()}), **t}
    return api.prefill_scaled(a["X"], a["Q"], p["cu_rows"], p["start_pos"], longest, a["W_S_K"], a["W_S_V"], a["U_K"],
                              a["U_V"], a["B_K"], a["B_V"], c or cache(), p["page_table"], ws=ws, stream=stream)


CALLS = [write, read, append, decode, prefill]


@pytest.mark.parametrize("call,made,outputs", [(write, 0, 0), (read, 4, 4), (append, 1, 0), (decode, 2, 1), (prefill, 2, 1)])
def test_buffers_of_a_call_come_from_its_stream(lib, monkeypatch, call, made, outputs):
    got, current, marked, empty = [], ["here"], [], torch.empty

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream.name)

        def __exit__(self, *exc):
            current.pop()

    def recorded(*args, **kw):
        got.append(current[-1])
        return empty(*args, **kw)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream(current[-1]))
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: recorded(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: marked.append(s.name))
    call(stream=Stream("side"))
    assert got == ["side"] * made and marked == ["here"] * outputs
    assert [args[-1] for _, args in lib.calls] == [Stream.cuda_stream]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field,bad", [
    ("S_K", z(5, PAGE, D_H)), ("S_V", z(5, PAGE, D_H + 16, dt=F8)), ("R_K", z(5, PAGE, H, R, dt=U8)),
    ("R_V", z(4, PAGE, H, R, dt=F8)), ("E_S_K", z(5, 2, 2, dt=U8)), ("E_S_V", z(5, 2, 1, dt=torch.int8)),
    ("E_R_K", z(5, 3, H, dt=U8)), ("E_R_K", z(5, 2, H + 1, dt=U8)), ("E_R_V", z(5, 4, H, dt=U8)),
    ("R_K", z(5, PAGE, R, H, dt=F8).transpose(2, 3)), ("E_R_V", None), ("S_K", z(6, PAGE, D_H, dt=F8))])
def test_caches_that_do_not_fit_are_refused(lib, call, field, bad):
    with pytest.raises((ValueError, TypeError)):
        call(c=cache(**{field: bad}))
    assert not lib.calls


@pytest.mark.parametrize("call", [write, read, append, prefill])
@pytest.mark.parametrize("field,bad", [("cu_rows", z(B, dt=I32)), ("cu_rows", z(B + 1, dt=torch.int64)),
                                       ("start_pos", z(B + 1, dt=I32)), ("page_table", z(B + 1, MAX_PAGES, dt=I32)),
                                       ("page_table", z(B, 2 * MAX_PAGES, dt=I32)[:, ::2]), ("start_pos", None)])
def test_places_that_do_not_fit_are_refused(lib, call, field, bad):
    with pytest.raises((ValueError, TypeError)):
        call(places=at(**{field: bad}))
    assert not lib.calls


@pytest.mark.parametrize("k,bad", [(0, z(N, D_H, dt=torch.float16)), (1, z(N, D_H, dt=torch.float32)), (1, z(N + 1, D_H)),
                                   (2, z(N, H, R + 8)), (2, z(N, R, H).transpose(1, 2)), (3, z(N, 2 * H, R)[:, ::2]),
                                   (0, z(N, 2 * D_H)[:, ::2]), (3, None), (1, z(N, 1, 1, D_H))])
def test_rows_that_do_not_fit_are_refused(lib, k, bad):
    x = rows()
    x[k] = bad
    with pytest.raises((ValueError, TypeError)):
        write(x=x)
    if isinstance(bad, torch.Tensor):
        with pytest.raises((ValueError, TypeError)):
            read(out=x)
    assert not lib.calls


def test_rows_with_a_stride_reach_the_library(lib):
    y = z(N, 2 * D_H + 2 * H * R)
    x = [y[:, :D_H], y[:, D_H:2 * D_H].view(N, 1, D_H), y[:, 2 * D_H:2 * D_H + H * R].unflatten(1, (H, R)), y[:, -H * R:]]
    write(x=x)
    read(out=x)
    for (_, a), first in zip(lib.calls, (0, 8)):
        assert [a[first + 1 + 2 * k] for k in range(4)] == [y.shape[1]] * 4
        assert [a[first + 2 * k] for k in range(4)] == [t.data_ptr() for t in x]


def test_a_single_row_needs_no_stride(lib):
    """torch gives a tensor of one row any stride in that dimension."""
    x = [torch.as_strided(z(4, D_H), (1, D_H), (3, 1)) for _ in range(2)] + rows(n=1)[2:]
    write(x=x)
    assert lib.calls[0][1][1] == D_H and lib.calls[0][1][5] == H * R


@pytest.mark.parametrize("dt,stride", [(BF, D_H + 1), (BF, 3 * D_H + 4), (torch.float32, D_H + 2), (BF, 1 << 40)])
def test_a_single_row_of_any_stride(lib, dt, stride):
    """The distance to a next row that is not there need not be one that the library takes."""
    x = [torch.as_strided(z(2, D_H, dt=dt), (1, D_H), (stride, 1)), torch.as_strided(z(2, D_H, dt=dt), (1, 1, D_H), (stride, 7, 1)),
         torch.as_strided(z(1, H * R, dt=dt), (1, H, R), (stride, R, 1)), z(1, H, R, dt=dt)]
    write(x=x)
    read(n=1, out=x)
    for (_, a), first in zip(lib.calls, (0, 8)):
        assert [a[first + 1 + 2 * k] for k in range(4)] == [D_H, D_H, H * R, H * R]


@pytest.mark.parametrize("call,names", [(decode, ("longest",)), (prefill, ("longest",)), (read, ("n",))])
def test_sizes_past_32_bits_are_refused(lib, call, names):
    for name in names:
        for size in (2 ** 31, 2 ** 32 + 40, -(2 ** 31) - 1):
            with pytest.raises(ValueError):
                call(**{name: size})
    assert not lib.calls


@pytest.mark.parametrize("call,field,bad", [
    (append, "X", z(N, D, dt=torch.float32)), (append, "U_K", z(H, R, D + 8)), (prefill, "Q", z(N, H, D_H + 16)),
    (prefill, "B_V", z(H, R, D_H)), (prefill, "W_S_V", z(2 * D_H, D)), (decode, "q", z(B, H, D_H, dt=torch.float32)),
    (decode, "B_K", z(H, D_H, R + 8)), (decode, "seq_lens", z(B + 1, dt=I32)), (decode, "page_table", z(B + 1, 3, dt=I32)),
    (decode, "q", z(B, D_H, H).transpose(1, 2)), (decode, "ws", z(512)), (append, "ws", z(512)), (prefill, "ws", z(512))])
def test_other_arguments_that_do_not_fit_are_refused(lib, call, field, bad):
    with pytest.raises((ValueError, TypeError)):
        call(**{field: bad})
    assert not lib.calls


def test_empty_needs_whole_blocks():
    with pytest.raises(ValueError):
        api.ScaledCache.empty(2, 64, H, D_H, R, block=48, device="cpu")
    c = api.ScaledCache.empty(2, 64, H, D_H, R, block=32, device="cpu", groups=2)
    assert c.block == 32 and c.groups == 2 and c.E_S_K.shape == (2, 2, 2)


# ---------------------------------------------------------------------------
# The library's own checks, on fake addresses: nothing here is launched
# ---------------------------------------------------------------------------
def desc(**kw):
    d = dict(num_pages=4, page_size=64, H=16, d_h=128, r=48, G=1, block=32, reserved=0, **{
        k: 16 for k in ("S_K", "S_V", "R_K", "R_V", "E_S_K", "E_S_V", "E_R_K", "E_R_V")})
    return ctypes.byref(_abi.ScaledDesc(**{**d, **kw}))


@pytest.fixture(scope="module")
def real():
    from rank_kv_attention_gb300 import build
    build.build()
    return _abi.lib()


BAD_DESC = [(dict(block=24), "SHAPE"), (dict(block=128), "SHAPE"), (dict(block=0), "SHAPE"), (dict(page_size=72), "SHAPE"),
            (dict(page_size=2048, block=64), "SHAPE"), (dict(H=0), "SHAPE"), (dict(H=129), "SHAPE"), (dict(d_h=120), "SHAPE"),
            (dict(r=12), "SHAPE"), (dict(H=3, r=8), "SHAPE"), (dict(G=3), "SHAPE"), (dict(G=-1), "SHAPE"),
            (dict(G=32), "SHAPE"), (dict(num_pages=0), "SHAPE"), (dict(num_pages=2 ** 25), "SHAPE"),
            (dict(S_K=None), "INVALID_ARG"), (dict(E_R_V=None), "INVALID_ARG"), (dict(R_V=24), "INVALID_ARG"),
            (dict(E_S_K=17), "INVALID_ARG"), (dict(reserved=1), "INVALID_ARG")]


def c_write(L, d=None, ld=(128, 128, 768, 768), dtype=1, cu=16, start=16, nreq=2, n=7, table=16, pages=3, x=16):
    a = [v for s in ld for v in (x, s)]
    return L.lrkv_write_scaled(*a, dtype, cu, start, nreq, n, d or desc(), table, pages, None, None)


def c_read(L, d=None, ld=(128, 128, 768, 768), dtype=1, cu=16, start=16, nreq=2, n=7, table=16, pages=3, x=16):
    a = [v for s in ld for v in (x, s)]
    return L.lrkv_read_scaled(d or desc(), cu, start, nreq, n, table, pages, dtype, *a, None, None)


def c_append(L, d=None, cu=16, start=16, nreq=2, n=7, table=16, pages=3, width=64, x=16, ws=256, size=1 << 40):
    return L.lrkv_append_scaled(x, cu, start, nreq, n, width, 16, 16, 16, 16, d or desc(), table, pages, ws, size, None, None)


def c_decode(L, d=None, nreq=2, pages=3, longest=100, q=16, out=16, lens=16, table=16, ws=256, size=1 << 40):
    return L.lrkv_decode_scaled(q, d or desc(), 16, 16, lens, table, nreq, pages, longest, out, ws, size, None, None)


def c_prefill(L, d=None, cu=16, start=16, nreq=2, n=7, table=16, pages=3, width=64, x=16, q=16, longest=100, ws=256,
              size=1 << 40):
    return L.lrkv_prefill_scaled(x, q, cu, start, nreq, n, longest, width, 16, 16, 16, 16, 16, 16, d or desc(), table, pages,
                                 16, ws, size, None, None)


@pytest.mark.parametrize("bad,code", BAD_DESC)
def test_bad_descriptors_are_refused(real, bad, code):
    want = getattr(_abi, "LRKV_E_" + code)
    for call in (c_write, c_read, c_append, c_decode, c_prefill):
        assert call(real, d=desc(**bad)) == want, call
    assert real.lrkv_append_scaled_workspace_bytes(desc(**bad), 7) == 0
    assert real.lrkv_decode_scaled_workspace_bytes(desc(**bad), 2, 100) == 0
    assert real.lrkv_prefill_scaled_workspace_bytes(desc(**bad), 2, 7, 100) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(n=-1), "SHAPE"), (dict(nreq=0), "SHAPE"), (dict(pages=0), "SHAPE"), (dict(pages=2 ** 25), "SHAPE"),
    (dict(nreq=2 ** 30), "SHAPE"), (dict(n=2 ** 31 - 1), "SHAPE"), (dict(cu=None), "INVALID_ARG"),
    (dict(start=None), "INVALID_ARG"), (dict(table=None), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"),
    (dict(x=8), "INVALID_ARG")])
def test_bad_rows_are_refused(real, bad, code):
    for call in (c_write, c_read, c_append, c_prefill):
        assert call(real, **bad) == getattr(_abi, "LRKV_E_" + code), call


def test_bad_strides_and_types_are_refused(real):
    for call in (c_write, c_read):
        for ld in ((120, 128, 768, 768), (128, 132, 768, 768), (128, 128, 760, 768), (128, 128, 768, -768)):
            assert call(real, ld=ld) == _abi.LRKV_E_SHAPE
        assert call(real, ld=(132, 128, 768, 772), dtype=1) == _abi.LRKV_E_SHAPE   # bf16 rows begin at 16 bytes
        for dt in (2, 3, -1):
            assert call(real, dtype=dt) == _abi.LRKV_E_DTYPE and call(real, dtype=dt, n=0) == _abi.LRKV_E_DTYPE


@pytest.mark.parametrize("call", [c_write, c_read, c_append, c_prefill])
def test_no_rows_is_a_call_without_work(real, call):
    kw = {} if call in (c_write, c_read) else dict(ws=None, size=0)
    assert call(real, n=0, cu=None, start=None, table=None, x=None, **kw) == _abi.LRKV_OK


def test_bad_decode_sizes_are_refused(real):
    S, A, W = _abi.LRKV_E_SHAPE, _abi.LRKV_E_INVALID_ARG, _abi.LRKV_E_WORKSPACE
    for kw, code in ((dict(nreq=0), S), (dict(pages=0), S), (dict(longest=0), S), (dict(longest=193), _abi.LRKV_E_BOUNDS),
                     (dict(nreq=2 ** 28), S), (dict(q=None), A), (dict(out=8), A), (dict(lens=None), A), (dict(table=None), A),
                     (dict(ws=None), W), (dict(ws=128), W), (dict(size=100), W)):
        assert c_decode(real, **kw) == code, kw


def test_bad_projection_and_prefill_sizes_are_refused(real):
    S, A, W = _abi.LRKV_E_SHAPE, _abi.LRKV_E_INVALID_ARG, _abi.LRKV_E_WORKSPACE
    for kw, code in ((dict(width=0), S), (dict(width=60), S), (dict(width=65544), S), (dict(ws=None), W), (dict(ws=64), W),
                     (dict(size=100), W)):
        assert c_append(real, **kw) == code and c_prefill(real, **kw) == code, kw
    for kw, code in ((dict(longest=0), S), (dict(longest=193), _abi.LRKV_E_BOUNDS), (dict(q=None), A), (dict(q=8), A)):
        assert c_prefill(real, **kw) == code, kw


def test_workspaces_grow_with_the_call(real):
    for d in (desc(), desc(H=6, r=40, d_h=32), desc(H=32, r=32), desc(G=2), desc(r=72)):
        last = 0
        for nreq in (1, 2, 3, 7, 64, 500):
            row = [real.lrkv_decode_scaled_workspace_bytes(d, nreq, n) for n in (1, 64, 65, 1000, 30000, 10 ** 6)]
            assert row == sorted(row) and row[0] > 0 and row[-1] >= last
            last = row[-1]
    assert real.lrkv_append_scaled_workspace_bytes(desc(), 100) >= 100 * 4 * 1792


def test_workspaces_of_the_largest_sizes(real):
    """The queries take any int32: the bytes of few requests neither fall nor run away where a length comes near 2^31."""
    for d in (desc(), desc(H=6, r=40, d_h=32), desc(G=2), desc(r=72)):
        for call in (lambda n: real.lrkv_decode_scaled_workspace_bytes(d, 3, n),
                     lambda n: real.lrkv_prefill_scaled_workspace_bytes(d, 3, 50, n)):
            sizes = [call(n) for n in (2 ** 20, 2 ** 30, 2 ** 31 - 200, 2 ** 31 - 1)]
            assert sizes == sorted(sizes) and 0 < sizes[0] and sizes[-1] < 2 ** 40, sizes


@pytest.mark.parametrize("B,n,max_ctx", [(8, 16384, 2048), (1, 512, 40000), (4, 100, 700), (3, 5, 9000)])
def test_prefill_workspace_holds_one_part_at_a_time(real, B, n, max_ctx):
    """The projected rows are done with when the values are laid out (or the rows' decode begins): one part over the other."""
    for kw in (dict(), dict(page_size=32), dict(r=72)):
        d, width = desc(num_pages=2 ** 14, **kw), 2 * (128 + 16 * kw.get("r", 48))
        tiled = not kw
        rows = min(B * -(-max_ctx // 64) * 64, 2 ** 14 * 64)
        staged = n * width * 4 + 4 * 256
        later = rows * width * 2 + 4 * B * -(-max_ctx // 64) + 5 * 256 if tiled else \
            real.lrkv_decode_scaled_workspace_bytes(d, n, max_ctx) + 8 * n + 2 * 256
        assert real.lrkv_prefill_scaled_workspace_bytes(d, B, n, max_ctx) <= max(staged, later)
