"""Windowed attention and the page plan: the definitions of oracle/window.py
against hand-worked cases, and every refusal of the entry points.  No call
here touches a GPU."""
import ctypes

import numpy as np
import pytest

import oracle
import oracle.window as W
from rank_kv_attention_gb300 import _abi
from rank_kv_attention_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _abi.lib()


def test_visible_rows():
    assert W.visible(0, 1, 0) == [0]
    assert W.visible(9, 3, 2) == [0, 1, 7, 8, 9]
    assert W.visible(9, 1, 0) == [9]
    assert W.visible(4, 3, 2) == [0, 1, 2, 3, 4]          # sinks reach the window
    assert W.visible(3, 100, 50) == [0, 1, 2, 3]


def test_full_window_is_the_plain_decode():
    rng = np.random.default_rng(0)
    H, d_h, r, ps, L = 2, 8, 4, 16, 21
    pools = [rng.standard_normal(s) for s in ((2, ps, d_h), (2, ps, d_h), (2, ps, H, r), (2, ps, H, r))]
    bases = [rng.standard_normal((H, d_h, r)) for _ in range(2)]
    q = rng.standard_normal((1, H, d_h))
    ref = oracle.decode(q, *pools, *bases, np.array([[1, 0]]), [L], ps)
    got = W.attend_query(q[0], *pools, *bases, [1, 0], L - 1, ps, 21, 0)
    assert np.allclose(got, ref[0], rtol=0, atol=1e-14)
    assert not np.allclose(W.attend_query(q[0], *pools, *bases, [1, 0], L - 1, ps, 20, 0), ref[0], atol=1e-6)
    # window 1 without sinks: the value of the query's own row
    own = pools[1][0, 4] + np.einsum("hr,hdr->hd", pools[3][0, 4], bases[1])
    assert np.allclose(W.attend_query(q[0], *pools, *bases, [1, 0], L - 1, ps, 1, 0), own, atol=1e-14)


def test_plan_by_hand():
    # two requests of pages of 16 rows, window 20, one sink: request 0 grows 60 -> 70, request 1 ends with 30 rows
    table = np.array([[7, 3, 4, 5, -1], [8, 9, -1, -1, -1]], np.int32)
    p = W.page_plan([60, 30], [10, -1], table, [0, 1, 2], 16, 12, 20, 1, 50)
    assert p["seq_lens"] == [70, 0] and p["cu_rows"] == [0, 10, 10]
    assert p["page_table"][0].tolist() == [7, 3, 4, 5, 2]     # page 4 comes off the end of the list
    assert p["slots"] == [5 * 16 + 12 + i for i in range(4)] + [2 * 16 + i for i in range(6)]
    # queries from 70 on see rows > 50: pages 1 and 2 (rows 16 .. 47) are gone; at 60 they saw rows > 40, page 1
    # (rows 16 .. 31) was gone before, so this step releases page 2
    assert p["free"] == [0, 1, 4, 8, 9]


WS = ctypes.c_void_p(256)


def _cache(dtype=1, **kw):
    c = _abi.CacheDesc(16, 16, 16, 16, 4, 64, 16, 128, 48, dtype)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_decode_window_refusals(lib):
    good = dict(q=16, BK=16, BV=16, sl=16, pt=16, B=2, mp=4, msl=100, win=64, snk=4, out=16, ws=WS, wsb=1 << 30)

    def call(cache=None, **over):
        a = dict(good, **over)
        return lib.lrkv_decode_window(a["q"], ctypes.byref(cache or _cache()), a["BK"], a["BV"], a["sl"], a["pt"],
                                      a["B"], a["mp"], a["msl"], a["win"], a["snk"], a["out"], a["ws"], a["wsb"],
                                      None, None)
    for name in ("q", "BK", "BV", "sl", "pt", "out"):
        assert call(**{name: None}) == _abi.LRKV_E_INVALID_ARG, name
    for name in ("q", "BK", "BV", "out"):
        assert call(**{name: 8}) == _abi.LRKV_E_INVALID_ARG, name
    for over in (dict(win=0), dict(win=-1), dict(snk=-1), dict(B=0), dict(mp=0), dict(msl=0), dict(mp=1 << 26),
                 dict(B=1 << 30, win=1 << 20)):
        assert call(**over) == _abi.LRKV_E_SHAPE, over
    assert call(msl=4 * 64 + 1) == _abi.LRKV_E_BOUNDS
    assert call(_cache(dtype=5)) == _abi.LRKV_E_DTYPE
    assert call(_cache(d_h=130)) == _abi.LRKV_E_SHAPE
    assert call(_cache(G=3)) == _abi.LRKV_E_SHAPE
    assert call(_cache(S_K=None)) == _abi.LRKV_E_INVALID_ARG
    assert lib.lrkv_decode_window(16, None, 16, 16, 16, 16, 2, 4, 100, 64, 4, 16, WS, 1 << 30, None, None) \
        == _abi.LRKV_E_INVALID_ARG
    # a workspace is checked for its alignment even where none is needed
    assert call(_cache(H=4), ws=ctypes.c_void_p(16)) == _abi.LRKV_E_WORKSPACE


def test_decode_window_workspace(lib):
    f = lib.lrkv_decode_window_workspace_bytes
    assert f(4, 6, 32, 8, 4096, 1024, 4, 0) == 0          # one launch, no scratch
    assert f(4, 6, 32, 8, 1 << 20, 2 ** 31 - 1, 2 ** 31 - 1, 0) == 0
    for bad in ((0, 6, 32, 8, 64, 64, 0, 0), (4, 6, 32, 8, 0, 64, 0, 0), (4, 6, 32, 8, 64, 0, 0, 0),
                (4, 6, 32, 8, 64, 64, -1, 0), (4, 6, 33, 8, 64, 64, 0, 0), (4, 6, 32, 8, 64, 64, 0, 9)):
        assert f(*bad) == 0, bad


def test_prefill_window_refusals(lib):
    good = dict(X=16, Q=16, cu=16, sp=16, B=2, n=10, ctx=100, d=64, w=16, BK=16, BV=16, pt=16, mp=4, win=64, snk=4,
                out=16, ws=WS, wsb=1 << 40)

    def call(cache=None, **over):
        a = dict(good, **over)
        return lib.lrkv_prefill_window(a["X"], a["Q"], a["cu"], a["sp"], a["B"], a["n"], a["ctx"], a["d"], a["w"], a["w"],
                                       a["w"], a["w"], a["BK"], a["BV"], ctypes.byref(cache or _cache()), a["pt"], a["mp"],
                                       a["win"], a["snk"], a["out"], a["ws"], a["wsb"], None, None)
    for name in ("X", "Q", "cu", "sp", "w", "BK", "BV", "pt", "out"):
        assert call(**{name: None}) == _abi.LRKV_E_INVALID_ARG, name
    for name in ("X", "Q", "w", "BK", "BV", "out"):
        assert call(**{name: 8}) == _abi.LRKV_E_INVALID_ARG, name
    for over in (dict(win=0), dict(win=-5), dict(snk=-1), dict(B=0), dict(mp=0), dict(n=-1), dict(ctx=0), dict(d=0), dict(d=63)):
        assert call(**over) == _abi.LRKV_E_SHAPE, over
    assert call(ctx=4 * 64 + 1) == _abi.LRKV_E_BOUNDS
    assert call(ws=None) == _abi.LRKV_E_WORKSPACE and call(wsb=64) == _abi.LRKV_E_WORKSPACE
    assert call(_cache(r=50)) == _abi.LRKV_E_SHAPE
    assert call(n=0) == _abi.LRKV_OK          # nothing to do


def test_page_plan_refusals(lib):
    names = ("sl", "nr", "pt", "fp", "nf", "so", "cu", "fo", "no")
    good = dict({k: 1024 * (i + 1) for i, k in enumerate(names)}, B=2, mp=4, ps=64, num=10, win=100, snk=4, rows=8,
                pos=16, ids=32, slots=48)

    def call(**over):
        a = dict(good, **over)
        return lib.lrkv_page_plan(a["sl"], a["nr"], a["B"], a["mp"], a["ps"], a["num"], a["win"], a["snk"], a["rows"],
                                  a["pt"], a["fp"], a["nf"], a["so"], a["cu"], a["pos"], a["ids"], a["slots"], a["fo"],
                                  a["no"], None, None)
    for name in names + ("pos", "ids", "slots"):
        assert call(**{name: None}) == _abi.LRKV_E_INVALID_ARG, name
    for over in (dict(B=0), dict(mp=0), dict(num=0), dict(rows=-1), dict(win=-1), dict(snk=-1), dict(ps=0), dict(ps=24),
                 dict(ps=2048), dict(mp=1 << 28), dict(num=1 << 28), dict(rows=2 ** 31 - 1)):
        assert call(**over) == _abi.LRKV_E_SHAPE, over
    for i in ("sl", "nr", "fp", "nf"):        # an output on top of an input
        for o in ("so", "cu", "fo", "no"):
            assert call(**{o: good[i]}) == _abi.LRKV_E_INVALID_ARG, (i, o)


def test_page_plan_refuses_tables_past_32_bit_counts(lib):
    """B * max_pages bounds the pages that a step can release; every array on its own lies in range."""
    p = [1024 * (i + 1) for i in range(12)]

    def call(B, max_pages, out=p[5]):
        return lib.lrkv_page_plan(p[0], p[1], B, max_pages, 16, 10, 100, 4, 8, p[2], p[3], p[4], p[6], p[7], out, p[8],
                                  p[9], p[10], p[11], None, None)
    assert call(1 << 12, 1 << 18) == _abi.LRKV_E_SHAPE
    assert call(2 ** 31 - 1, 1) == _abi.LRKV_E_SHAPE
    for i in range(2):
        assert call(2, 4, out=p[i]) == _abi.LRKV_E_INVALID_ARG  # positions on top of an input


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch

    from rank_kv_attention_gb300 import api
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    cache = api.PagedCache(z(2, 64, 128), z(2, 64, 128), z(2, 64, 16, 48), z(2, 64, 16, 48))
    with pytest.raises((ValueError, TypeError)):
        api.decode_window(z(1, 16, 128), cache, z(16, 128, 48), z(16, 128, 48), i(1), i(1, 2), 64, 10)
    with pytest.raises(ValueError):
        api.decode_window(z(16, 128), cache, z(16, 128, 48), z(16, 128, 48), i(1), i(1, 2), 64, 10)
    with pytest.raises(ValueError):
        api.prefill_window(z(4), z(4, 16, 128), i(2), i(1), 64, *[z(1)] * 6, cache, i(1, 2), 10)
    with pytest.raises((ValueError, TypeError)):
        api.page_plan(i(2), i(2), i(2, 4), i(8), i(1), 64, 4)
    with pytest.raises(ValueError):
        api.page_plan(i(2, 2), i(2), i(2, 4), i(8), i(1), 64, 4)
