"""What the binding does around a library call (most of it for the windowed
operators), on host tensors and a library that only records what it is asked.  No call here
touches a GPU."""
import ctypes

import pytest
import torch

from rank_kv_attention_gb300 import _abi, api

H, D_H, R, PAGE, B, MAX_PAGES, N, D = 4, 128, 16, 64, 2, 3, 7, 64


class Stream:
    cuda_stream = 77

    def __init__(self, name):
        self.name = name


class Library:
    """Entry points that record their arguments; a sizing query answers 512, a call without a workspace asks for one."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("_bytes"):
                return 512
            self.calls.append((name, args))
            # (address and size of the workspace: fourth and third argument from the end)
            return _abi.LRKV_E_WORKSPACE if name.endswith("_window") and args[-4] is None else _abi.LRKV_OK
        return entry


@pytest.fixture
def lib(monkeypatch):
    fake = Library()
    monkeypatch.setattr(_abi, "lib", lambda: fake)
    monkeypatch.setattr(api, "_device_of", lambda t, name: -1)  # (what host tensors answer)
    return fake


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def cache():
    return api.PagedCache(bf(5, PAGE, D_H), bf(5, PAGE, D_H), bf(5, PAGE, H, R), bf(5, PAGE, H, R))


def decode(longest=100, window=40, sinks=2, **kw):
    return api.decode_window(bf(B, H, D_H), cache(), bf(H, D_H, R), bf(H, D_H, R), i32(B), i32(B, MAX_PAGES), longest, window,
                             sinks, **kw)


def prefill(longest=100, window=40, sinks=2, **kw):
    return api.prefill_window(bf(N, D), bf(N, H, D_H), i32(B + 1), i32(B), longest, bf(D_H, D), bf(D_H, D), bf(H, R, D),
                              bf(H, R, D), bf(H, D_H, R), bf(H, D_H, R), cache(), i32(B, MAX_PAGES), window, sinks, **kw)


def plan(page=PAGE, rows=9, window=40, sinks=2, **kw):
    return api.page_plan(i32(B), i32(B), i32(B, MAX_PAGES), i32(5), i32(1), page, rows, window=window, sinks=sinks, **kw)


def full_decode(**kw):
    return api.decode(bf(B, H, D_H), cache(), bf(H, D_H, R), bf(H, D_H, R), i32(B), i32(B, MAX_PAGES), 100, **kw)


def full_step(**kw):
    return api.decode_step(bf(B, D), bf(D_H, D), bf(D_H, D), bf(H, R, D), bf(H, R, D), bf(B, H, D_H), cache(),
                           bf(H, D_H, R), bf(H, D_H, R), i32(B), i32(B, MAX_PAGES), 100, **kw)


def full_prefill(**kw):
    return api.prefill(bf(N, D), bf(N, H, D_H), i32(B + 1), i32(B), 100, bf(D_H, D), bf(D_H, D), bf(H, R, D), bf(H, R, D),
                       bf(H, D_H, R), bf(H, D_H, R), cache(), i32(B, MAX_PAGES), **kw)


def table():
    return api.RopeTable(torch.zeros(4, dtype=torch.uint8), D_H, 100)


def rope_decode(**kw):
    return api.decode_rope(bf(B, H, D_H), cache(), bf(H, D_H, R), bf(H, D_H, R), i32(B), i32(B, MAX_PAGES), 100, table(), **kw)


def rope_prefill(**kw):
    return api.prefill_rope(bf(N, D), bf(N, H, D_H), i32(B + 1), i32(B), 100, bf(D_H, D), bf(D_H, D), bf(H, R, D),
                            bf(H, R, D), bf(H, D_H, R), bf(H, D_H, R), cache(), i32(B, MAX_PAGES), table(), **kw)


def rope_table(stream):
    return api.rope_table(D_H, 100, device="cpu", stream=stream)


@pytest.mark.parametrize("call,made,outputs", [(decode, 2, 1), (prefill, 2, 1), (plan, 2, 2), (full_decode, 2, 1),
                                               (full_step, 2, 1), (full_prefill, 2, 1), (rope_decode, 2, 1),
                                               (rope_prefill, 2, 1), (rope_table, 1, 1)])
def test_buffers_of_a_call_come_from_its_stream(lib, monkeypatch, call, made, outputs):
    """Whatever a call on another stream allocates (outputs and scratch) comes from that stream's memory, and outputs
    wait for the current stream before they are reused."""
    at, current, marked, empty, need = [], ["here"], [], torch.empty, api._need

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream.name)

        def __exit__(self, *exc):
            current.pop()

    def recorded(*args, **kw):
        at.append(current[-1])
        return empty(*args, **kw)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream(current[-1]))
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: recorded(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: marked.append(s.name))
    monkeypatch.setattr(api, "_need", lambda t, name, dtype=None, device=True: need(t, name, dtype, False))
    call(stream=Stream("side"))
    assert at == ["side"] * made
    assert marked == ["here"] * outputs
    assert all(getattr(args[-1], "value", args[-1]) == Stream.cuda_stream for _, args in lib.calls)


WRAPS = [2 ** 31, 2 ** 32 + 40, -(2 ** 31) - 1, -(2 ** 32) + 40, -(2 ** 33)]


@pytest.mark.parametrize("size", WRAPS)
@pytest.mark.parametrize("call,names", [(decode, ("longest", "window", "sinks")), (prefill, ("longest", "window", "sinks")),
                                        (plan, ("page", "rows", "window", "sinks"))])
def test_sizes_past_32_bits_are_refused(lib, call, names, size):
    """A size that would wrap is refused, also a negative one (2^32 below a valid one) and also beside a negative one."""
    for name in names:
        with pytest.raises(ValueError):
            call(**{name: size})
        for other in set(names) - {name, "rows"}:
            with pytest.raises(ValueError):
                call(**{name: size, other: -1})
        if call is decode:
            sizes = dict(dict(longest=100, window=40, sinks=2), **{name: size})
            with pytest.raises(ValueError):
                api.decode_window_workspace_bytes(B, H, D_H, R, sizes["longest"], sizes["window"], sizes["sinks"])
    assert not lib.calls


def test_sizes_within_32_bits_reach_the_library(lib, monkeypatch):
    """Refusing them is the library's part."""
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 5, raising=False)
    for size in (2 ** 31 - 1, -1, -(2 ** 31)):
        decode(window=size, sinks=size, longest=size, ws=torch.empty(512, dtype=torch.uint8))
        prefill(window=size, sinks=size, longest=size, ws=torch.empty(512, dtype=torch.uint8))
        plan(window=size, sinks=size, page=size)
    assert [len(lib.calls), {args[-1] for _, args in lib.calls}] == [9, {5}]


def test_prefill_is_bounded_by_its_window():
    """Rows times context may pass 2^30 where each row sees a window of it; the full prefill counts those rows in 32 bits."""
    from rank_kv_attention_gb300 import build
    build.build()
    real, desc = _abi.lib(), ctypes.byref(_abi.CacheDesc(16, 16, 16, 16, 40, 64, 4, 32, 8, _abi.LRKV_F32))

    def call(n, ctx, window):
        head = (16, 16, 16, 16, 2, n, ctx, 64, 16, 16, 16, 16, 16, 16, desc, 16, 1 << 20)
        if window:
            return real.lrkv_prefill_window(*head, window, 4, 16, None, 0, None, None)
        return real.lrkv_prefill(*head, 16, None, 0, None, None)
    # (an fp32 call always needs a workspace: a call that passes its checks asks for it, and nothing is launched)
    for n, ctx in ((8200, 139272), (65535 * 32, 1 << 26), (1, 1 << 26)):
        assert call(n, ctx, 1024) == _abi.LRKV_E_WORKSPACE, (n, ctx)
    for n, ctx in ((65535 * 32 + 1, 64), (2 ** 30, 64), (2 ** 31 - 1, 1)):
        assert call(n, ctx, 1024) == _abi.LRKV_E_SHAPE, (n, ctx)
    assert call(8200, 139272, 0) == _abi.LRKV_E_SHAPE and call(8200, 64, 0) == _abi.LRKV_E_WORKSPACE
