"""PyTorch-facing binding of the LRKV C ABI.

Every function here only checks tensor properties, builds the C arguments
and calls the library on the current CUDA stream, or on `stream`: inputs have
to be ready there, a reader on another stream waits for it as with any work of
two streams, and what a call allocates for itself is in order on it.  All
arithmetic runs in the library's CUDA kernels.  Tensors must be contiguous CUDA tensors of the
cache's dtype (torch.bfloat16 or torch.float32); integer metadata is int32.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import NamedTuple

import torch

from . import _abi

_DT = {torch.float32: _abi.LRKV_F32, torch.bfloat16: _abi.LRKV_BF16,
       torch.float8_e4m3fn: _abi.LRKV_FP8_E4M3}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype=None, device=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


@dataclass
class PagedCache:
    """Caller-owned paged factored cache (four pools sharing page ids).

    S_K, S_V: [num_pages, page_size, d_h], or [num_pages, page_size, G, d_h]
    for G shared groups (head h reads group h // (H // G)); R_K, R_V:
    [num_pages, page_size, H, r].
    Pools of torch.float8_e4m3fn hold 8-bit codes whose values are the codes
    times ``scale`` (one scale per pool: S_K, S_V, R_K, R_V); the activations
    used with such a cache are bf16.  ``N_K`` ([num_pages, page_size, H] in
    the activation dtype, or None) holds the reciprocal joint key norms with
    ``norm_eps`` (see lrkv_key_norms).
    """
    S_K: torch.Tensor
    S_V: torch.Tensor
    R_K: torch.Tensor
    R_V: torch.Tensor
    scale: tuple = (1.0, 1.0, 1.0, 1.0)
    N_K: "torch.Tensor | None" = None
    norm_eps: float = 0.0

    @classmethod
    def empty(cls, num_pages, page_size, H, d_h, r, dtype=torch.bfloat16, device="cuda", groups=1):
        mk = lambda *s: torch.empty(s, dtype=dtype, device=device)
        sh = (num_pages, page_size, d_h) if groups == 1 else (num_pages, page_size, groups, d_h)
        return cls(mk(*sh), mk(*sh), mk(num_pages, page_size, H, r), mk(num_pages, page_size, H, r))

    @property
    def groups(self):
        """Shared key/value groups (1: one shared basis)."""
        return self.S_K.shape[2] if self.S_K.dim() == 4 else 1

    @property
    def dtype(self):
        return self.S_K.dtype

    @property
    def act_dtype(self):
        """dtype of every other floating tensor used with this cache."""
        return torch.bfloat16 if self.dtype == torch.float8_e4m3fn else self.dtype

    def desc(self) -> _abi.CacheDesc:
        for n in ("S_K", "S_V", "R_K", "R_V"):
            _need(getattr(self, n), n, self.dtype)
        npg, ps, d_h = self.S_K.shape[0], self.S_K.shape[1], self.S_K.shape[-1]
        _, _, H, r = self.R_K.shape
        if tuple(self.S_V.shape) != tuple(self.S_K.shape):
            raise ValueError("S_K and S_V must have the same shape")
        if self.N_K is not None:
            _need(self.N_K, "N_K", self.act_dtype)
            if tuple(self.N_K.shape) != (npg, ps, H):
                raise ValueError(f"N_K must be [{npg}, {ps}, {H}], got {tuple(self.N_K.shape)}")
        return _abi.CacheDesc(self.S_K.data_ptr(), self.S_V.data_ptr(), self.R_K.data_ptr(),
                              self.R_V.data_ptr(), npg, ps, H, d_h, r, _DT[self.dtype],
                              (ctypes.c_float * 4)(*[float(x) for x in self.scale]),
                              self.N_K.data_ptr() if self.N_K is not None else None,
                              float(self.norm_eps), self.groups)


def prefill_kernel_kind(cache: PagedCache) -> int:
    """LRKV_PREFILL_TILED or LRKV_PREFILL_PER_ROW: the attention kernel
    lrkv_prefill runs for this cache."""
    L = _abi.lib()
    st = L.lrkv_prefill_kernel_kind(ctypes.byref(cache.desc()))
    if st < 0:
        raise _abi.LrkvError("lrkv_prefill_kernel_kind", st, L)
    return st


def cache_bytes(H, d_h, r, tokens, dtype=torch.bfloat16, groups=1) -> int:
    return int(_abi.lib().lrkv_cache_bytes_grouped(H, d_h, r, groups, tokens, _DT[dtype]))


def decode_workspace_bytes(B, H, d_h, r, max_seq_len, dtype=torch.bfloat16) -> int:
    return int(_abi.lib().lrkv_decode_workspace_bytes(B, H, d_h, r, max_seq_len, _DT[dtype]))


def prefill_workspace_bytes(B, n, H, d_h, r, max_ctx, dtype=torch.bfloat16) -> int:
    return int(_abi.lib().lrkv_prefill_workspace_bytes(B, n, H, d_h, r, max_ctx, _DT[dtype]))


def workspace(nbytes, device="cuda") -> torch.Tensor:
    """A byte buffer usable as workspace (torch allocations are 256-byte aligned)."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _own_buffer(shape, dtype, dev, stream, scratch=False):
    """A buffer made for a call on `stream`, from that stream's memory: work still
    queued on the current stream cannot hold it.  Unless it is scratch, it is
    not reused before the current stream, where the result is read, has passed
    the point at which it is freed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if not scratch:
        t.record_stream(here)
    return t


def _scratch(nbytes, dev, stream):
    """A workspace made for a call on `stream`."""
    return _own_buffer((max(int(nbytes), 1),), torch.uint8, dev, stream, scratch=True)


def append(X, positions, seq_ids, W_S_K, W_S_V, U_K, U_V, cache: PagedCache, page_table,
           status=None, stream=None):
    """lrkv_append: project rows X and store them at (seq_ids, positions)."""
    dt = cache.act_dtype
    for n, t in (("X", X), ("W_S_K", W_S_K), ("W_S_V", W_S_V), ("U_K", U_K), ("U_V", U_V)):
        _need(t, n, dt)
    for n, t in (("positions", positions), ("seq_ids", seq_ids), ("page_table", page_table)):
        _need(t, n, torch.int32)
    if status is not None:
        _need(status, "status", torch.int32)
    n, d = X.shape
    B, max_pages = page_table.shape
    desc = cache.desc()
    code = _abi.lib().lrkv_append(_ptr(X), _ptr(positions), _ptr(seq_ids), n, d, _ptr(W_S_K),
                                  _ptr(W_S_V), _ptr(U_K), _ptr(U_V), ctypes.byref(desc),
                                  _ptr(page_table), B, max_pages, _ptr(status), _stream(stream))
    _abi.check("lrkv_append", code)


def decode(q, cache: PagedCache, B_K, B_V, seq_lens, page_table, max_seq_len, out=None,
           ws=None, status=None, stream=None):
    """lrkv_decode: per-head attention output [B, H, d_h] of one decode step."""
    dt = cache.act_dtype
    for n, t in (("q", q), ("B_K", B_K), ("B_V", B_V)):
        _need(t, n, dt)
    _need(seq_lens, "seq_lens", torch.int32)
    _need(page_table, "page_table", torch.int32)
    B, H, d_h = q.shape
    r = cache.R_K.shape[3]
    if out is None:
        out = _own_buffer(q.shape, dt, q.device, stream)
    _need(out, "out", dt)
    need = decode_workspace_bytes(B, H, d_h, r, max_seq_len, dt)
    if ws is None:
        ws = _scratch(need, q.device, stream)
    _need(ws, "ws", torch.uint8)
    desc = cache.desc()
    code = _abi.lib().lrkv_decode(_ptr(q), ctypes.byref(desc), _ptr(B_K), _ptr(B_V),
                                  _ptr(seq_lens), _ptr(page_table), B, page_table.shape[1],
                                  max_seq_len, _ptr(out), _ptr(ws), ws.numel(), _ptr(status),
                                  _stream(stream))
    _abi.check("lrkv_decode", code)
    return out


def decode_step_workspace_bytes(B, H, d_h, r, max_seq_len, dtype=torch.bfloat16) -> int:
    return _abi.lib().lrkv_decode_step_workspace_bytes(B, H, d_h, r, max_seq_len, _DT[dtype])


def decode_step(X, W_S_K, W_S_V, U_K, U_V, q, cache: PagedCache, B_K, B_V, seq_lens, page_table,
                max_seq_len, out=None, ws=None, status=None, stream=None):
    """lrkv_decode_step: append each request's new row X[b] at position
    seq_lens[b] - 1, then decode; returns out [B, H, d_h]."""
    dt = cache.act_dtype
    for n, t in (("X", X), ("W_S_K", W_S_K), ("W_S_V", W_S_V), ("U_K", U_K), ("U_V", U_V),
                 ("q", q), ("B_K", B_K), ("B_V", B_V)):
        _need(t, n, dt)
    _need(seq_lens, "seq_lens", torch.int32)
    _need(page_table, "page_table", torch.int32)
    B, H, d_h = q.shape
    r = cache.R_K.shape[3]
    if out is None:
        out = _own_buffer(q.shape, dt, q.device, stream)
    _need(out, "out", dt)
    need = decode_step_workspace_bytes(B, H, d_h, r, max_seq_len, dt)
    if ws is None:
        ws = _scratch(need, q.device, stream)
    _need(ws, "ws", torch.uint8)
    desc = cache.desc()
    code = _abi.lib().lrkv_decode_step(_ptr(X), X.shape[1], _ptr(W_S_K), _ptr(W_S_V), _ptr(U_K),
                                       _ptr(U_V), _ptr(q), ctypes.byref(desc), _ptr(B_K), _ptr(B_V),
                                       _ptr(seq_lens), _ptr(page_table), B, page_table.shape[1],
                                       max_seq_len, _ptr(out), _ptr(ws), ws.numel(), _ptr(status),
                                       _stream(stream))
    _abi.check("lrkv_decode_step", code)
    return out


def decode_step_host_workspace_bytes(B, H, d_h, r, d, max_seq_len, dtype=torch.bfloat16) -> int:
    return _abi.lib().lrkv_decode_step_host_workspace_bytes(B, H, d_h, r, d, max_seq_len, _DT[dtype])


def decode_step_host(X, W_S_K, W_S_V, U_K, U_V, q, cache: PagedCache, B_K, B_V, seq_lens,
                     page_table, max_seq_len, out=None, ws=None, status=None, stream=None):
    """lrkv_decode_step_host: the decode step with X, q, seq_lens and out in
    host memory (CPU tensors, best pinned); the copies and the step are
    enqueued on the stream, which the caller synchronises before reading out."""
    dt = cache.act_dtype
    for n, t in (("X", X), ("q", q)):
        _need(t, n, dt, device=False)
        if t.is_cuda:
            raise ValueError(f"{n} must be a host tensor")
    _need(seq_lens, "seq_lens", torch.int32, device=False)
    if seq_lens.is_cuda:
        raise ValueError("seq_lens must be a host tensor")
    for n, t in (("W_S_K", W_S_K), ("W_S_V", W_S_V), ("U_K", U_K), ("U_V", U_V), ("B_K", B_K),
                 ("B_V", B_V)):
        _need(t, n, dt)
    _need(page_table, "page_table", torch.int32)
    B, H, d_h = q.shape
    r = cache.R_K.shape[3]
    d = X.shape[1]
    if out is None:
        out = torch.empty(q.shape, dtype=dt, pin_memory=True)
    _need(out, "out", dt, device=False)
    if out.is_cuda:
        raise ValueError("out must be a host tensor")
    need = decode_step_host_workspace_bytes(B, H, d_h, r, d, max_seq_len, dt)
    if ws is None:
        ws = _scratch(need, page_table.device, stream)
    _need(ws, "ws", torch.uint8)
    desc = cache.desc()
    code = _abi.lib().lrkv_decode_step_host(_ptr(X), d, _ptr(W_S_K), _ptr(W_S_V), _ptr(U_K),
                                            _ptr(U_V), _ptr(q), ctypes.byref(desc), _ptr(B_K),
                                            _ptr(B_V), _ptr(seq_lens), _ptr(page_table), B,
                                            page_table.shape[1], max_seq_len, _ptr(out), _ptr(ws),
                                            ws.numel(), _ptr(status), _stream(stream))
    _abi.check("lrkv_decode_step_host", code)
    return out


class StepGraph:
    """lrkv_step_graph_*: the host-buffer decode step recorded once as a
    CUDA graph and replayed with one launch per step.  The graph keeps every
    tensor it was made with (held here so they stay allocated): refill X, q
    and seq_lens (pinned host tensors) between steps, launch, synchronise
    the stream, then read out."""

    def __init__(self, X, W_S_K, W_S_V, U_K, U_V, q, cache: PagedCache, B_K, B_V, seq_lens,
                 page_table, max_seq_len, out=None, ws=None, status=None):
        dt = cache.act_dtype
        for n, t in (("X", X), ("q", q)):
            _need(t, n, dt, device=False)
            if t.is_cuda or not t.is_pinned():
                raise ValueError(f"{n} must be a pinned host tensor")
        _need(seq_lens, "seq_lens", torch.int32, device=False)
        if seq_lens.is_cuda or not seq_lens.is_pinned():
            raise ValueError("seq_lens must be a pinned host tensor")
        for n, t in (("W_S_K", W_S_K), ("W_S_V", W_S_V), ("U_K", U_K), ("U_V", U_V),
                     ("B_K", B_K), ("B_V", B_V)):
            _need(t, n, dt)
        _need(page_table, "page_table", torch.int32)
        B, H, d_h = q.shape
        r, d = cache.R_K.shape[3], X.shape[1]
        if out is None:
            out = torch.empty(q.shape, dtype=dt, pin_memory=True)
        if out.is_cuda or not out.is_pinned():
            raise ValueError("out must be a pinned host tensor")
        _need(out, "out", dt, device=False)
        if ws is None:
            ws = workspace(decode_step_host_workspace_bytes(B, H, d_h, r, d, max_seq_len, dt),
                           page_table.device)
        _need(ws, "ws", torch.uint8)
        self._desc = cache.desc()
        self._keep = (X, W_S_K, W_S_V, U_K, U_V, q, cache, B_K, B_V, seq_lens, page_table, ws,
                      status)
        self.X, self.q, self.seq_lens, self.out = X, q, seq_lens, out
        h = ctypes.c_void_p()
        code = _abi.lib().lrkv_step_graph_create(
            ctypes.byref(h), _ptr(X), d, _ptr(W_S_K), _ptr(W_S_V), _ptr(U_K), _ptr(U_V), _ptr(q),
            ctypes.byref(self._desc), _ptr(B_K), _ptr(B_V), _ptr(seq_lens), _ptr(page_table), B,
            page_table.shape[1], max_seq_len, _ptr(out), _ptr(ws), ws.numel(), _ptr(status))
        _abi.check("lrkv_step_graph_create", code)
        self._h = h

    def launch(self, stream=None):
        """Enqueue one step (copies in, kernels, copy out) on the stream."""
        if self._h is None:
            raise ValueError("graph destroyed")
        _abi.check("lrkv_step_graph_launch", _abi.lib().lrkv_step_graph_launch(self._h, _stream(stream)))
        return self.out

    def close(self):
        """Destroy the graph once every launch of it has finished."""
        if self._h is not None:
            torch.cuda.synchronize()
            _abi.lib().lrkv_step_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def prefill(X, Q, cu_rows, start_pos, max_ctx, W_S_K, W_S_V, U_K, U_V, B_K, B_V,
            cache: PagedCache, page_table, out=None, ws=None, status=None, stream=None):
    """lrkv_prefill: append the chunk X, then causal attention for each row's Q."""
    dt = cache.act_dtype
    for n, t in (("X", X), ("Q", Q), ("W_S_K", W_S_K), ("W_S_V", W_S_V), ("U_K", U_K),
                 ("U_V", U_V), ("B_K", B_K), ("B_V", B_V)):
        _need(t, n, dt)
    for n, t in (("cu_rows", cu_rows), ("start_pos", start_pos), ("page_table", page_table)):
        _need(t, n, torch.int32)
    n, d = X.shape
    _, H, d_h = Q.shape
    r = cache.R_K.shape[3]
    B = start_pos.shape[0]
    if out is None:
        out = _own_buffer(Q.shape, dt, Q.device, stream)
    need = prefill_workspace_bytes(B, n, H, d_h, r, max_ctx, dt)
    if ws is None:
        ws = _scratch(need, X.device, stream)
    desc = cache.desc()
    code = _abi.lib().lrkv_prefill(_ptr(X), _ptr(Q), _ptr(cu_rows), _ptr(start_pos), B, n,
                                   max_ctx, d, _ptr(W_S_K), _ptr(W_S_V), _ptr(U_K), _ptr(U_V),
                                   _ptr(B_K), _ptr(B_V), ctypes.byref(desc), _ptr(page_table),
                                   page_table.shape[1], _ptr(out), _ptr(ws), ws.numel(),
                                   _ptr(status), _stream(stream))
    _abi.check("lrkv_prefill", code)
    return out


# ----------------------------------------------------------------------------
# Sliding window with sinks, and the page plan of such a cache (see
# include/lrkv.h).  These check every shape, and that all tensors lie on the
# current device, before the library is called.  A decode step takes less time
# than a careful look at its arguments, so each function compares everything in
# one expression and looks for the fault only when something differs.
# ----------------------------------------------------------------------------
_i32, _u8, _Tensor = torch.int32, torch.uint8, torch.Tensor


def _refuse(args, dev):
    """Raise for the first of (tensor, name, dtype, shape) that is not such a contiguous tensor on device `dev`."""
    for t, name, dtype, shape in args:
        _need(t, name, dtype)
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, not on the current device cuda:{dev}")


def _fits(args, dev):
    for t, name, dtype, shape in args:
        if not (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
                and t.is_contiguous()):
            _refuse(args, dev)


def _cache_arg(cache, dev):
    """(PagedCache.desc() as bytes, activation dtype, H, d_h, r, groups, LRKV_* dtype) with all pools' shapes and
    devices checked."""
    S_K, S_V, R_K, R_V, N_K = cache.S_K, cache.S_V, cache.R_K, cache.R_V, cache.N_K
    if not (isinstance(S_K, _Tensor) and isinstance(R_K, _Tensor)) or S_K.dim() not in (3, 4) or R_K.dim() != 4:
        raise ValueError("S_K must be [num_pages, page_size, (G,) d_h] and R_K [num_pages, page_size, H, r]")
    dt, ss, rs = S_K.dtype, S_K.shape, R_K.shape
    n, ps, H, r = rs
    if dt not in _DT:
        raise TypeError(f"cache dtype {dt} is not supported")
    if ss[0] != n or ss[1] != ps:
        raise ValueError(f"S_K {list(ss)} and R_K {list(rs)} must have the same pages")
    act = torch.bfloat16 if dt is torch.float8_e4m3fn else dt
    if not (isinstance(S_V, _Tensor) and isinstance(R_V, _Tensor) and S_V.dtype is dt and R_K.dtype is dt
            and R_V.dtype is dt and S_V.shape == ss and R_V.shape == rs and S_K.get_device() == dev
            and S_V.get_device() == dev and R_K.get_device() == dev and R_V.get_device() == dev
            and S_K.is_contiguous() and S_V.is_contiguous() and R_K.is_contiguous() and R_V.is_contiguous()):
        _refuse(((S_K, "S_K", dt, ss), (S_V, "S_V", dt, ss), (R_K, "R_K", dt, rs), (R_V, "R_V", dt, rs)), dev)
    nk = 0
    if N_K is not None:
        _fits(((N_K, "N_K", act, (n, ps, H)),), dev)
        nk = N_K.data_ptr()
    d_h, G, code = ss[-1], ss[2] if len(ss) == 4 else 1, _DT[dt]
    s0, s1, s2, s3 = cache.scale
    return _abi.pack_cache(S_K.data_ptr(), S_V.data_ptr(), R_K.data_ptr(), R_V.data_ptr(), n, ps, H, d_h, r, code,
                           s0, s1, s2, s3, nk, cache.norm_eps, G), act, H, d_h, r, G, code


_LEAST, _MOST = -2 ** 31, 2 ** 31 - 1  # (a size past these would wrap on its way into the library)


def _past_32_bits(**sizes):
    raise ValueError(", ".join(f"{k} = {v}" for k, v in sizes.items()) + ": sizes are 32-bit")


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _device_of(t, name):
    """The current device, where the first argument has to be."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return torch._C._cuda_getDevice()  # (CUDA is initialised: t is on it)


def _dim(t, name, n):
    if not isinstance(t, _Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a tensor of {n} dimension(s)")
    return t.shape


def _workspace(ws, dev):
    """(address, bytes) of a caller's workspace."""
    if ws is None:
        return None, 0
    n = ws.numel()
    _fits(((ws, "ws", _u8, (n,)),), dev)
    return ws.data_ptr(), n


def _status(status, dev):
    if status is None:
        return None
    _fits(((status, "status", _i32, (1,)),), dev)
    return status.data_ptr()


def decode_window_workspace_bytes(B, H, d_h, r, max_seq_len, window, sinks=0, dtype=torch.bfloat16) -> int:
    """lrkv_decode_window_workspace_bytes: enough for this call and for every smaller one."""
    if not (_LEAST <= max_seq_len <= _MOST and _LEAST <= window <= _MOST and _LEAST <= sinks <= _MOST):
        _past_32_bits(max_seq_len=max_seq_len, window=window, sinks=sinks)
    return _abi.lib().lrkv_decode_window_workspace_bytes(B, H, d_h, r, max_seq_len, window, sinks, _DT[dtype])


def decode_window(q, cache: PagedCache, B_K, B_V, seq_lens, page_table, max_seq_len, window, sinks=0,
                  out=None, ws=None, status=None, stream=None):
    """lrkv_decode_window: one decode step in which request b sees its last
    ``window`` rows and its first ``sinks`` rows; returns out [B, H, d_h].  With
    ``ws`` (decode_window_workspace_bytes uint8) few requests may be laid out
    faster; without it one is made where a long call needs it."""
    dev = _device_of(q, "q")
    desc, dt, H, d_h, r, G, code = _cache_arg(cache, dev)
    B, max_pages = _dim(q, "q", 3)[0], _dim(page_table, "page_table", 2)[1]
    if out is None:
        out = torch.empty_like(q) if stream is None else _own_buffer(q.shape, q.dtype, q.device, stream)
    shape, base = (B, H, d_h), (H, d_h, r)
    if not (isinstance(B_K, _Tensor) and isinstance(B_V, _Tensor) and isinstance(seq_lens, _Tensor)
            and isinstance(out, _Tensor) and q.dtype is dt and B_K.dtype is dt and B_V.dtype is dt and out.dtype is dt
            and seq_lens.dtype is _i32 and page_table.dtype is _i32 and q.shape == shape and out.shape == shape
            and B_K.shape == base and B_V.shape == base and seq_lens.shape == (B,) and page_table.shape[0] == B
            and q.get_device() == dev and B_K.get_device() == dev and B_V.get_device() == dev
            and seq_lens.get_device() == dev and page_table.get_device() == dev and out.get_device() == dev
            and q.is_contiguous() and B_K.is_contiguous() and B_V.is_contiguous() and seq_lens.is_contiguous()
            and page_table.is_contiguous() and out.is_contiguous()):
        _refuse(((q, "q", dt, shape), (B_K, "B_K", dt, base), (B_V, "B_V", dt, base), (seq_lens, "seq_lens", _i32, (B,)),
                 (page_table, "page_table", _i32, (B, max_pages)), (out, "out", dt, shape)), dev)
    L = _abi.lib()
    if not (_LEAST <= max_seq_len <= _MOST and _LEAST <= window <= _MOST and _LEAST <= sinks <= _MOST):
        _past_32_bits(max_seq_len=max_seq_len, window=window, sinks=sinks)
    args = (q.data_ptr(), desc, B_K.data_ptr(), B_V.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(), B,
            max_pages, max_seq_len, window, sinks, out.data_ptr())
    tail = (None if status is None else _status(status, dev),
            torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    err = (L.lrkv_decode_window(*args, None, 0, *tail) if ws is None
           else L.lrkv_decode_window(*args, *_workspace(ws, dev), *tail))
    if err == _abi.LRKV_E_WORKSPACE and ws is None:  # (most calls need none)
        n = L.lrkv_decode_window_workspace_bytes(B, H, d_h, r, max_seq_len, window, sinks, code)
        ws = _scratch(n, q.device, stream)
        err = L.lrkv_decode_window(*args, ws.data_ptr(), n, *tail)
    if err:
        _abi.check("lrkv_decode_window", err)
    return out


def prefill_window(X, Q, cu_rows, start_pos, max_ctx, W_S_K, W_S_V, U_K, U_V, B_K, B_V,
                   cache: PagedCache, page_table, window, sinks=0, out=None, ws=None, status=None,
                   stream=None):
    """lrkv_prefill_window: append the chunk X, then attention of each row's Q
    over the last ``window`` rows up to its own and the first ``sinks`` rows."""
    dev = _device_of(X, "X")
    desc, dt, H, d_h, r, G, code = _cache_arg(cache, dev)
    n, d = _dim(X, "X", 2)
    (B,) = _dim(start_pos, "start_pos", 1)
    max_pages = _dim(page_table, "page_table", 2)[1]
    shape, base, shared, private = (n, H, d_h), (H, d_h, r), (G * d_h, d), (H, r, d)
    if out is None:
        out = _own_buffer(shape, dt, X.device, stream)
    T = _Tensor
    if not (isinstance(Q, T) and isinstance(cu_rows, T) and isinstance(W_S_K, T) and isinstance(W_S_V, T)
            and isinstance(U_K, T) and isinstance(U_V, T) and isinstance(B_K, T) and isinstance(B_V, T)
            and isinstance(out, T) and X.dtype is dt and Q.dtype is dt and cu_rows.dtype is _i32
            and start_pos.dtype is _i32 and W_S_K.dtype is dt and W_S_V.dtype is dt and U_K.dtype is dt
            and U_V.dtype is dt and B_K.dtype is dt and B_V.dtype is dt and page_table.dtype is _i32 and out.dtype is dt
            and Q.shape == shape and cu_rows.shape == (B + 1,) and W_S_K.shape == shared and W_S_V.shape == shared
            and U_K.shape == private and U_V.shape == private and B_K.shape == base and B_V.shape == base
            and page_table.shape[0] == B and out.shape == shape
            and X.get_device() == dev and Q.get_device() == dev and cu_rows.get_device() == dev
            and start_pos.get_device() == dev and W_S_K.get_device() == dev and W_S_V.get_device() == dev
            and U_K.get_device() == dev and U_V.get_device() == dev and B_K.get_device() == dev
            and B_V.get_device() == dev and page_table.get_device() == dev and out.get_device() == dev
            and X.is_contiguous() and Q.is_contiguous() and cu_rows.is_contiguous() and start_pos.is_contiguous()
            and W_S_K.is_contiguous() and W_S_V.is_contiguous() and U_K.is_contiguous() and U_V.is_contiguous()
            and B_K.is_contiguous() and B_V.is_contiguous() and page_table.is_contiguous() and out.is_contiguous()):
        _refuse(((X, "X", dt, (n, d)), (Q, "Q", dt, shape), (cu_rows, "cu_rows", _i32, (B + 1,)),
                 (start_pos, "start_pos", _i32, (B,)), (W_S_K, "W_S_K", dt, shared), (W_S_V, "W_S_V", dt, shared),
                 (U_K, "U_K", dt, private), (U_V, "U_V", dt, private), (B_K, "B_K", dt, base), (B_V, "B_V", dt, base),
                 (page_table, "page_table", _i32, (B, max_pages)), (out, "out", dt, shape)), dev)
    if not (_LEAST <= max_ctx <= _MOST and _LEAST <= window <= _MOST and _LEAST <= sinks <= _MOST):
        _past_32_bits(max_ctx=max_ctx, window=window, sinks=sinks)
    L = _abi.lib()
    args = (X.data_ptr(), Q.data_ptr(), cu_rows.data_ptr(), start_pos.data_ptr(), B, n, max_ctx, d, W_S_K.data_ptr(),
            W_S_V.data_ptr(), U_K.data_ptr(), U_V.data_ptr(), B_K.data_ptr(), B_V.data_ptr(), desc,
            page_table.data_ptr(), max_pages, window, sinks, out.data_ptr())
    tail = _status(status, dev), _raw_stream(stream, dev)
    err = L.lrkv_prefill_window(*args, *_workspace(ws, dev), *tail)
    if err == _abi.LRKV_E_WORKSPACE and ws is None:  # (few rows, or the per-row path)
        m = L.lrkv_prefill_workspace_bytes(B, n, H, d_h, r, max_ctx, code)
        ws = _scratch(m, X.device, stream)
        err = L.lrkv_prefill_window(*args, ws.data_ptr(), m, *tail)
    if err:
        _abi.check("lrkv_prefill_window", err)
    return out


class PagePlan(NamedTuple):
    """What lrkv_page_plan writes beside the page table: the lengths after the
    step, each request's rows as cu_rows offsets, the rows' positions, requests
    and pool rows (slots), and the free list after the step with its count."""
    seq_lens: torch.Tensor
    cu_rows: torch.Tensor
    positions: torch.Tensor
    seq_ids: torch.Tensor
    slots: torch.Tensor
    free_pages: torch.Tensor
    n_free: torch.Tensor


def page_plan(seq_lens, new_rows, page_table, free_pages, n_free, page_size, max_rows, free_out=None,
              window=0, sinks=0, status=None, stream=None) -> PagePlan:
    """lrkv_page_plan: pages and slots of one step, in which request b gains
    new_rows[b] rows (-1: it ends).  page_table is updated in place; free_out
    ([num_pages]) takes the free list after the step."""
    dev = _device_of(seq_lens, "seq_lens")
    (B,), (num_pages,) = _dim(seq_lens, "seq_lens", 1), _dim(free_pages, "free_pages", 1)
    max_pages = _dim(page_table, "page_table", 2)[1]
    if max_rows < 0:
        raise ValueError("max_rows must not be negative")
    if not (max_rows <= _MOST and _LEAST <= page_size <= _MOST and _LEAST <= window <= _MOST
            and _LEAST <= sinks <= _MOST):
        _past_32_bits(max_rows=max_rows, page_size=page_size, window=window, sinks=sinks)
    if free_out is None:
        free_out = _own_buffer((num_pages,), _i32, seq_lens.device, stream)
    if not (isinstance(new_rows, _Tensor) and isinstance(n_free, _Tensor) and isinstance(free_out, _Tensor)
            and seq_lens.dtype is _i32 and new_rows.dtype is _i32 and page_table.dtype is _i32
            and free_pages.dtype is _i32 and n_free.dtype is _i32 and free_out.dtype is _i32
            and new_rows.shape == (B,) and page_table.shape[0] == B and n_free.shape == (1,)
            and free_out.shape == (num_pages,) and seq_lens.get_device() == dev and new_rows.get_device() == dev
            and page_table.get_device() == dev and free_pages.get_device() == dev and n_free.get_device() == dev
            and free_out.get_device() == dev and seq_lens.is_contiguous() and new_rows.is_contiguous()
            and page_table.is_contiguous() and free_pages.is_contiguous() and free_out.is_contiguous()):
        _refuse(((seq_lens, "seq_lens", _i32, (B,)), (new_rows, "new_rows", _i32, (B,)),
                 (page_table, "page_table", _i32, (B, max_pages)), (free_pages, "free_pages", _i32, (num_pages,)),
                 (n_free, "n_free", _i32, (1,)), (free_out, "free_out", _i32, (num_pages,))), dev)
    # one buffer for the small outputs
    sizes = (max_rows, max_rows, max_rows, B, B + 1, 1)
    parts = _own_buffer((3 * max_rows + 2 * B + 2,), _i32, seq_lens.device, stream)
    p, row = parts.data_ptr(), 4 * max_rows
    after = p + 3 * row
    cu = after + 4 * B
    code = _abi.lib().lrkv_page_plan(
        seq_lens.data_ptr(), new_rows.data_ptr(), B, max_pages, page_size, num_pages, window, sinks, max_rows,
        page_table.data_ptr(), free_pages.data_ptr(), n_free.data_ptr(), after, cu, p, p + row, p + 2 * row,
        free_out.data_ptr(), cu + 4 * (B + 1), _status(status, dev), _raw_stream(stream, dev))
    if code:
        _abi.check("lrkv_page_plan", code)
    pos, ids, slots, lens, cu_rows, left = parts.unsafe_split_with_sizes(sizes)  # (nothing here is differentiated)
    return PagePlan(lens, cu_rows, pos, ids, slots, free_out, left)


# ----------------------------------------------------------------------------
# Block-scaled cache (see include/lrkv.h): 8-bit codes with a power-of-two scale
# for each block of tokens and head.  Checked like the windowed functions.
# ----------------------------------------------------------------------------
_POOLS = ("S_K", "S_V", "R_K", "R_V")


@dataclass
class ScaledCache:
    """Caller-owned paged cache in 8 bits that finds its scales itself.

    S_K, S_V: codes [num_pages, page_size, d_h] (or [.., G, d_h] for G shared
    groups); R_K, R_V: [num_pages, page_size, H, r], all torch.float8_e4m3fn.
    E_S_K, E_S_V: [num_pages, page_size // block, G] and E_R_K, E_R_V: [..., H],
    torch.uint8: a code's value is code * 2^(byte - 127) with the byte of its
    block of ``block`` tokens and its head (group).  Nothing needs initialising:
    the functions that write rows set the scales of the blocks they begin.
    """
    S_K: torch.Tensor
    S_V: torch.Tensor
    R_K: torch.Tensor
    R_V: torch.Tensor
    E_S_K: torch.Tensor
    E_S_V: torch.Tensor
    E_R_K: torch.Tensor
    E_R_V: torch.Tensor

    @classmethod
    def empty(cls, num_pages, page_size, H, d_h, r, block=64, device="cuda", groups=1):
        if block < 1 or page_size % block:
            raise ValueError(f"block = {block} must divide page_size = {page_size}")
        code = lambda *s: torch.empty(s, dtype=torch.float8_e4m3fn, device=device)
        exp = lambda n: torch.empty((num_pages, page_size // block, n), dtype=torch.uint8, device=device)
        sh = (num_pages, page_size, d_h) if groups == 1 else (num_pages, page_size, groups, d_h)
        return cls(code(*sh), code(*sh), code(num_pages, page_size, H, r), code(num_pages, page_size, H, r),
                   exp(groups), exp(groups), exp(H), exp(H))

    @property
    def block(self):
        """Tokens that share a scale."""
        return self.R_K.shape[1] // self.E_R_K.shape[1]

    @property
    def groups(self):
        """Shared key/value groups (1: one shared basis)."""
        return self.S_K.shape[2] if self.S_K.dim() == 4 else 1


class ScaledRows(NamedTuple):
    """Rows read back: S_K, S_V [n, d_h] (or [n, G, d_h]), R_K, R_V [n, H, r]."""
    S_K: torch.Tensor
    S_V: torch.Tensor
    R_K: torch.Tensor
    R_V: torch.Tensor


_f8, _bf16, _f32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


def _scaled_arg(cache, dev):
    """(lrkv_scaled_t as bytes, H, d_h, r, groups) with all tensors' shapes and devices checked."""
    S_K, S_V, R_K, R_V = cache.S_K, cache.S_V, cache.R_K, cache.R_V
    E_S_K, E_S_V, E_R_K, E_R_V = cache.E_S_K, cache.E_S_V, cache.E_R_K, cache.E_R_V
    try:
        ss, rs, er = S_K.shape, R_K.shape, E_R_K.shape
        n, ps, H, r = rs
        _, nb, _ = er
        d_h, G = ss[-1], ss[2] if len(ss) == 4 else 1
        es = E_S_K.shape
        good = (len(ss) in (3, 4) and ss[0] == n and ss[1] == ps and nb > 0 and ps % nb == 0 and er[0] == n
                and er[2] == H and es[0] == n and es[1] == nb and es[2] == G and S_V.shape == ss and R_V.shape == rs
                and E_S_V.shape == es and E_R_V.shape == er and len(es) == 3
                and S_K.dtype is _f8 and S_V.dtype is _f8 and R_K.dtype is _f8 and R_V.dtype is _f8
                and E_S_K.dtype is _u8 and E_S_V.dtype is _u8 and E_R_K.dtype is _u8 and E_R_V.dtype is _u8
                and S_K.get_device() == dev and S_V.get_device() == dev and R_K.get_device() == dev
                and R_V.get_device() == dev and E_S_K.get_device() == dev and E_S_V.get_device() == dev
                and E_R_K.get_device() == dev and E_R_V.get_device() == dev and S_K.is_contiguous()
                and S_V.is_contiguous() and R_K.is_contiguous() and R_V.is_contiguous() and E_S_K.is_contiguous()
                and E_S_V.is_contiguous() and E_R_K.is_contiguous() and E_R_V.is_contiguous())
    except (AttributeError, IndexError, TypeError, ValueError):  # (no tensors, or of other dimensions)
        good = False
    if not good:
        _refuse_scaled(cache, dev)
    return _abi.pack_scaled(S_K.data_ptr(), S_V.data_ptr(), R_K.data_ptr(), R_V.data_ptr(), E_S_K.data_ptr(),
                            E_S_V.data_ptr(), E_R_K.data_ptr(), E_R_V.data_ptr(), n, ps, H, d_h, r, G, ps // nb,
                            0), H, d_h, r, G


def _refuse_scaled(cache, dev):
    """Say what is wrong with a ScaledCache."""
    S_K, R_K, E_R_K = cache.S_K, cache.R_K, cache.E_R_K
    if not (isinstance(S_K, _Tensor) and isinstance(R_K, _Tensor) and isinstance(E_R_K, _Tensor)) \
            or S_K.dim() not in (3, 4) or R_K.dim() != 4 or E_R_K.dim() != 3:
        raise ValueError("S_K must be [num_pages, page_size, (G,) d_h], R_K [num_pages, page_size, H, r] and E_R_K "
                         "[num_pages, page_size / block, H]")
    ss, rs, nb = S_K.shape, R_K.shape, E_R_K.shape[1]
    n, ps, H, _ = rs
    if ss[0] != n or ss[1] != ps:
        raise ValueError(f"S_K {list(ss)} and R_K {list(rs)} must have the same pages")
    if nb < 1 or ps % nb:
        raise ValueError(f"E_R_K {list(E_R_K.shape)} does not divide pages of {ps} tokens into blocks")
    es, er = (n, nb, ss[2] if len(ss) == 4 else 1), (n, nb, H)
    _refuse(((S_K, "S_K", _f8, ss), (cache.S_V, "S_V", _f8, ss), (R_K, "R_K", _f8, rs), (cache.R_V, "R_V", _f8, rs),
             (cache.E_S_K, "E_S_K", _u8, es), (cache.E_S_V, "E_S_V", _u8, es), (E_R_K, "E_R_K", _u8, er),
             (cache.E_R_V, "E_R_V", _u8, er)), dev)
    raise ValueError("the cache's tensors do not fit together")


def _row_args(cu_rows, start_pos, page_table, dev):
    """(B, max_pages) of the requests' rows of a call."""
    try:
        (B,), (rows, max_pages) = start_pos.shape, page_table.shape
        good = (cu_rows.dtype is _i32 and start_pos.dtype is _i32 and page_table.dtype is _i32 and rows == B
                and cu_rows.shape == (B + 1,) and cu_rows.get_device() == dev and start_pos.get_device() == dev
                and page_table.get_device() == dev and cu_rows.is_contiguous() and start_pos.is_contiguous()
                and page_table.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        (B,), max_pages = _dim(start_pos, "start_pos", 1), _dim(page_table, "page_table", 2)[1]
        _refuse(((cu_rows, "cu_rows", _i32, (B + 1,)), (start_pos, "start_pos", _i32, (B,)),
                 (page_table, "page_table", _i32, (B, max_pages))), dev)
        raise ValueError("cu_rows, start_pos and page_table do not fit together")
    return B, max_pages


def _strided_rows(rows, n, H, d_h, r, G, dev):
    """Address and row stride of the four pools' rows one after the other, and their dtype.  A row is dense; rows may
    lie apart (slices of one projection's output)."""
    a, b, c, e = rows
    try:
        dt, sa, sb, sc, se = a.dtype, a.stride(), b.stride(), c.stride(), e.stride()
        shared, private = G * d_h, H * r
        # rows of a matrix, or of heads that lie next to each other
        flat = lambda t, st, heads, width: (  # noqa: E731
            t.shape == (n, heads * width) and st[1] == 1 or
            t.shape == (n, heads, width) and st[2] == 1 and (st[1] == width or heads == 1))
        good = (n > 1 and (dt is _bf16 or dt is _f32) and b.dtype is dt and c.dtype is dt and e.dtype is dt
                and a.get_device() == dev and b.get_device() == dev and c.get_device() == dev
                and e.get_device() == dev and flat(a, sa, G, d_h) and flat(b, sb, G, d_h) and flat(c, sc, H, r)
                and flat(e, se, H, r))
    except (AttributeError, IndexError, TypeError):
        good = False
    if good:
        return (a.data_ptr(), sa[0], b.data_ptr(), sb[0], c.data_ptr(), sc[0], e.data_ptr(), se[0]), dt
    out, dt = [], None
    for name, t in zip(_POOLS, rows):
        if not isinstance(t, _Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        shape, ld = t.shape, t.stride()
        flat, deep = ((n, G * d_h), (n, G, d_h)) if name[0] == "S" else ((n, H * r), (n, H, r))
        if dt is None:
            dt = t.dtype
            if dt is not _bf16 and dt is not _f32:
                raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {dt}")
        if t.dtype is not dt:
            raise TypeError(f"{name} must be {dt}, got {t.dtype}")
        if shape != flat and shape != deep:
            raise ValueError(f"{name} must be {list(deep)} or {list(flat)}, got {list(shape)}")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{dev}")
        if n and not (ld[-1] == 1 and (len(shape) == 2 or ld[1] == shape[2] or shape[1] == 1)):
            raise ValueError(f"{name}: the values of a row must be contiguous")
        # (one row has no distance to a next one)
        out += [t.data_ptr(), flat[1] if n <= 1 else ld[0]]
    return out, dt


def write_scaled(S_K, S_V, R_K, R_V, cu_rows, start_pos, cache: ScaledCache, page_table, status=None, stream=None):
    """lrkv_write_scaled: quantise rows (S_K, S_V [n, d_h] or [n, G, d_h]; R_K, R_V [n, H, r] or [n, H * r], bf16 or
    fp32, rows may have a stride) of requests b = rows cu_rows[b] .. cu_rows[b + 1] - 1 into the cache at positions
    start_pos[b], start_pos[b] + 1, ..."""
    dev = _device_of(S_K, "S_K")
    desc, H, d_h, r, G = _scaled_arg(cache, dev)
    B, max_pages = _row_args(cu_rows, start_pos, page_table, dev)
    n = S_K.shape[0] if S_K.dim() else 0
    rows, dt = _strided_rows((S_K, S_V, R_K, R_V), n, H, d_h, r, G, dev)
    code = _abi.lib().lrkv_write_scaled(*rows, _DT[dt], cu_rows.data_ptr(), start_pos.data_ptr(), B, n, desc,
                                        page_table.data_ptr(), max_pages,
                                        None if status is None else _status(status, dev),
                                        _raw_stream(stream, dev))
    if code:
        _abi.check("lrkv_write_scaled", code)


def read_scaled(cu_rows, start_pos, n, cache: ScaledCache, page_table, dtype=torch.bfloat16, out=None, status=None,
                stream=None) -> ScaledRows:
    """lrkv_read_scaled: the values of n rows, addressed as by write_scaled, in bf16 or fp32 (exact in both).  Rows of
    ``out`` (a ScaledRows) that no request owns, or that lie on no page, stay as they are."""
    dev = _device_of(cu_rows, "cu_rows")
    desc, H, d_h, r, G = _scaled_arg(cache, dev)
    B, max_pages = _row_args(cu_rows, start_pos, page_table, dev)
    if n < 0:
        raise ValueError("n must not be negative")
    if n > _MOST:
        _past_32_bits(n=n)
    if out is None:
        shared = (n, d_h) if cache.S_K.dim() == 3 else (n, G, d_h)
        if dtype is not _bf16 and dtype is not _f32:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
        at, private = cu_rows.device, (n, H, r)
        a, b, c, e = out = ScaledRows(*[_own_buffer(s, dtype, at, stream) for s in (shared, shared, private, private)])
        rows, dt = (a.data_ptr(), G * d_h, b.data_ptr(), G * d_h, c.data_ptr(), H * r, e.data_ptr(), H * r), dtype
    else:
        rows, dt = _strided_rows(out, n, H, d_h, r, G, dev)
        out = ScaledRows(*out)
    code = _abi.lib().lrkv_read_scaled(desc, cu_rows.data_ptr(), start_pos.data_ptr(), B, n, page_table.data_ptr(),
                                       max_pages, _DT[dt], *rows, None if status is None else _status(status, dev),
                                       _raw_stream(stream, dev))
    if code:
        _abi.check("lrkv_read_scaled", code)
    return out


def _projection_args(X, W_S_K, W_S_V, U_K, U_V, H, d_h, r, G, dev):
    """(n, d) with the projection's tensors checked."""
    try:
        n, d = X.shape
        shared, private = (G * d_h, d), (H, r, d)
        good = (X.dtype is _bf16 and W_S_K.dtype is _bf16 and W_S_V.dtype is _bf16
                and U_K.dtype is _bf16 and U_V.dtype is _bf16 and W_S_K.shape == shared and W_S_V.shape == shared
                and U_K.shape == private and U_V.shape == private and X.get_device() == dev
                and W_S_K.get_device() == dev and W_S_V.get_device() == dev and U_K.get_device() == dev
                and U_V.get_device() == dev and X.is_contiguous() and W_S_K.is_contiguous() and W_S_V.is_contiguous()
                and U_K.is_contiguous() and U_V.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        n, d = _dim(X, "X", 2)
        shared, private = (G * d_h, d), (H, r, d)
        _refuse(((X, "X", _bf16, (n, d)), (W_S_K, "W_S_K", _bf16, shared), (W_S_V, "W_S_V", _bf16, shared),
                 (U_K, "U_K", _bf16, private), (U_V, "U_V", _bf16, private)), dev)
        raise ValueError("X and the weights do not fit together")
    return n, d


def _own_workspace(ws, need, dev, device, stream):
    """(address, bytes) of the caller's workspace, or of one made for the call; the tensor, to keep it until then."""
    if ws is None:
        ws = torch.empty(need or 1, dtype=_u8, device=device) if stream is None else _scratch(need, device, stream)
        return ws.data_ptr(), need, ws
    return *_workspace(ws, dev), ws


def append_scaled_workspace_bytes(cache: ScaledCache, n) -> int:
    """lrkv_append_scaled_workspace_bytes: for up to n rows."""
    return _abi.lib().lrkv_append_scaled_workspace_bytes(_scaled_arg(cache, cache.S_K.get_device())[0], n)


def append_scaled(X, cu_rows, start_pos, W_S_K, W_S_V, U_K, U_V, cache: ScaledCache, page_table, ws=None, status=None,
                  stream=None):
    """lrkv_append_scaled: project rows X and quantise them into the cache, addressed as by write_scaled."""
    dev = _device_of(X, "X")
    desc, H, d_h, r, G = _scaled_arg(cache, dev)
    B, max_pages = _row_args(cu_rows, start_pos, page_table, dev)
    n, d = _projection_args(X, W_S_K, W_S_V, U_K, U_V, H, d_h, r, G, dev)
    L = _abi.lib()
    need = L.lrkv_append_scaled_workspace_bytes(desc, n) if ws is None else 0
    addr, size, ws = _own_workspace(ws, need, dev, X.device, stream)
    code = L.lrkv_append_scaled(X.data_ptr(), cu_rows.data_ptr(), start_pos.data_ptr(), B, n, d, W_S_K.data_ptr(),
                                W_S_V.data_ptr(), U_K.data_ptr(), U_V.data_ptr(), desc, page_table.data_ptr(),
                                max_pages, addr, size, None if status is None else _status(status, dev), _raw_stream(stream, dev))
    if code:
        _abi.check("lrkv_append_scaled", code)


def decode_scaled_workspace_bytes(cache: ScaledCache, B, max_seq_len) -> int:
    """lrkv_decode_scaled_workspace_bytes: enough for this call and for every smaller one."""
    if not (_LEAST <= max_seq_len <= _MOST):
        _past_32_bits(max_seq_len=max_seq_len)
    return _abi.lib().lrkv_decode_scaled_workspace_bytes(_scaled_arg(cache, cache.S_K.get_device())[0], B, max_seq_len)


def decode_scaled(q, cache: ScaledCache, B_K, B_V, seq_lens, page_table, max_seq_len, out=None, ws=None, status=None,
                  stream=None):
    """lrkv_decode_scaled: per-head attention output [B, H, d_h] (bf16) of one decode step over the cache."""
    dev = _device_of(q, "q")
    desc, H, d_h, r, G = _scaled_arg(cache, dev)
    B, max_pages = _dim(q, "q", 3)[0], _dim(page_table, "page_table", 2)[1]
    if out is None:
        out = torch.empty_like(q) if stream is None else _own_buffer(q.shape, q.dtype, q.device, stream)
    shape, base = (B, H, d_h), (H, d_h, r)
    try:
        good = (q.dtype is _bf16 and B_K.dtype is _bf16 and B_V.dtype is _bf16
                and out.dtype is _bf16 and seq_lens.dtype is _i32 and page_table.dtype is _i32 and q.shape == shape
                and out.shape == shape and B_K.shape == base and B_V.shape == base and seq_lens.shape == (B,)
                and page_table.shape[0] == B and q.get_device() == dev and B_K.get_device() == dev
                and B_V.get_device() == dev and seq_lens.get_device() == dev and page_table.get_device() == dev
                and out.get_device() == dev and q.is_contiguous() and B_K.is_contiguous() and B_V.is_contiguous()
                and seq_lens.is_contiguous() and page_table.is_contiguous() and out.is_contiguous())
    except AttributeError:
        good = False
    if not good:
        _refuse(((q, "q", _bf16, shape), (B_K, "B_K", _bf16, base), (B_V, "B_V", _bf16, base),
                 (seq_lens, "seq_lens", _i32, (B,)), (page_table, "page_table", _i32, (B, max_pages)),
                 (out, "out", _bf16, shape)), dev)
    if not (_LEAST <= max_seq_len <= _MOST):
        _past_32_bits(max_seq_len=max_seq_len)
    L = _abi.lib()
    need = L.lrkv_decode_scaled_workspace_bytes(desc, B, max_seq_len) if ws is None else 0
    addr, size, ws = _own_workspace(ws, need, dev, q.device, stream)
    code = L.lrkv_decode_scaled(q.data_ptr(), desc, B_K.data_ptr(), B_V.data_ptr(), seq_lens.data_ptr(),
                                page_table.data_ptr(), B, max_pages, max_seq_len, out.data_ptr(), addr, size,
                                None if status is None else _status(status, dev), _raw_stream(stream, dev))
    if code:
        _abi.check("lrkv_decode_scaled", code)
    return out


def prefill_scaled_workspace_bytes(cache: ScaledCache, B, n, max_ctx) -> int:
    """lrkv_prefill_scaled_workspace_bytes of a call of n rows of B requests."""
    if not (_LEAST <= max_ctx <= _MOST):
        _past_32_bits(max_ctx=max_ctx)
    return _abi.lib().lrkv_prefill_scaled_workspace_bytes(_scaled_arg(cache, cache.S_K.get_device())[0], B, n, max_ctx)


def prefill_scaled(X, Q, cu_rows, start_pos, max_ctx, W_S_K, W_S_V, U_K, U_V, B_K, B_V, cache: ScaledCache, page_table,
                   out=None, ws=None, status=None, stream=None):
    """lrkv_prefill_scaled: append the chunk X, then causal attention of each row's Q over its request's rows."""
    dev = _device_of(X, "X")
    desc, H, d_h, r, G = _scaled_arg(cache, dev)
    B, max_pages = _row_args(cu_rows, start_pos, page_table, dev)
    n, d = _projection_args(X, W_S_K, W_S_V, U_K, U_V, H, d_h, r, G, dev)
    shape, base = (n, H, d_h), (H, d_h, r)
    if out is None:
        out = _own_buffer(shape, _bf16, X.device, stream)
    _fits(((Q, "Q", _bf16, shape), (B_K, "B_K", _bf16, base), (B_V, "B_V", _bf16, base), (out, "out", _bf16, shape)), dev)
    if not (_LEAST <= max_ctx <= _MOST):
        _past_32_bits(max_ctx=max_ctx)
    L = _abi.lib()
    need = L.lrkv_prefill_scaled_workspace_bytes(desc, B, n, max_ctx) if ws is None else 0
    addr, size, ws = _own_workspace(ws, need, dev, X.device, stream)
    code = L.lrkv_prefill_scaled(X.data_ptr(), Q.data_ptr(), cu_rows.data_ptr(), start_pos.data_ptr(), B, n, max_ctx, d,
                                 W_S_K.data_ptr(), W_S_V.data_ptr(), U_K.data_ptr(), U_V.data_ptr(), B_K.data_ptr(),
                                 B_V.data_ptr(), desc, page_table.data_ptr(), max_pages, out.data_ptr(), addr, size,
                                 _status(status, dev), _raw_stream(stream, dev))
    if code:
        _abi.check("lrkv_prefill_scaled", code)
    return out


# ----------------------------------------------------------------------------
# Exact rotary position embedding (see include/lrkv.h)
# ----------------------------------------------------------------------------
class RopeTable:
    """The rotary table of lrkv_rope_table: one device buffer holding the
    (cos, sin) of position * base^(-2c/d_h) as float pairs [max_pos, d_h/2, 2]
    and, after them, the same pairs as f16."""

    def __init__(self, buf: torch.Tensor, d_h: int, max_pos: int):
        self.buf, self.d_h, self.max_pos = buf, d_h, max_pos

    @property
    def cos_sin(self) -> torch.Tensor:
        """The float pairs, [max_pos, d_h/2, 2] fp32 (a view of the buffer)."""
        n = self.max_pos * self.d_h
        return self.buf[: 4 * n].view(torch.float32).view(self.max_pos, self.d_h // 2, 2)

    @property
    def cos_sin_f16(self) -> torch.Tensor:
        """The f16 pairs, [max_pos, d_h/2, 2] (a view of the buffer)."""
        n = self.max_pos * self.d_h
        o = (4 * n + 255) // 256 * 256
        return self.buf[o: o + 2 * n].view(torch.float16).view(self.max_pos, self.d_h // 2, 2)


def rope_table_bytes(d_h, max_pos) -> int:
    return int(_abi.lib().lrkv_rope_table_bytes(d_h, max_pos))


def rope_table(d_h, max_pos, base=10000.0, device="cuda", stream=None) -> RopeTable:
    """lrkv_rope_table: (cos, sin) of position * base^(-2c/d_h) for positions
    below max_pos, in fp32 and f16."""
    nbytes = rope_table_bytes(d_h, max_pos)
    if nbytes == 0:
        raise ValueError(f"invalid rotary table size d_h={d_h} max_pos={max_pos}")
    buf = _own_buffer((nbytes,), torch.uint8, device, stream)
    _abi.check("lrkv_rope_table", _abi.lib().lrkv_rope_table(float(base), d_h, max_pos, _ptr(buf),
                                                             _stream(stream)))
    return RopeTable(buf, d_h, max_pos)


def decode_rope_workspace_bytes(B, H, d_h, r, max_seq_len, dtype=torch.bfloat16) -> int:
    return int(_abi.lib().lrkv_decode_rope_workspace_bytes(B, H, d_h, r, max_seq_len, _DT[dtype]))


def _need_table(table, d_h):
    if not isinstance(table, RopeTable):
        raise TypeError("table must be a RopeTable (rope_table())")
    if table.d_h != d_h:
        raise ValueError(f"table is for d_h={table.d_h}, not {d_h}")
    _need(table.buf, "table", torch.uint8)


def decode_rope(q, cache: PagedCache, B_K, B_V, seq_lens, page_table, max_seq_len, table,
                out=None, ws=None, status=None, stream=None):
    """lrkv_decode_rope: decode with the exact rotary embedding; the query of
    request b sits at position seq_lens[b] - 1."""
    dt = cache.act_dtype
    for n, t in (("q", q), ("B_K", B_K), ("B_V", B_V)):
        _need(t, n, dt)
    _need(seq_lens, "seq_lens", torch.int32)
    _need(page_table, "page_table", torch.int32)
    B, H, d_h = q.shape
    _need_table(table, d_h)
    r = cache.R_K.shape[3]
    if out is None:
        out = _own_buffer(q.shape, dt, q.device, stream)
    _need(out, "out", dt)
    if ws is None:
        ws = _scratch(decode_rope_workspace_bytes(B, H, d_h, r, max_seq_len, dt), q.device, stream)
    _need(ws, "ws", torch.uint8)
    desc = cache.desc()
    code = _abi.lib().lrkv_decode_rope(_ptr(q), ctypes.byref(desc), _ptr(B_K), _ptr(B_V),
                                       _ptr(seq_lens), _ptr(page_table), B, page_table.shape[1],
                                       max_seq_len, _ptr(table.buf), table.max_pos, _ptr(out),
                                       _ptr(ws), ws.numel(), _ptr(status), _stream(stream))
    _abi.check("lrkv_decode_rope", code)
    return out


def prefill_rope(X, Q, cu_rows, start_pos, max_ctx, W_S_K, W_S_V, U_K, U_V, B_K, B_V,
                 cache: PagedCache, page_table, table, out=None, ws=None, status=None,
                 stream=None):
    """lrkv_prefill_rope: append the chunk X, then causal attention with the
    exact rotary embedding (each row's query at its own position)."""
    dt = cache.act_dtype
    for n, t in (("X", X), ("Q", Q), ("W_S_K", W_S_K), ("W_S_V", W_S_V), ("U_K", U_K),
                 ("U_V", U_V), ("B_K", B_K), ("B_V", B_V)):
        _need(t, n, dt)
    for n, t in (("cu_rows", cu_rows), ("start_pos", start_pos), ("page_table", page_table)):
        _need(t, n, torch.int32)
    n, d = X.shape
    _, H, d_h = Q.shape
    _need_table(table, d_h)
    r = cache.R_K.shape[3]
    B = start_pos.shape[0]
    if out is None:
        out = _own_buffer(Q.shape, dt, Q.device, stream)
    if ws is None:
        ws = _scratch(prefill_workspace_bytes(B, n, H, d_h, r, max_ctx, dt), X.device, stream)
    desc = cache.desc()
    code = _abi.lib().lrkv_prefill_rope(_ptr(X), _ptr(Q), _ptr(cu_rows), _ptr(start_pos), B, n,
                                        max_ctx, d, _ptr(W_S_K), _ptr(W_S_V), _ptr(U_K),
                                        _ptr(U_V), _ptr(B_K), _ptr(B_V), ctypes.byref(desc),
                                        _ptr(page_table), page_table.shape[1], _ptr(table.buf),
                                        table.max_pos, _ptr(out), _ptr(ws), ws.numel(),
                                        _ptr(status), _stream(stream))
    _abi.check("lrkv_prefill_rope", code)
    return out


def key_norms(positions, seq_ids, B_K, cache: PagedCache, page_table, status=None, stream=None):
    """lrkv_key_norms: store the reciprocal joint key norms of the given rows."""
    _need(B_K, "B_K", cache.act_dtype)
    for n, t in (("positions", positions), ("seq_ids", seq_ids), ("page_table", page_table)):
        _need(t, n, torch.int32)
    if cache.N_K is None:
        raise ValueError("cache.N_K is None")
    desc = cache.desc()
    B, max_pages = page_table.shape
    code = _abi.lib().lrkv_key_norms(_ptr(positions), _ptr(seq_ids), positions.shape[0], _ptr(B_K),
                                     ctypes.byref(desc), _ptr(page_table), B, max_pages,
                                     _ptr(status), _stream(stream))
    _abi.check("lrkv_key_norms", code)
