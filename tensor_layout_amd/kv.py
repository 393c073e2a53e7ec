"""Paged key/value cache: rotation and appending of new tokens, and attention.

``PagedCache`` names the two pools of pages that a program holds (and the
scales of an e4m3 one); ``append`` rotates a batch's new keys and queries to
their positions and writes keys and values into their pages; ``attend`` lets
the queries attend to what the cache holds.  A batch is packed: sequence ``b``
owns rows ``starts[b]:starts[b + 1]`` of the token tensors, ``lengths[b]``
tokens with those, and the pages that its row of ``table`` names in order (a
negative entry is a page that is not there).  Both run on torch's current
stream without waiting, read ``table``, ``starts`` and ``lengths`` on the
device only, and may be captured into a graph.

Arguments are checked here for their types and shapes, and by the C entry
points of include/tpl_kv.h, which every call ends in; a refused call raises
``TplError`` and has launched nothing.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

from . import tpl
from .tpl import TplError

BF16, FP16, E4M3 = 0, 1, 2
MAX_AXES = 4

EXPORTED = ("tpl_kv_append", "tpl_kv_attend", "tpl_kv_attend_workspace")

_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Cache(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("k", "v", "k_scale", "v_scale")]
                + [(n, _I64) for n in ("pages", "k_page", "k_token", "k_head", "v_page", "v_token", "v_head",
                                       "ks_page", "ks_head", "ks_block", "vs_page", "vs_head", "vs_block")]
                + [(n, _I32) for n in ("type", "page", "block", "kv_heads", "dim")])


class Batch(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("table", "starts", "lengths")] + [("table_row", _I64)]
                + [(n, _I32) for n in ("batch", "width", "tokens")])


class New(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("k", "v", "q", "q_out", "inv_freq", "positions")]
                + [(n, _I64) for n in ("k_token", "k_head", "v_token", "v_head", "q_token", "q_head", "o_token",
                                       "o_head", "positions_row")]
                + [(n, _I32) for n in ("type", "heads", "rot", "interleaved", "axes")]
                + [("sections", _I32 * MAX_AXES)])


class Query(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("q", "out", "lse")]
                + [(n, _I64) for n in ("q_token", "q_head", "o_token", "o_head", "l_token", "l_head")]
                + [("scale", ctypes.c_float)] + [(n, _I32) for n in ("type", "heads", "window", "sinks")])


_lib = None


def load():
    """libtpl.so with this module's entry points declared."""
    global _lib
    if _lib is None:
        lib = tpl.load()
        c, b = ctypes.POINTER(Cache), ctypes.POINTER(Batch)
        lib.tpl_kv_append.argtypes = [c, b, ctypes.POINTER(New), _P]
        lib.tpl_kv_append.restype = ctypes.c_int
        lib.tpl_kv_attend.argtypes = [c, b, ctypes.POINTER(Query), _P, _I64, _P]
        lib.tpl_kv_attend.restype = ctypes.c_int
        lib.tpl_kv_attend_workspace.argtypes = [c, b, ctypes.POINTER(Query)]
        lib.tpl_kv_attend_workspace.restype = _I64
        _lib = lib
    return _lib


_types = None


def _type(t) -> int:
    """The C type of a tensor's dtype, or -1."""
    global _types
    if _types is None:
        import torch
        _types = {torch.bfloat16: BF16, torch.float16: FP16, torch.float8_e4m3fn: E4M3}
    return _types.get(t.dtype, -1)


def _need(ok: bool, message: str, status: int = tpl.TPL_E_ARG) -> None:
    if not ok:
        raise TplError(status, message)


def _ints(name, t, device, *shape):
    """A device array of 32-bit numbers; None in `shape` is any size."""
    import torch
    _need(t.dtype == torch.int32, f"{name} must be int32", tpl.TPL_E_DTYPE)
    s = t.shape
    _need(len(s) == len(shape) and all(w is None or w == x for w, x in zip(shape, s)),
          f"{name} has shape {tuple(s)}", tpl.TPL_E_EXTENT)
    _need(t.device == device, f"{name} must be on {device}")
    _need(s[-1] < 2 or t.stride(-1) == 1, f"{name} must be contiguous", tpl.TPL_E_LAYOUT)


def _heads(name, t, like, tokens, heads, dim):
    """A [tokens, heads, dim] tensor of `like`'s type whose channels are contiguous."""
    _need(tuple(t.shape) == (tokens, heads, dim), f"{name} has shape {tuple(t.shape)}, not {(tokens, heads, dim)}",
          tpl.TPL_E_EXTENT)
    _need(t.dtype == like.dtype, f"{name} is {t.dtype}, not {like.dtype}", tpl.TPL_E_DTYPE)
    _need(t.device == like.device, f"{name} must be on {like.device}")
    _need(t.stride(2) == 1, f"{name}'s channels must be contiguous", tpl.TPL_E_LAYOUT)


class PagedCache:
    """The pools ``k`` and ``v`` [pages, page, kv_heads, dim], in bf16 or fp16, or in
    e4m3 with ``k_scale`` and ``v_scale`` [pages, kv_heads, page / block] in fp32.

    Any order in memory is taken as long as a head's channels are contiguous
    and pages, tokens and heads lie on 16 bytes: [pages, kv_heads, page, dim]
    storage goes in as its transposed view.  The object keeps the tensors and
    their sizes and strides, nothing of their values."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        _need(k.dim() == 4 and tuple(k.shape) == tuple(v.shape), "k and v must be [pages, page, kv_heads, dim]",
              tpl.TPL_E_EXTENT)
        _need(_type(k) >= 0 and k.dtype == v.dtype, "a cache holds bf16, fp16 or e4m3", tpl.TPL_E_DTYPE)
        _need(k.device == v.device, "k and v must be on one device")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "the channels of a head must be contiguous", tpl.TPL_E_LAYOUT)
        pages, page, kv_heads, dim = k.shape
        strides, block, ptr = [0] * 6, 0, [None, None]
        if k.dtype == torch.float8_e4m3fn:
            _need(k_scale is not None and v_scale is not None, "an e4m3 cache needs its scales")
            for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
                _need(s.dtype == torch.float32, f"{name} must be fp32", tpl.TPL_E_DTYPE)
                _need(s.device == k.device, f"{name} must be on {k.device}")
                _need(s.dim() == 3 and tuple(s.shape) == tuple(k_scale.shape) and tuple(s.shape[:2]) == (pages, kv_heads)
                      and s.shape[2] >= 1 and page % s.shape[2] == 0,
                      f"{name} must be [pages, kv_heads, page / block]", tpl.TPL_E_EXTENT)
            block = page // k_scale.shape[2]
            strides = [*k_scale.stride(), *v_scale.stride()]
            ptr = [k_scale.data_ptr(), v_scale.data_ptr()]
        else:
            _need(k_scale is None and v_scale is None, "only an e4m3 cache has scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.kv_heads, self.dim, self.page, self.block = k.device, kv_heads, dim, page, block
        self._c = Cache(k.data_ptr(), v.data_ptr(), *ptr, pages, *k.stride()[:3], *v.stride()[:3], *strides,
                        _type(k), page, block, kv_heads, dim)
        self._ref = ctypes.byref(self._c)


def _batch(cache, table, starts, lengths, tokens):
    device = cache.device
    _ints("table", table, device, None, None)
    n, width = table.shape
    _ints("starts", starts, device, n + 1)
    _ints("lengths", lengths, device, n)
    return Batch(table.data_ptr(), starts.data_ptr(), lengths.data_ptr(), table.stride(0), n, width, tokens)


class _On:
    """The device of a call made current, and its stream."""

    def __init__(self, device, stream):
        import torch
        _need(device.type == "cuda", "tensors must live on the GPU")
        self.stream = torch.cuda.current_stream(device).cuda_stream if stream is None else int(stream)
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.stream

    def __exit__(self, *a):
        if self.guard is not None:
            self.guard.__exit__(*a)


def _raise(status):
    raise TplError(status, tpl.tpl_last_error() or tpl.tpl_status_string(status))


def append(cache: PagedCache, k, v, table, starts, lengths, *, q=None, q_out=None, inv_freq=None, positions=None,
           sections: Optional[Sequence[int]] = None, interleaved: bool = False, stream: Optional[int] = None):
    """Rotate ``k`` [tokens, kv_heads, dim] and ``q`` [tokens, heads, dim] and write ``k`` and ``v`` into the cache.

    inv_freq      fp32 [rot / 2]: the first ``rot`` channels of each head turn, pair c by position * inv_freq[c];
                  None: nothing turns.
    positions     int32 [axes, tokens]; None: each token's index in its sequence.
    sections      with more axes than one, how many pairs turn by each, in order.
    interleaved   pairs are channels (2c, 2c + 1), otherwise (c, c + rot / 2).
    q_out         takes the rotated queries (default: a new tensor); may be ``q``.

    ``lengths`` counts the new tokens.  Returns ``q_out``."""
    import torch
    _need(k.dim() == 3, "k must be [tokens, kv_heads, dim]", tpl.TPL_E_EXTENT)
    tokens, device = k.shape[0], cache.device
    t = _type(k)
    _need(t in (BF16, FP16), "k must be bf16 or fp16", tpl.TPL_E_DTYPE)
    _need(k.device == device, f"k must be on {device}")
    _heads("k", k, k, tokens, cache.kv_heads, cache.dim)
    _heads("v", v, k, tokens, cache.kv_heads, cache.dim)
    batch = _batch(cache, table, starts, lengths, tokens)
    a = New(k.data_ptr(), v.data_ptr())
    a.k_token, a.k_head, _ = k.stride()
    a.v_token, a.v_head, _ = v.stride()
    a.type, a.axes = t, 1
    if q is not None:
        _need(q.dim() == 3, "q must be [tokens, heads, dim]", tpl.TPL_E_EXTENT)
        heads = q.shape[1]
        _heads("q", q, k, tokens, heads, cache.dim)
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        _heads("q_out", q_out, k, tokens, heads, cache.dim)
        a.q, a.q_out, a.heads = q.data_ptr(), q_out.data_ptr(), heads
        a.q_token, a.q_head, _ = q.stride()
        a.o_token, a.o_head, _ = q_out.stride()
    else:
        _need(q_out is None, "q_out needs q")
    if inv_freq is not None:
        _need(inv_freq.dtype == torch.float32, "inv_freq must be fp32", tpl.TPL_E_DTYPE)
        _need(inv_freq.device == device, f"inv_freq must be on {device}")
        _need(inv_freq.dim() == 1 and inv_freq.is_contiguous(), "inv_freq must be one contiguous row", tpl.TPL_E_LAYOUT)
        a.inv_freq, a.rot, a.interleaved = inv_freq.data_ptr(), 2 * inv_freq.shape[0], bool(interleaved)
    if positions is not None:
        _ints("positions", positions, device, None, tokens)
        a.positions, a.positions_row, axes = positions.data_ptr(), positions.stride(0), positions.shape[0]
        _need(1 <= axes <= MAX_AXES, f"positions must have 1 .. {MAX_AXES} axes")
        _need(axes == (len(sections) if sections is not None else 1), "sections must have one number for each axis")
        a.axes = axes
    if sections is not None:
        _need(positions is not None, "sections need positions")
        _need(inv_freq is not None, "sections need inv_freq")
        _need(sum(sections) * 2 == a.rot and all(x >= 0 for x in sections), "sections must add up to the rotated pairs")
        for i, x in enumerate(sections):
            a.sections[i] = x
    with _On(device, stream) as s:
        status = (_lib or load()).tpl_kv_append(cache._ref, ctypes.byref(batch), ctypes.byref(a), s)
    if status:
        _raise(status)
    return q_out


def attend(q, cache: PagedCache, table, starts, lengths, *, scale: Optional[float] = None, window: int = 0,
           sinks: int = 0, out=None, lse=None, stream: Optional[int] = None):
    """softmax(scale * q k^T) v for each row of ``q`` [tokens, heads, dim] over its sequence's tokens in the cache.

    A row at position p sees tokens 0 .. p; with a ``window``, the last ``window`` of them and the first ``sinks``.
    Query head h reads head h // (heads / kv_heads) of the cache.

    scale   default dim ** -0.5.
    out     takes the result (default: a new tensor).
    lse     fp32 [tokens, heads]: takes the logarithm of each row's sum of exponentials.

    A row that sees nothing gets zeros and an lse of minus infinity.  Returns ``out``."""
    import torch
    _need(q.dim() == 3, "q must be [tokens, heads, dim]", tpl.TPL_E_EXTENT)
    tokens, heads, dim = q.shape
    device = cache.device
    t = _type(q)
    _need(t in (BF16, FP16), "q must be bf16 or fp16", tpl.TPL_E_DTYPE)
    _need(q.device == device, f"q must be on {device}")
    _heads("q", q, q, tokens, heads, cache.dim)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _heads("out", out, q, tokens, heads, dim)
    batch = _batch(cache, table, starts, lengths, tokens)
    a = Query(q.data_ptr(), out.data_ptr())
    a.q_token, a.q_head, _ = q.stride()
    a.o_token, a.o_head, _ = out.stride()
    a.scale = dim ** -0.5 if scale is None else scale
    a.type, a.heads, a.window, a.sinks = t, heads, window, sinks
    if lse is not None:
        _need(lse.dtype == torch.float32, "lse must be fp32", tpl.TPL_E_DTYPE)
        _need(tuple(lse.shape) == (tokens, heads), f"lse has shape {tuple(lse.shape)}", tpl.TPL_E_EXTENT)
        _need(lse.device == device, f"lse must be on {device}")
        a.lse = lse.data_ptr()
        a.l_token, a.l_head = lse.stride()
    lib = _lib or load()
    b, r = ctypes.byref(batch), ctypes.byref(a)
    size = lib.tpl_kv_attend_workspace(cache._ref, b, r)
    if size < 0:
        raise TplError(tpl.TPL_E_ARG, tpl.tpl_last_error())
    with _On(device, stream) as s:
        # The workspace is the call's own: the allocator gives it to nobody
        # else until this stream's work has passed.
        if stream is None:
            ws = torch.empty(size, dtype=torch.uint8, device=device)
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(s, device=device)):
                ws = torch.empty(size, dtype=torch.uint8, device=device)
        status = lib.tpl_kv_attend(cache._ref, b, r, ws.data_ptr(), size, s)
    if status:
        _raise(status)
    return out
