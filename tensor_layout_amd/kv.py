"""Paged key/value cache: rotation and appending of new tokens, and attention.

``PagedCache`` names the two pools of pages that a program holds (and the
scales of an e4m3 one); ``append`` rotates a batch's new keys and queries to
their positions and writes keys and values into their pages; ``attend`` lets
the queries attend to what the cache holds, and ``attend_shared`` does so for
sequences that share their first tokens; ``read`` takes tokens out of the pages
again.  A batch is packed: sequence ``b``
owns rows ``starts[b]:starts[b + 1]`` of the token tensors, ``lengths[b]``
tokens with those, and the pages that its row of ``table`` names in order (a
negative entry is a page that is not there).  Rows of no sequence, and of one
that is skipped because its numbers are out of order, are left as they are.
All run on torch's current stream, or a named one, without waiting, read
``table``, ``starts``, ``lengths`` and groups on the device only, and may be captured
into a graph.

Arguments are checked here for their types and shapes, and by the C entry
points of include/tpl_kv.h, which every call ends in; a refused call raises
``TplError`` and has launched nothing.
"""

from __future__ import annotations

import ctypes
import struct
from typing import Optional, Sequence

import torch

from . import tpl
from .tpl import TplError

BF16, FP16, E4M3 = 0, 1, 2
MAX_AXES = 4
COUNTERS = 4096   # TPL_KV_COUNTERS: the bytes of a workspace that a call finds zero and leaves zero

EXPORTED = ("tpl_kv_append", "tpl_kv_attend", "tpl_kv_attend_workspace", "tpl_kv_attend_shared",
            "tpl_kv_attend_shared_workspace", "tpl_kv_read")

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


class Rows(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("k", "v")] + [(n, _I64) for n in ("k_token", "k_head", "v_token", "v_head")] + [("type", _I32)])


class Groups(ctypes.Structure):
    _fields_ = [("groups", _P), ("shared", _P), ("count", _I32)]


# The same layouts for packing a call's numbers in one go.
_pack_batch = struct.Struct("3Pq3i4x").pack
_pack_new = struct.Struct("6P9q5i4i4x").pack
_pack_query = struct.Struct("3P6qf4i4x").pack
_pack_rows = struct.Struct("2P4qi4x").pack
_pack_groups = struct.Struct("2Pi4x").pack

# attend's workspaces: (address, bytes, tensor) by device, then stream.
_workspaces = {}

_lib = None
_calls = []   # as EXPORTED
_append = _attend = _attend_shared = _read = None   # the extension's, which read the tensors too


def load():
    """libtpl.so with this module's entry points declared."""
    global _lib, _append, _attend, _attend_shared, _read
    if _lib is None:
        lib = tpl.load()
        held = ctypes.PyDLL(lib._name)
        c, b, n, q, r, g = (ctypes.POINTER(x) for x in (Cache, Batch, New, Query, Rows, Groups))
        for name, args, rest, res in (("tpl_kv_append", [n], [_P], ctypes.c_int),
                                      ("tpl_kv_attend", [q], [_P, _I64, _P], ctypes.c_int),
                                      ("tpl_kv_attend_workspace", [q], [], _I64),
                                      ("tpl_kv_attend_shared", [g, q], [_P, _I64, _P], ctypes.c_int),
                                      ("tpl_kv_attend_shared_workspace", [g, q], [], _I64),
                                      ("tpl_kv_read", [r], [_P], ctypes.c_int)):
            f = getattr(lib, name)
            f.argtypes, f.restype = [c, b] + args + rest, res
            # A second handle, which takes packed bytes in the structures' places.  It keeps the interpreter's lock, as
            # the extension does: the launches of one call follow one another on a stream whose workspace others use.
            f = held[name]
            f.argtypes, f.restype = [_P] * (2 + len(args)) + rest, res
            _calls.append(f)
        try:
            from . import _kv_call
        except ImportError as e:
            raise RuntimeError("tensor_layout_amd/_kv_call.so is missing or was built for another torch: build it "
                               "(python -c 'import __graft_entry__ as g; g.build()')") from e
        _kv_call.bind(*(ctypes.cast(getattr(lib, n), _P).value for n in EXPORTED))
        _append, _attend, _attend_shared, _read = _kv_call.append, _kv_call.attend, _kv_call.attend_shared, _kv_call.read
        _lib = lib
    return _lib


# The current device and a stream's handle without building the objects that
# the public functions return (1 us a call) where this torch has them.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
           or (lambda index: torch.cuda.current_stream(index).cuda_stream))

_TYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float8_e4m3fn: E4M3}
_INT32 = torch.int32
_FLOAT_MAX = torch.finfo(torch.float32).max


def _need(ok: bool, message: str, status: int = tpl.TPL_E_ARG) -> None:
    if not ok:
        raise TplError(status, message)


# The checks come in two forms: a call first asks whether everything is right
# (_ints_ok, _heads_ok), and only for one that is not looks for what is wrong.


def _ints_ok(t, index, *shape):
    """Whether `t` is an array of 32-bit numbers on the device; None in `shape` is any size."""
    s = t.shape
    if t.dtype is not _INT32 or t.get_device() != index or len(s) != len(shape):
        return False
    for w, x in zip(shape, s):
        if w is not None and w != x:
            return False
    return s[-1] < 2 or t.stride(-1) == 1


def _ints(name, t, device, *shape):
    _need(t.dtype == torch.int32, f"{name} must be int32", tpl.TPL_E_DTYPE)
    s = t.shape
    _need(len(s) == len(shape) and all(w is None or w == x for w, x in zip(shape, s)),
          f"{name} has shape {tuple(s)}", tpl.TPL_E_EXTENT)
    _need(t.device == device, f"{name} must be on {device}")
    _need(s[-1] < 2 or t.stride(-1) == 1, f"{name} must be contiguous", tpl.TPL_E_LAYOUT)


def _heads_ok(t, dtype, index, shape):
    """Whether `t` is a [tokens, heads, dim] tensor of this type whose channels are contiguous."""
    return t.dtype is dtype and t.get_device() == index and t.shape == shape and t.stride(2) == 1


def _heads(name, t, dtype, device, shape):
    _need(t.dim() == 3 and tuple(t.shape) == tuple(shape), f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}",
          tpl.TPL_E_EXTENT)
    _need(t.dtype == dtype, f"{name} is {t.dtype}, not {dtype}", tpl.TPL_E_DTYPE)
    _need(t.device == device, f"{name} must be on {device}")
    _need(t.stride(2) == 1, f"{name}'s channels must be contiguous", tpl.TPL_E_LAYOUT)


class PagedCache:
    """The pools ``k`` and ``v`` [pages, page, kv_heads, dim], in bf16 or fp16, or in
    e4m3 with ``k_scale`` and ``v_scale`` [pages, kv_heads, page / block] in fp32.

    Any order in memory is taken as long as a head's channels are contiguous
    and pages, tokens and heads lie on 16 bytes: [pages, kv_heads, page, dim]
    storage goes in as its transposed view.  The object keeps the tensors and
    their sizes and strides, nothing of their values.  The workspaces that
    ``attend`` needs are one for each device and stream, shared by all caches
    (a model has one a layer) and kept for the next call."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _need(k.dim() == 4 and tuple(k.shape) == tuple(v.shape), "k and v must be [pages, page, kv_heads, dim]",
              tpl.TPL_E_EXTENT)
        _need(k.dtype in _TYPES and k.dtype == v.dtype, "a cache holds bf16, fp16 or e4m3", tpl.TPL_E_DTYPE)
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
                        _TYPES[k.dtype], page, block, kv_heads, dim)
        self._at = ctypes.addressof(self._c)
        self._index = k.get_device()
        self._work = _workspaces.setdefault(self._index, {})


def _batch(cache, table, starts, lengths, tokens):
    index = cache._index
    if not (_ints_ok(table, index, None, None) and _ints_ok(starts, index, table.shape[0] + 1)
            and _ints_ok(lengths, index, table.shape[0])):
        device = cache.device
        _ints("table", table, device, None, None)
        _ints("starts", starts, device, table.shape[0] + 1)
        _ints("lengths", lengths, device, table.shape[0])
    n, width = table.shape
    return n, width, _pack_batch(table.data_ptr(), starts.data_ptr(), lengths.data_ptr(), table.stride(0), n, width, tokens)


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
    stream        the handle of the stream to run on (default: torch's current one).

    ``lengths`` counts the new tokens.  Returns ``q_out``."""
    if _lib is None:
        load()
    if q is not None and q_out is None:
        q_out = _result(q, cache, stream)
    index = cache._index
    if index >= 0 and _device() == index:
        status = _append(cache._at, index, k, v, table, starts, lengths, q, q_out, inv_freq, positions, sections, interleaved,
                         _stream(index) if stream is None else int(stream))
        if status == 0:
            return q_out
        if status > 0:
            _raise(status)
    return _append_checked(cache, k, v, table, starts, lengths, q, q_out, inv_freq, positions, sections, interleaved, stream)


def _append_checked(cache, k, v, table, starts, lengths, q, q_out, inv_freq, positions, sections, interleaved, stream):
    """The same, each argument by itself: says what is wrong, or makes the call."""
    index, dtype = cache._index, k.dtype
    tokens = k.shape[0] if k.dim() else 0
    shape = (tokens, cache.kv_heads, cache.dim)
    if not (dtype in _TYPES and dtype is not torch.float8_e4m3fn and _heads_ok(k, dtype, index, shape)
            and _heads_ok(v, dtype, index, shape)):
        _need(k.dim() == 3, "k must be [tokens, kv_heads, dim]", tpl.TPL_E_EXTENT)
        _need(dtype in (torch.bfloat16, torch.float16), "k must be bf16 or fp16", tpl.TPL_E_DTYPE)
        _heads("k", k, dtype, cache.device, shape)
        _heads("v", v, dtype, cache.device, shape)
    n, width, batch = _batch(cache, table, starts, lengths, tokens)
    qp = op = qt = qh = ot = oh = heads = 0
    if q is not None:
        heads = q.shape[1] if q.dim() == 3 else 0
        shape = (tokens, heads, cache.dim)
        if not (_heads_ok(q, dtype, index, shape) and _heads_ok(q_out, dtype, index, shape)):
            _need(q.dim() == 3, "q must be [tokens, heads, dim]", tpl.TPL_E_EXTENT)
            _heads("q", q, dtype, cache.device, shape)
            _heads("q_out", q_out, dtype, cache.device, shape)
        qp, op = q.data_ptr(), q_out.data_ptr()
        qt, qh, _ = q.stride()
        ot, oh, _ = q_out.stride()
    elif q_out is not None:
        _need(False, "q_out needs q")
    fp = rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        if not (inv_freq.dtype is torch.float32 and inv_freq.get_device() == index and inv_freq.dim() == 1
                and (rot < 4 or inv_freq.stride(0) == 1)):
            _need(inv_freq.dtype == torch.float32, "inv_freq must be fp32", tpl.TPL_E_DTYPE)
            _need(inv_freq.device == cache.device, f"inv_freq must be on {cache.device}")
            _need(False, "inv_freq must be one contiguous row", tpl.TPL_E_LAYOUT)
        fp = inv_freq.data_ptr()
    pp, row, axes, parts = 0, 0, 1, (0, 0, 0, 0)
    if positions is not None:
        if not _ints_ok(positions, index, None, tokens):
            _ints("positions", positions, cache.device, None, tokens)
        pp, row, axes = positions.data_ptr(), positions.stride(0), positions.shape[0]
        _need(1 <= axes <= MAX_AXES, "positions must have 1 .. 4 axes")
        _need(axes == (1 if sections is None else len(sections)), "sections must have one number for each axis")
    if sections is not None:
        _need(positions is not None, "sections need positions")
        _need(inv_freq is not None, "sections need inv_freq")
        _need(sum(sections) * 2 == rot and min(sections) >= 0, "sections must add up to the rotated pairs")
        parts = (*sections, 0, 0, 0, 0)[:4]
    kt, kh, _ = k.stride()
    vt, vh, _ = v.stride()
    args = _pack_new(k.data_ptr(), v.data_ptr(), qp, op, fp, pp, kt, kh, vt, vh, qt, qh, ot, oh, row,
                     _TYPES[dtype], heads, rot, bool(interleaved), axes, *parts)
    _need(index >= 0, "tensors must live on the GPU")
    if _device() == index:
        s = _stream(index) if stream is None else int(stream)
        status = _calls[0](cache._at, batch, args, s)
    else:
        with torch.cuda.device(index):
            s = _stream(index) if stream is None else int(stream)
            status = _calls[0](cache._at, batch, args, s)
    if status:
        _raise(status)
    return q_out


def _workspace(cache, call, *args):
    """Of `call` (1: attend, 3: attend_shared) for these packed arguments."""
    load()
    size = _calls[call + 1](cache._at, *args)
    if size < 0:
        _raise(_calls[call](cache._at, *args, None, 0, None))   # refused the same way, before anything is looked at on the device
    return size


def _on(cache, s, stream):
    """The call's stream as torch's current one: `s`, where the call names it."""
    return torch.cuda.stream(None if stream is None else torch.cuda.ExternalStream(s, device=cache.device))


def _result(q, cache, stream):
    """A new tensor like `q` for the call to write: memory of the call's own stream, not what the current one has just given back."""
    if stream is None or cache._index < 0:
        return torch.empty_like(q, memory_format=torch.contiguous_format)
    with _on(cache, int(stream), stream):
        return torch.empty_like(q, memory_format=torch.contiguous_format)


def _capturing(cache, s, stream):
    """Whether the call's own stream is being captured, whatever torch's current one is."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with _on(cache, s, stream):
        return torch.cuda.is_current_stream_capturing()


def _attend_packed(cache, call, args, size, stream):
    """The call itself, with a workspace of the stream's own."""
    index = cache._index
    s = _stream(index) if stream is None else int(stream)
    ws = cache._work.get(s)
    if ws is None or ws[1] < size or _capturing(cache, s, stream):
        ws = _new_workspace(cache, size, s, stream)
    return _calls[call](cache._at, *args, ws[0], size, s)


def _new_workspace(cache, size, s, stream):
    """(address, size, tensor), its counters cleared once: every call leaves them zero.

    Calls on one stream follow one another and share it, whatever their caches.  A captured call has
    one to itself, whose counters the graph clears: it may be replayed beside eager
    calls on the stream it was captured on."""
    with _on(cache, s, stream):
        capturing = torch.cuda.is_current_stream_capturing()
        t = torch.empty(size if capturing else max(size, 1 << 20), dtype=torch.uint8, device=cache.device)
        t[:COUNTERS].zero_()
        ws = (t.data_ptr(), t.numel(), t)
        if not capturing:
            cache._work[s] = ws
    return ws


def attend(q, cache: PagedCache, table, starts, lengths, *, scale: Optional[float] = None, window: int = 0,
           sinks: int = 0, out=None, lse=None, stream: Optional[int] = None):
    """softmax(scale * q k^T) v for each row of ``q`` [tokens, heads, dim] over its sequence's tokens in the cache.

    A row at position p sees tokens 0 .. p; with a ``window``, the last ``window`` of them and the first ``sinks``.
    Query head h reads head h // (heads / kv_heads) of the cache.

    scale   default dim ** -0.5.
    out     takes the result (default: a new tensor).
    lse     fp32 [tokens, heads]: takes the logarithm of each row's sum of exponentials.
    stream  the handle of the stream to run on (default: torch's current one).

    A row that sees nothing gets zeros and an lse of minus infinity.  Returns ``out``."""
    if _lib is None:
        load()
    if out is None:
        out = _result(q, cache, stream)
    index = cache._index
    if index >= 0 and _device() == index:
        s = _stream(index) if stream is None else int(stream)
        ws = cache._work.get(s)
        if ws is not None and not _capturing(cache, s, stream):
            status = _attend(cache._at, index, q, table, starts, lengths, scale, window, sinks, out, lse, ws[0], ws[1], s)
            if status == 0:
                return out
            if status > 0:
                _raise(status)
    return _attend_checked(q, cache, table, starts, lengths, None, None, scale, window, sinks, out, lse, stream)


def attend_shared(q, cache: PagedCache, table, starts, lengths, groups, shared, *, scale: Optional[float] = None, out=None,
                  lse=None, stream: Optional[int] = None):
    """``attend`` for sequences that share their first tokens, which are read and multiplied once for all of a group's rows.

    groups  int32 [n + 1]: group g is sequences groups[g] .. groups[g + 1] - 1.
    shared  int32 [n]: how many first tokens they share, held in the pages that their first one's row of ``table`` names.

    From there on each sequence has the tokens of its own row of ``table``.  A sequence in no group, or with new tokens
    among the shared ones, attends by itself to its own row's pages, which has the same result where those begin with the
    shared pages (a page that is shared in part is copied: ``read``, ``append``).  Groups follow one another: rows of two
    that overlap have no defined result.

    The rest is ``attend``'s; there is no window.  Returns ``out``."""
    if _lib is None:
        load()
    if out is None:
        out = _result(q, cache, stream)
    index = cache._index
    if index >= 0 and _device() == index:
        s = _stream(index) if stream is None else int(stream)
        ws = cache._work.get(s)
        if ws is not None and not _capturing(cache, s, stream):
            status = _attend_shared(cache._at, index, q, table, starts, lengths, groups, shared, scale, out, lse, ws[0], ws[1], s)
            if status == 0:
                return out
            if status > 0:
                _raise(status)
    return _attend_checked(q, cache, table, starts, lengths, groups, shared, scale, 0, 0, out, lse, stream)


def _attend_checked(q, cache, table, starts, lengths, groups, shared, scale, window, sinks, out, lse, stream):
    """The same, each argument by itself: says what is wrong, or makes the call, with a new workspace where it needs one."""
    index, dtype = cache._index, q.dtype
    shape = q.shape
    if not (len(shape) == 3 and shape[2] == cache.dim and dtype in _TYPES and dtype is not torch.float8_e4m3fn
            and _heads_ok(q, dtype, index, shape)):
        _need(q.dim() == 3, "q must be [tokens, heads, dim]", tpl.TPL_E_EXTENT)
        _need(dtype in (torch.bfloat16, torch.float16), "q must be bf16 or fp16", tpl.TPL_E_DTYPE)
        _heads("q", q, dtype, cache.device, (shape[0], shape[1], cache.dim))
    tokens, heads, dim = shape
    if not _heads_ok(out, dtype, index, shape):
        _heads("out", out, dtype, cache.device, shape)
    n, width, batch = _batch(cache, table, starts, lengths, tokens)
    lp = lt = lh = 0
    if lse is not None:
        if not (lse.dtype is torch.float32 and lse.shape == (tokens, heads) and lse.get_device() == index):
            _need(lse.dtype == torch.float32, "lse must be fp32", tpl.TPL_E_DTYPE)
            _need(tuple(lse.shape) == (tokens, heads), f"lse has shape {tuple(lse.shape)}", tpl.TPL_E_EXTENT)
            _need(False, f"lse must be on {cache.device}")
        lp = lse.data_ptr()
        lt, lh = lse.stride()
    scale = dim ** -0.5 if scale is None else scale
    # What the structure can hold; the entry point judges it.
    _need(-_FLOAT_MAX <= scale <= _FLOAT_MAX, "scale must be a finite number over zero")
    _need(abs(window) < 1 << 31 and abs(sinks) < 1 << 31, "window and sinks must be 0 .. 2^30")
    qt, qh, _ = q.stride()
    ot, oh, _ = out.stride()
    args = _pack_query(q.data_ptr(), out.data_ptr(), lp, qt, qh, ot, oh, lt, lh, scale,
                       _TYPES[dtype], heads, window, sinks)
    call, packed = 1, (batch, args)
    if groups is not None:
        if not (_ints_ok(groups, index, None) and groups.shape[0] > 0 and _ints_ok(shared, index, groups.shape[0] - 1)):
            _ints("groups", groups, cache.device, None)
            _need(groups.shape[0] > 0, "groups must have a number more than there are groups", tpl.TPL_E_EXTENT)
            _ints("shared", shared, cache.device, groups.shape[0] - 1)
        call, packed = 3, (batch, _pack_groups(groups.data_ptr(), shared.data_ptr(), shared.shape[0]), args)
    size = _workspace(cache, call, *packed)
    _need(index >= 0, "tensors must live on the GPU")
    if _device() == index:
        status = _attend_packed(cache, call, packed, size, stream)
    else:
        with torch.cuda.device(index):
            status = _attend_packed(cache, call, packed, size, stream)
    if status:
        _raise(status)
    return out


def read(cache: PagedCache, table, starts, lengths, k=None, v=None, *, stream: Optional[int] = None) -> None:
    """Write each sequence's last tokens, as many as it has rows, out of the cache into ``k`` and ``v`` [tokens, kv_heads, dim].

    They are what ``append`` with the same ``table``, ``starts`` and ``lengths`` wrote: an e4m3 value times its block's
    scale, rounded once to the tensors' type (bf16 or fp16); a 16-bit cache is read as its own type, bit for bit.  Other
    tokens are read by naming other lengths: ``lengths`` = n and n rows read a sequence's first n.  Either of ``k`` and
    ``v`` may be None; they must not lie over each other.  A token whose page is not there gives zeros."""
    if _lib is None:
        load()
    index = cache._index
    if index >= 0 and _device() == index:
        status = _read(cache._at, index, table, starts, lengths, k, v, _stream(index) if stream is None else int(stream))
        if status == 0:
            return
        if status > 0:
            _raise(status)
    _need(k is not None or v is not None, "k and v must not both be None")
    some = v if k is None else k
    _need(some.dim() == 3, "k and v must be [tokens, kv_heads, dim]", tpl.TPL_E_EXTENT)
    _need(some.dtype in (torch.bfloat16, torch.float16), "k and v must be bf16 or fp16", tpl.TPL_E_DTYPE)
    tokens = some.shape[0]
    ptr, strides = [], []
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _heads(name, t, some.dtype, cache.device, (tokens, cache.kv_heads, cache.dim))
        ptr.append(0 if t is None else t.data_ptr())
        strides += (0, 0) if t is None else t.stride()[:2]
    _, _, batch = _batch(cache, table, starts, lengths, tokens)
    args = _pack_rows(*ptr, *strides, _TYPES[some.dtype])
    _need(index >= 0, "tensors must live on the GPU")
    with torch.cuda.device(index):
        status = _calls[5](cache._at, batch, args, _stream(index) if stream is None else int(stream))
    if status:
        _raise(status)
