"""Linear attention with a decay for each head over a pool of states.

``StatePool`` names what a layer keeps between calls: slots of one state a head
and the heads' decays.  ``attend`` takes a batch's new queries, keys and values
through the recurrence

    S = exp(decay) S + k v^T,    out = scale * q S

for each of a sequence's tokens in order, prompts in chunks through the matrix
units, a few tokens one by one.  A batch is packed as those of ``kv`` are:
sequence ``b`` owns rows ``starts[b]:starts[b + 1]``, reads the state of slot
``sources[b]`` and writes that of slot ``slots[b]``.  Rows of no sequence, and of
one that is skipped because its numbers are out of order, are left as they are.
It runs on torch's current stream, or a named one, without waiting, reads
``slots``, ``sources`` and ``starts`` on the device only, and may be captured
into a graph.

Arguments are checked here for their types and shapes, and by the C entry point
of include/tpl_linear.h, which every call ends in; a refused call raises
``TplError`` and has launched nothing.
"""

from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import kv, tpl
from .kv import _P, _FLOAT_MAX, _I32, _I64, _device, _heads, _ints, _need, _raise, _stream

EXPORTED = ("tpl_linear_attend", "tpl_linear_attend_workspace")


class Pool(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("state", "decay")] + [(n, _I64) for n in ("s_slot", "s_head", "s_key", "slots")]
                + [(n, _I32) for n in ("heads", "key_dim", "value_dim")])


class Batch(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("slots", "sources", "starts")] + [(n, _I32) for n in ("batch", "tokens")]


class New(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("q", "k", "v", "out")]
                + [(n, _I64) for n in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head", "o_token", "o_head")]
                + [("scale", ctypes.c_float)] + [(n, _I32) for n in ("type", "key_heads")])


# The same layouts for packing a call's numbers in one go.
_pack_batch = struct.Struct("3P2i").pack
_pack_new = struct.Struct("4P8qf2i4x").pack

_lib = None
_calls = []   # as EXPORTED
_attend = None   # the extension's, which reads the tensors too


def load():
    """libtpl.so with this module's entry points declared."""
    global _lib, _attend
    if _lib is None:
        lib = kv.load()
        held = ctypes.PyDLL(lib._name)
        for name, rest, res in (("tpl_linear_attend", [_P, _I64, _P], ctypes.c_int), ("tpl_linear_attend_workspace", [], _I64)):
            f = getattr(lib, name)
            f.argtypes, f.restype = [ctypes.POINTER(x) for x in (Pool, Batch, New)] + rest, res
            f = held[name]   # takes packed bytes in the structures' places
            f.argtypes, f.restype = [_P, _P, _P] + rest, res
            _calls.append(f)
        from . import _kv_call
        _kv_call.bind_linear(*(ctypes.cast(getattr(lib, n), _P).value for n in EXPORTED))
        _attend = _kv_call.linear_attend
        _lib = lib
    return _lib


class StatePool:
    """States [slots, heads, key_dim, value_dim] in fp32, and ``decay`` fp32 [heads]: logarithms, at most zero (what is over it counts as zero).

    Any order in memory is taken as long as a state's value channels are contiguous and slots, heads and key channels lie
    on 16 bytes.  The object keeps the tensors and their sizes and strides, nothing of their values."""

    def __init__(self, state, decay):
        _need(state.dim() == 4, "state must be [slots, heads, key_dim, value_dim]", tpl.TPL_E_EXTENT)
        _need(state.dtype == torch.float32 and decay.dtype == torch.float32, "state and decay must be fp32", tpl.TPL_E_DTYPE)
        slots, heads, key_dim, value_dim = state.shape
        _need(tuple(decay.shape) == (heads,), "decay must have one number for each head", tpl.TPL_E_EXTENT)
        _need(state.device == decay.device, "state and decay must be on one device")
        _need(state.stride(3) == 1, "the value channels of a state must be contiguous", tpl.TPL_E_LAYOUT)
        _need(heads < 2 or decay.stride(0) == 1, "decay must be contiguous", tpl.TPL_E_LAYOUT)
        s_slot, s_head, s_key, _ = state.stride()
        _need((slots < 2 or s_slot > 0) and (heads < 2 or s_head > 0) and (key_dim < 2 or s_key >= value_dim),
              "states must not lie over one another", tpl.TPL_E_LAYOUT)
        self.state, self.decay, self.device = state, decay, state.device
        self.heads, self.key_dim, self.value_dim = heads, key_dim, value_dim
        self._c = Pool(state.data_ptr(), decay.data_ptr(), s_slot, s_head, s_key, slots, heads, key_dim, value_dim)
        self._at = ctypes.addressof(self._c)
        self._index = state.get_device()


def attend(q, k, v, pool: StatePool, slots, starts, *, sources=None, scale: Optional[float] = None, out=None,
           stream: Optional[int] = None):
    """Take ``q`` and ``k`` [tokens, key_heads, key_dim] and ``v`` [tokens, heads, value_dim] through the states of ``pool``.

    slots    int32 [batch]: the slot that takes a sequence's state after its tokens; one that is not there takes none.
    starts   int32 [batch + 1]: its rows.
    sources  int32 [batch]: the slot of its state before them (default: ``slots``); one that is not there is a state of zeros.
             A slot that a call writes is written by one sequence and read by no other.
    scale    default key_dim ** -0.5.
    out      takes the result (default: a new tensor); not over q or k.
    stream   the handle of the stream to run on (default: torch's current one).

    Head h reads q and k of head h // (heads / key_heads).  Returns ``out`` [tokens, heads, value_dim]."""
    if _lib is None:
        load()
    if out is None:
        out = kv._result(v, pool, stream)
    index = pool._index
    if index >= 0 and _device() == index:
        status = _attend(pool._at, index, q, k, v, slots, starts, sources, scale, out, _stream(index) if stream is None else int(stream))
        if status == 0:
            return out
        if status > 0:
            _raise(status)
    return _attend_checked(q, k, v, pool, slots, starts, sources, scale, out, stream)


def _attend_checked(q, k, v, pool, slots, starts, sources, scale, out, stream):
    """The same, each argument by itself: says what is wrong, or makes the call, with a workspace where it needs one."""
    device, index, dtype = pool.device, pool._index, q.dtype
    _need(q.dim() == 3, "q must be [tokens, key_heads, key_dim]", tpl.TPL_E_EXTENT)
    _need(dtype in (torch.bfloat16, torch.float16), "q must be bf16 or fp16", tpl.TPL_E_DTYPE)
    tokens, key_heads = q.shape[:2]
    _heads("q", q, dtype, device, (tokens, key_heads, pool.key_dim))
    _heads("k", k, dtype, device, (tokens, key_heads, pool.key_dim))
    _heads("v", v, dtype, device, (tokens, pool.heads, pool.value_dim))
    _heads("out", out, dtype, device, (tokens, pool.heads, pool.value_dim))
    _ints("slots", slots, device, None)
    n = slots.shape[0]
    _ints("starts", starts, device, n + 1)
    if sources is not None:
        _ints("sources", sources, device, n)
    scale = pool.key_dim ** -0.5 if scale is None else scale
    # What the structure can hold; the entry point judges it.
    _need(-_FLOAT_MAX <= scale <= _FLOAT_MAX, "scale must be a finite number")
    batch = _pack_batch(slots.data_ptr(), 0 if sources is None else sources.data_ptr(), starts.data_ptr(), n, tokens)
    args = _pack_new(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), *(x for t in (q, k, v, out) for x in t.stride()[:2]), scale,
                     kv._TYPES[dtype], key_heads)
    size = _calls[1](pool._at, batch, args)
    if size < 0:
        _raise(_calls[0](pool._at, batch, args, None, 0, None))   # refused the same way, before anything is looked at on the device
    _need(index >= 0, "tensors must live on the GPU")
    with torch.cuda.device(index):
        s = _stream(index) if stream is None else int(stream)
        with kv._on(pool, s, stream):   # the workspace is memory of the call's own stream, given back in its order
            ws = torch.empty(size, dtype=torch.uint8, device=device) if size else None
        status = _calls[0](pool._at, batch, args, 0 if ws is None else ws.data_ptr(), size, s)
    if status:
        _raise(status)
    return out
