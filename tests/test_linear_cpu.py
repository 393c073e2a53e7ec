"""Linear attention's entry points on the CPU: exports, refusals and workspace sizes.

Every refusal is made before anything is launched, so pointers that name no memory are enough for the C entry points."""

from __future__ import annotations

import os
import re

import pytest
import torch

from tensor_layout_amd import kv, linear, tpl
from tensor_layout_amd.tpl import TplError

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_exports():
    with open(os.path.join(ROOT, "include", "tpl_linear.h")) as f:
        names = set(re.findall(r"^\s*(?:int|int64_t)\s+(tpl_linear_\w+)\s*\(", f.read(), re.M))
    assert names == set(linear.EXPORTED)
    lib = linear.load()
    for n in names:
        assert hasattr(lib, n)


def c_pool(**kw):
    d = dict(state=4096, decay=4096, s_slot=2 * 64 * 64, s_head=64 * 64, s_key=64, slots=4, heads=2, key_dim=64, value_dim=64)
    d.update(kw)
    return linear.Pool(**d)


def c_batch(**kw):
    d = dict(slots=4096, sources=4096, starts=4096, batch=2, tokens=40)
    d.update(kw)
    return linear.Batch(**d)


def c_new(**kw):
    d = dict(q=4096, k=4096, v=4096, out=8192, q_token=128, q_head=64, k_token=128, k_head=64, v_token=128, v_head=64, o_token=128,
             o_head=64, scale=0.125, type=kv.BF16, key_heads=2)
    d.update(kw)
    return linear.New(**d)


def call(c, b, n, ws=4096, size=1 << 40):
    return linear.load().tpl_linear_attend(c, b, n, ws, size, None)


@pytest.mark.parametrize("bad", [dict(state=None), dict(decay=None), dict(state=4104), dict(s_slot=2), dict(s_head=6), dict(s_key=63), dict(slots=0),
                                 dict(slots=1 << 31), dict(heads=0), dict(heads=70_000), dict(key_dim=0), dict(key_dim=24), dict(key_dim=272),
                                 dict(value_dim=8), dict(value_dim=272), dict(s_slot=1 << 41)])
def test_pools(bad):
    assert call(c_pool(**bad), c_batch(), c_new()) == tpl.TPL_E_ARG
    assert tpl.tpl_last_error()
    assert linear.load().tpl_linear_attend_workspace(c_pool(**bad), c_batch(), c_new()) == -1


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(tokens=-1), dict(slots=None), dict(starts=None), dict(batch=1 << 21), dict(tokens=1 << 29)])
def test_batches(bad):
    assert call(c_pool(), c_batch(**bad), c_new()) == tpl.TPL_E_ARG


@pytest.mark.parametrize("bad,status", [
    (dict(type=kv.E4M3), tpl.TPL_E_DTYPE), (dict(type=7), tpl.TPL_E_DTYPE), (dict(key_heads=0), tpl.TPL_E_ARG), (dict(key_heads=3), tpl.TPL_E_ARG),
    (dict(key_heads=4), tpl.TPL_E_ARG), (dict(scale=float("nan")), tpl.TPL_E_ARG), (dict(scale=float("inf")), tpl.TPL_E_ARG),
    (dict(scale=float("-inf")), tpl.TPL_E_ARG), (dict(q=None), tpl.TPL_E_ARG), (dict(k=None), tpl.TPL_E_ARG), (dict(v=None), tpl.TPL_E_ARG),
    (dict(out=None), tpl.TPL_E_ARG), (dict(q=4098), tpl.TPL_E_LAYOUT), (dict(k_token=124), tpl.TPL_E_LAYOUT), (dict(v_head=4), tpl.TPL_E_LAYOUT),
    (dict(out=4104), tpl.TPL_E_LAYOUT)])
def test_rows(bad, status):
    assert call(c_pool(), c_batch(), c_new(**bad)) == status
    assert tpl.tpl_last_error()


def test_workspace():
    lib = linear.load()
    size = lib.tpl_linear_attend_workspace(c_pool(), c_batch(batch=1, tokens=5000), c_new())
    assert size > 0 and size % (2 * 64 * 64 * 4) == 0
    for ws, n in ((None, size), (4100, size), (4096, size - 1)):
        assert call(c_pool(), c_batch(batch=1, tokens=5000), c_new(), ws, n) == tpl.TPL_E_ARG
    for b in (c_batch(tokens=2), c_batch(batch=600, tokens=5000), c_batch(batch=1, tokens=16)):
        assert lib.tpl_linear_attend_workspace(c_pool(), b, c_new()) == 0
    assert call(None, c_batch(), c_new()) == call(c_pool(), None, c_new()) == call(c_pool(), c_batch(), None) == tpl.TPL_E_ARG


def test_nothing_to_do():
    assert call(c_pool(), c_batch(batch=0, slots=None, starts=None), c_new(), None, 0) == tpl.TPL_OK
    assert call(c_pool(), c_batch(tokens=0), c_new(q=None, k=None, v=None, out=None), None, 0) == tpl.TPL_OK


def test_python_refusals():
    state, decay = torch.zeros((3, 2, 64, 32)), torch.zeros(2)

    def refused(f, status, *args, **kw):
        with pytest.raises(TplError) as e:
            f(*args, **kw)
        assert e.value.status == status and str(e.value)
    for s, d, status in ((state[0], decay, tpl.TPL_E_EXTENT), (state.double(), decay, tpl.TPL_E_DTYPE), (state, decay.half(), tpl.TPL_E_DTYPE),
                         (state, decay[:1], tpl.TPL_E_EXTENT), (state.transpose(2, 3), decay, tpl.TPL_E_LAYOUT),
                         (state, torch.zeros(4)[::2], tpl.TPL_E_LAYOUT), (state[:1].expand(3, 2, 64, 32), decay, tpl.TPL_E_LAYOUT),
                         (state[:, :, :1].expand(3, 2, 64, 32), decay, tpl.TPL_E_LAYOUT), (state[:, :1].expand(3, 2, 64, 32), decay, tpl.TPL_E_LAYOUT)):
        refused(linear.StatePool, status, s, d)
    pool = linear.StatePool(state, decay)
    q, v = torch.zeros((5, 2, 64), dtype=torch.bfloat16), torch.zeros((5, 2, 32), dtype=torch.bfloat16)
    slots, starts = (torch.tensor(x, dtype=torch.int32) for x in ([0, 1], [0, 2, 5]))

    def run(status, q=q, k=q, v=v, slots=slots, starts=starts, **kw):
        refused(linear.attend, status, q, k, v, pool, slots, starts, **kw)
    run(tpl.TPL_E_ARG)   # not on a GPU
    run(tpl.TPL_E_EXTENT, q=q[0])
    run(tpl.TPL_E_DTYPE, q=q.float())
    run(tpl.TPL_E_DTYPE, k=q.half())
    run(tpl.TPL_E_DTYPE, v=v.half(), out=v)
    run(tpl.TPL_E_EXTENT, k=q[:4])
    run(tpl.TPL_E_EXTENT, k=q[:, :1])
    run(tpl.TPL_E_EXTENT, v=v[:, :1], out=v)
    run(tpl.TPL_E_EXTENT, out=q)
    run(tpl.TPL_E_LAYOUT, q=torch.zeros((5, 2, 128), dtype=torch.bfloat16)[..., ::2])
    run(tpl.TPL_E_DTYPE, slots=slots.long())
    run(tpl.TPL_E_EXTENT, starts=starts[:2])
    run(tpl.TPL_E_EXTENT, slots=slots[None])
    run(tpl.TPL_E_LAYOUT, slots=torch.zeros(4, dtype=torch.int32)[::2])
    run(tpl.TPL_E_EXTENT, sources=slots[:1])
    run(tpl.TPL_E_DTYPE, sources=slots.float())
    run(tpl.TPL_E_ARG, scale=float("inf"))
    run(tpl.TPL_E_ARG, scale=float("nan"))
    odd = torch.zeros((5, 3, 64), dtype=torch.bfloat16)
    run(tpl.TPL_E_ARG, q=odd, k=odd)   # 2 heads, 3 of keys
