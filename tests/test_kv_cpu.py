"""The paged key/value cache entry points on the CPU: exports and refusals.

Every refusal is made before anything is launched, so pointers that name no
memory are enough for the C entry points."""

from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

from oracle import kv_oracle
from tensor_layout_amd import kv, tpl
from tensor_layout_amd.tpl import TplError

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_exports():
    with open(os.path.join(ROOT, "include", "tpl_kv.h")) as f:
        names = set(re.findall(r"^\s*(?:int|int64_t)\s+(tpl_kv_\w+)\s*\(", f.read(), re.M))
    assert names == set(kv.EXPORTED)
    lib = kv.load()
    for n in names:
        assert hasattr(lib, n)


def c_cache(**kw):
    d = dict(k=4096, v=8192, k_scale=4096, v_scale=4096, pages=4, k_page=32 * 2 * 64, k_token=128, k_head=64, v_page=32 * 2 * 64,
             v_token=128, v_head=64, ks_page=4, ks_head=2, ks_block=1, vs_page=4, vs_head=2, vs_block=1, type=kv.E4M3, page=32,
             block=16, kv_heads=2, dim=64)
    d.update(kw)
    return kv.Cache(**d)


def c_batch(**kw):
    d = dict(table=4096, starts=4096, lengths=4096, table_row=4, batch=2, width=4, tokens=2)
    d.update(kw)
    return kv.Batch(**d)


def c_query(**kw):
    d = dict(q=4096, out=8192, lse=None, q_token=256, q_head=64, o_token=256, o_head=64, scale=0.125, type=kv.BF16, heads=4)
    d.update(kw)
    return kv.Query(**d)


def c_new(**kw):
    d = dict(k=4096, v=4096, q=4096, q_out=4096, inv_freq=4096, k_token=128, k_head=64, v_token=128, v_head=64, q_token=256,
             q_head=64, o_token=256, o_head=64, type=kv.BF16, heads=4, rot=64, axes=1)
    sections = d.pop("sections", kw.pop("sections", ()))
    d.update(kw)
    n = kv.New(**d)
    for i, x in enumerate(sections):
        n.sections[i] = x
    return n


BAD_CACHES = [dict(type=3), dict(type=-1), dict(k=None), dict(v=None), dict(pages=0), dict(pages=1 << 31), dict(dim=0), dict(dim=72),
              dict(dim=272), dict(kv_heads=0), dict(page=0), dict(page=24), dict(k_scale=None), dict(v_scale=None), dict(block=0),
              dict(block=8), dict(block=64), dict(k=4097), dict(v=4104), dict(k_token=120), dict(k_head=8), dict(v_page=4100)]
BAD_BATCHES = [dict(batch=-1), dict(tokens=-1), dict(width=-1), dict(width=1 << 26), dict(table=None), dict(starts=None),
               dict(lengths=None), dict(batch=1 << 21), dict(tokens=1 << 29)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_caches_that_both_refuse(bad):
    lib, c, b = kv.load(), c_cache(**bad), c_batch()
    assert lib.tpl_kv_append(c, b, c_new(), None) == tpl.TPL_E_ARG
    assert tpl.tpl_last_error()
    assert lib.tpl_kv_attend(c, b, c_query(), 4096, 1 << 40, None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend_workspace(c, b, c_query()) == -1


@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_batches_that_both_refuse(bad):
    lib, c, b = kv.load(), c_cache(), c_batch(**bad)
    assert lib.tpl_kv_append(c, b, c_new(), None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend(c, b, c_query(), 4096, 1 << 40, None) == tpl.TPL_E_ARG


@pytest.mark.parametrize("bad,status", [
    (dict(type=kv.E4M3), tpl.TPL_E_DTYPE), (dict(type=9), tpl.TPL_E_DTYPE), (dict(heads=0), tpl.TPL_E_ARG),
    (dict(heads=5), tpl.TPL_E_ARG), (dict(scale=0.0), tpl.TPL_E_ARG), (dict(scale=-1.0), tpl.TPL_E_ARG),
    (dict(scale=float("nan")), tpl.TPL_E_ARG), (dict(scale=float("inf")), tpl.TPL_E_ARG), (dict(window=-1), tpl.TPL_E_ARG),
    (dict(sinks=-1), tpl.TPL_E_ARG), (dict(q=None), tpl.TPL_E_ARG), (dict(out=None), tpl.TPL_E_ARG),
    (dict(q=4098), tpl.TPL_E_LAYOUT), (dict(o_token=252), tpl.TPL_E_LAYOUT), (dict(q_head=4), tpl.TPL_E_LAYOUT)])
def test_queries_that_are_refused(bad, status):
    lib = kv.load()
    assert lib.tpl_kv_attend(c_cache(), c_batch(), c_query(**bad), 4096, 1 << 40, None) == status
    assert tpl.tpl_last_error()


def test_workspace():
    lib, c, b, q = kv.load(), c_cache(), c_batch(), c_query()
    size = lib.tpl_kv_attend_workspace(c, b, q)
    assert size > 0
    assert lib.tpl_kv_attend(c, b, q, None, size, None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend(c, b, q, 4100, size, None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend(c, b, q, 4096, size - 1, None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend(None, b, q, 4096, size, None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend(c, None, q, 4096, size, None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend(c, b, None, 4096, size, None) == tpl.TPL_E_ARG


@pytest.mark.parametrize("bad,status", [
    (dict(type=kv.E4M3), tpl.TPL_E_DTYPE), (dict(rot=0), tpl.TPL_E_ARG), (dict(rot=3), tpl.TPL_E_ARG), (dict(rot=66), tpl.TPL_E_ARG),
    (dict(axes=0), tpl.TPL_E_ARG), (dict(axes=5), tpl.TPL_E_ARG), (dict(axes=2, sections=(16, 16)), tpl.TPL_E_ARG),
    (dict(axes=2, sections=(16, 15), positions=4096), tpl.TPL_E_ARG), (dict(axes=2, sections=(33, -1), positions=4096), tpl.TPL_E_ARG),
    (dict(heads=0), tpl.TPL_E_ARG), (dict(k=None), tpl.TPL_E_ARG), (dict(v=None), tpl.TPL_E_ARG), (dict(q_out=None), tpl.TPL_E_ARG),
    (dict(k=4098), tpl.TPL_E_LAYOUT), (dict(v_token=100), tpl.TPL_E_LAYOUT), (dict(o_head=4), tpl.TPL_E_LAYOUT)])
def test_new_tokens_that_are_refused(bad, status):
    lib = kv.load()
    assert lib.tpl_kv_append(c_cache(), c_batch(), c_new(**bad), None) == status
    assert tpl.tpl_last_error()


def test_a_16_bit_cache_takes_its_own_type():
    lib = kv.load()
    c = c_cache(type=kv.FP16, k_scale=None, v_scale=None)
    assert lib.tpl_kv_append(c, c_batch(), c_new(), None) == tpl.TPL_E_DTYPE
    assert lib.tpl_kv_attend(c, c_batch(), c_query(), 4096, 1 << 40, None) == tpl.TPL_E_DTYPE


def test_nothing_to_do():
    lib = kv.load()
    for b in (c_batch(tokens=0), c_batch(batch=0, starts=None, lengths=None, table=None)):
        assert lib.tpl_kv_append(c_cache(), b, c_new(), None) == tpl.TPL_OK
        assert lib.tpl_kv_attend_workspace(c_cache(), b, c_query()) == 0
        assert lib.tpl_kv_attend(c_cache(), b, c_query(), None, 0, None) == tpl.TPL_OK


def pools(dtype=torch.bfloat16):
    return [torch.zeros((3, 32, 2, 64)).to(dtype) for _ in range(2)]


def test_the_binding_refuses():
    k, v = pools()
    cache = kv.PagedCache(k, v)
    i32 = dict(dtype=torch.int32)
    t, s, n = torch.zeros((1, 3), **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    q, new = torch.zeros((1, 4, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    f = torch.zeros(32)
    ok = dict(q=q, inv_freq=f)

    def refused(status, call):
        with pytest.raises(TplError) as e:
            call()
        assert e.value.status == status, e.value

    arg, ext, dt, lay = tpl.TPL_E_ARG, tpl.TPL_E_EXTENT, tpl.TPL_E_DTYPE, tpl.TPL_E_LAYOUT
    # On the CPU everything else is right.
    refused(arg, lambda: kv.attend(q, cache, t, s, n))
    refused(arg, lambda: kv.append(cache, new, new, t, s, n, **ok))
    refused(dt, lambda: kv.attend(q, cache, t.long(), s, n))
    refused(ext, lambda: kv.attend(q, cache, t, t[0], n))
    refused(ext, lambda: kv.attend(q[0], cache, t, s, n))
    refused(ext, lambda: kv.attend(q[..., :32], cache, t, s, n))
    refused(dt, lambda: kv.attend(q.float(), cache, t, s, n))
    refused(dt, lambda: kv.attend(q, cache, t, s, n, out=torch.zeros_like(q, dtype=torch.float16)))
    refused(ext, lambda: kv.attend(q, cache, t, s, n, out=q[:, :2]))
    refused(dt, lambda: kv.attend(q, cache, t, s, n, lse=torch.zeros((1, 4), dtype=torch.float64)))
    refused(ext, lambda: kv.attend(q, cache, t, s, n, lse=torch.zeros((1, 3))))
    refused(arg, lambda: kv.attend(q, cache, t, s, n, scale=0.0))
    refused(arg, lambda: kv.attend(q[:, :3], cache, t, s, n))
    refused(lay, lambda: kv.attend(q.transpose(1, 2).contiguous().transpose(1, 2), cache, t, s, n))
    refused(ext, lambda: kv.append(cache, q, q, t, s, n))
    refused(dt, lambda: kv.append(cache, new, new.half(), t, s, n))
    refused(arg, lambda: kv.append(cache, new, new, t, s, n, q_out=q))
    refused(dt, lambda: kv.append(cache, new, new, t, s, n, inv_freq=f.double()))
    refused(arg, lambda: kv.append(cache, new, new, t, s, n, inv_freq=f, sections=(16, 16)))
    refused(arg, lambda: kv.append(cache, new, new, t, s, n, inv_freq=f, sections=(16, 15), positions=torch.zeros((2, 1), **i32)))
    refused(arg, lambda: kv.append(cache, new, new, t, s, n, inv_freq=f, positions=torch.zeros((2, 1), **i32)))
    refused(dt, lambda: kv.append(cache, new, new, t, s, n, inv_freq=f, positions=torch.zeros((1, 1))))
    refused(ext, lambda: kv.append(cache, new, new, t, s, n, inv_freq=f, positions=torch.zeros((1, 2), **i32)))


def test_caches_that_the_binding_refuses():
    k, v = pools()
    sc = torch.ones((3, 2, 2))
    e = pools(torch.float8_e4m3fn)
    for args in ((k, v[:2]), (k, v.half()), (k.float(), v.float()), (k, v, sc, sc), (e[0], e[1]), (e[0], e[1], sc, None),
                 (e[0], e[1], sc.double(), sc), (e[0], e[1], sc[:, :1], sc[:, :1]), (e[0], e[1], sc, sc[..., :1]),
                 (e[0], e[1], torch.ones((3, 2, 3)), torch.ones((3, 2, 3))), (k.transpose(2, 3), v.transpose(2, 3)), (k[0], v[0])):
        with pytest.raises(TplError):
            kv.PagedCache(*args)
    assert kv.PagedCache(e[0], e[1], sc, sc).block == 16


def test_the_statement_itself():
    """One row over two tokens, by hand; a window of one; a block's scale at its border."""
    q = torch.tensor([[[1.0, 0.0]]])
    k = torch.tensor([[[[0.0, 3.0]], [[2.0, 5.0]]]])
    v = torch.tensor([[[[1.0, 10.0]], [[3.0, 20.0]]]])
    out, lse, _, _ = kv_oracle.attend(q, k, v, None, None, [[0]], [0, 1], [2], 0.5)
    e = float(torch.tensor(1.0, dtype=torch.float64).exp())
    assert torch.allclose(out[0, 0], torch.tensor([(1 + 3 * e) / (1 + e), (10 + 20 * e) / (1 + e)], dtype=torch.float64))
    assert abs(float(lse) - float(torch.tensor(1 + e).log())) < 1e-6
    out, lse, _, _ = kv_oracle.attend(q, k, v, None, None, [[0]], [0, 1], [2], 0.5, window=1)
    assert out[0, 0].tolist() == [3.0, 20.0] and float(lse) == 1.0
    assert kv_oracle.block_scale(448.0) == 1.0 and kv_oracle.block_scale(448.1) == 2.0 and kv_oracle.block_scale(0.0) == 2.0 ** -126
