"""Shared first tokens and reading of a cache, on the CPU: refusals and workspace sizes.

Every refusal is made before anything is launched, so pointers that name no memory are enough for the C entry points."""

from __future__ import annotations

import pytest
import torch

from tensor_layout_amd import kv, tpl
from tensor_layout_amd.tpl import TplError
from tests.test_kv_cpu import BAD_BATCHES, BAD_CACHES, c_batch, c_cache, c_query


def c_rows(**kw):
    d = dict(k=4096, v=8192, k_token=128, k_head=64, v_token=128, v_head=64, type=kv.BF16)
    d.update(kw)
    return kv.Rows(**d)


def c_groups(**kw):
    d = dict(groups=4096, shared=4096, count=1)
    d.update(kw)
    return kv.Groups(**d)


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_caches(bad):
    lib, c, b = kv.load(), c_cache(**bad), c_batch()
    assert lib.tpl_kv_read(c, b, c_rows(), None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend_shared(c, b, c_groups(), c_query(), 4096, 1 << 40, None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend_shared_workspace(c, b, c_groups(), c_query()) == -1


@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_batches(bad):
    lib, c, b = kv.load(), c_cache(), c_batch(**bad)
    assert lib.tpl_kv_read(c, b, c_rows(), None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend_shared(c, b, c_groups(), c_query(), 4096, 1 << 40, None) == tpl.TPL_E_ARG


@pytest.mark.parametrize("bad,status", [
    (dict(type=kv.E4M3), tpl.TPL_E_DTYPE), (dict(heads=5), tpl.TPL_E_ARG), (dict(scale=0.0), tpl.TPL_E_ARG),
    (dict(scale=float("nan")), tpl.TPL_E_ARG), (dict(window=5), tpl.TPL_E_ARG), (dict(sinks=1), tpl.TPL_E_ARG),
    (dict(window=-1), tpl.TPL_E_ARG), (dict(q=None), tpl.TPL_E_ARG), (dict(out=None), tpl.TPL_E_ARG),
    (dict(q=4098), tpl.TPL_E_LAYOUT), (dict(o_token=252), tpl.TPL_E_LAYOUT)])
def test_queries(bad, status):
    lib = kv.load()
    assert lib.tpl_kv_attend_shared(c_cache(), c_batch(), c_groups(), c_query(**bad), 4096, 1 << 40, None) == status
    assert tpl.tpl_last_error()


@pytest.mark.parametrize("bad", [dict(groups=None), dict(shared=None), dict(count=-1), dict(count=1 << 21)])
def test_groups(bad):
    lib = kv.load()
    assert lib.tpl_kv_attend_shared(c_cache(), c_batch(), c_groups(**bad), c_query(), 4096, 1 << 40, None) == tpl.TPL_E_ARG
    assert lib.tpl_kv_attend_shared_workspace(c_cache(), c_batch(), c_groups(**bad), c_query()) == -1
    assert lib.tpl_kv_attend_shared(c_cache(), c_batch(), None, c_query(), 4096, 1 << 40, None) == tpl.TPL_E_ARG


@pytest.mark.parametrize("tokens,count,width,batch", [(2, 1, 4, 2), (2, 1, 1 << 20, 2), (2, 2, 1 << 20, 2), (100, 1, 1 << 20, 2), (900, 1, 1 << 20, 2),
                                                      (3000, 200, 1 << 16, 600), (20_000, 1, 4, 2)])
def test_workspace(tokens, count, width, batch):
    """Room for the results between two launches, or attention's own where there is one."""
    lib, c, b, q, s = kv.load(), c_cache(), c_batch(tokens=tokens, width=width, batch=batch), c_query(), c_groups(count=count)
    size = lib.tpl_kv_attend_shared_workspace(c, b, s, q)
    directly = width == 4 or tokens * 2 >= batch * 128
    if directly:
        assert size == lib.tpl_kv_attend_workspace(c, b, q)
    else:
        assert size >= kv.COUNTERS + tokens * 4 * (64 * 4 + 8)
    if size:
        assert lib.tpl_kv_attend_shared(c, b, s, q, None, size, None) == tpl.TPL_E_ARG
        assert lib.tpl_kv_attend_shared(c, b, s, q, 4100, size, None) == tpl.TPL_E_ARG
        assert lib.tpl_kv_attend_shared(c, b, s, q, 4096, size - 1, None) == tpl.TPL_E_ARG


def test_nothing_to_do():
    lib = kv.load()
    for b in (c_batch(batch=0), c_batch(tokens=0)):
        assert lib.tpl_kv_attend_shared(c_cache(), b, c_groups(), c_query(), None, 0, None) == tpl.TPL_OK
        assert lib.tpl_kv_read(c_cache(), b, c_rows(), None) == tpl.TPL_OK
    # No groups: the call is tpl_kv_attend's, its workspace too.
    s = c_groups(count=0, groups=None, shared=None)
    assert lib.tpl_kv_attend_shared_workspace(c_cache(), c_batch(), s, c_query()) == lib.tpl_kv_attend_workspace(c_cache(), c_batch(), c_query())


@pytest.mark.parametrize("bad,status", [
    (dict(type=kv.E4M3), tpl.TPL_E_DTYPE), (dict(type=9), tpl.TPL_E_DTYPE), (dict(k=None, v=None), tpl.TPL_E_ARG), (dict(v=4096), tpl.TPL_E_ARG),
    (dict(k=4098), tpl.TPL_E_LAYOUT), (dict(v_token=124), tpl.TPL_E_LAYOUT), (dict(k_head=4), tpl.TPL_E_LAYOUT),
    (dict(k_token=0), tpl.TPL_E_LAYOUT), (dict(k_head=0), tpl.TPL_E_LAYOUT), (dict(v_token=64), tpl.TPL_E_LAYOUT), (dict(v_head=56), tpl.TPL_E_LAYOUT)])
def test_rows(bad, status):
    lib = kv.load()
    assert lib.tpl_kv_read(c_cache(), c_batch(), c_rows(**bad), None) == status
    assert tpl.tpl_last_error()


def test_rows_of_a_16_bit_cache_are_its_type():
    lib, c = kv.load(), c_cache(type=kv.FP16, k_page=32 * 2 * 64, v_page=32 * 2 * 64)
    assert lib.tpl_kv_read(c, c_batch(), c_rows(), None) == tpl.TPL_E_DTYPE


def cpu_call():
    pool = torch.zeros((3, 32, 2, 64), dtype=torch.bfloat16)
    return kv.PagedCache(pool, pool.clone()), [torch.tensor(x, dtype=torch.int32) for x in ([[0, 1], [0, 2]], [0, 1, 2], [40, 41])]


def test_python_refusals():
    cache, ints = cpu_call()
    q, rows = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    groups, shared = (torch.tensor(x, dtype=torch.int32) for x in ([0, 2], [32]))

    def refused(call, status, *args, **kw):
        with pytest.raises(TplError) as e:
            call(*args, **kw)
        assert e.value.status == status and str(e.value)
    share = lambda *a, **kw: kv.attend_shared(q, cache, *ints, *a, **kw)   # noqa: E731
    refused(share, tpl.TPL_E_ARG, groups, shared)   # not on a GPU
    refused(share, tpl.TPL_E_DTYPE, groups.long(), shared)
    refused(share, tpl.TPL_E_DTYPE, groups, shared.float())
    refused(share, tpl.TPL_E_EXTENT, groups, torch.zeros(2, dtype=torch.int32))
    refused(share, tpl.TPL_E_EXTENT, torch.zeros(0, dtype=torch.int32), shared)
    refused(share, tpl.TPL_E_EXTENT, groups[None], shared)
    refused(share, tpl.TPL_E_LAYOUT, torch.zeros(4, dtype=torch.int32)[::2], shared)
    refused(share, tpl.TPL_E_ARG, groups, shared, scale=0.0)
    refused(share, tpl.TPL_E_EXTENT, groups, shared, out=torch.zeros((2, 4, 32), dtype=torch.bfloat16))
    refused(share, tpl.TPL_E_DTYPE, groups, shared, lse=torch.zeros((2, 4), dtype=torch.float64))
    read = lambda *a: kv.read(cache, *ints, *a)   # noqa: E731
    refused(read, tpl.TPL_E_ARG, rows, rows.clone())   # not on a GPU
    refused(read, tpl.TPL_E_ARG)
    refused(read, tpl.TPL_E_DTYPE, rows.float())
    refused(read, tpl.TPL_E_DTYPE, rows, rows.half())
    refused(read, tpl.TPL_E_EXTENT, rows[0])
    refused(read, tpl.TPL_E_EXTENT, rows, rows[:1])
    refused(read, tpl.TPL_E_EXTENT, torch.zeros((2, 3, 64), dtype=torch.bfloat16))
    refused(read, tpl.TPL_E_LAYOUT, torch.zeros((2, 2, 128), dtype=torch.bfloat16)[..., ::2])
    refused(kv.read, tpl.TPL_E_DTYPE, cache, ints[0].long(), *ints[1:], rows)
