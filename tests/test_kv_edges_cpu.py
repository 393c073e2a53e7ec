"""The paged key/value cache entry points on the CPU: what calls owe each other, and refusals at the limits."""

from __future__ import annotations

import pytest
import torch

from tensor_layout_amd import kv, tpl
from tensor_layout_amd.tpl import TplError
from tests.test_kv_cpu import c_batch, c_cache, c_query, pools


def test_a_split_prompts_parts_lie_behind_the_counters():
    """One sequence of 100 tokens on many: parts of 128 rows of 64 sums, a reference and a sum of weights, after the counters."""
    size = kv.load().tpl_kv_attend_workspace(c_cache(), c_batch(batch=1, tokens=100, width=940), c_query())
    part = 128 * (64 + 2) * 4
    assert size > kv.COUNTERS and (size - kv.COUNTERS) % part == 0


def test_attend_says_what_the_entry_point_says():
    """A refusal's status is the entry point's, not one for all."""
    cache = kv.PagedCache(*pools())
    i32 = dict(dtype=torch.int32)
    t, s, n = torch.zeros((1, 3), **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    q = torch.zeros((1, 4, 64), dtype=torch.float16)
    for status, kw in ((tpl.TPL_E_DTYPE, {}), (tpl.TPL_E_DTYPE, dict(window=-1)), (tpl.TPL_E_ARG, dict(q=q[:, :3].to(torch.bfloat16)))):
        with pytest.raises(TplError) as e:
            kv.attend(kw.pop("q", q), cache, t, s, n, **kw)
        assert e.value.status == status, e.value


def test_numbers_that_no_structure_holds_are_refused():
    """Out of the entry points' ranges, they are a refused call like any other."""
    cache = kv.PagedCache(*pools())
    i32 = dict(dtype=torch.int32)
    t, s, n = torch.zeros((1, 3), **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    for kw in (dict(window=1 << 40), dict(window=-(1 << 40)), dict(window=16, sinks=1 << 31), dict(scale=1e300), dict(scale=-1e300),
               dict(scale=float("inf")), dict(scale=1e-300)):
        with pytest.raises(TplError) as e:
            kv.attend(q, cache, t, s, n, **kw)
        assert e.value.status == tpl.TPL_E_ARG
