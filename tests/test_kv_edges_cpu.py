"""The paged key/value cache entry points on the CPU: what calls owe each other, and refusals at the limits."""

from __future__ import annotations

from tensor_layout_amd import kv
from tests.test_kv_cpu import c_batch, c_cache, c_query


def test_a_split_prompts_parts_lie_behind_the_counters():
    """One sequence of 100 tokens on many: parts of 128 rows of 64 sums, a reference and a sum of weights, after the counters."""
    size = kv.load().tpl_kv_attend_workspace(c_cache(), c_batch(batch=1, tokens=100, width=940), c_query())
    part = 128 * (64 + 2) * 4
    assert size > kv.COUNTERS and (size - kv.COUNTERS) % part == 0
