"""The example of many answers to one prompt: reading, appending, shared attention and linear attention together."""

from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from oracle import kv_oracle, linear_oracle
from tests.test_gpu_kv import compare_attend

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("shared_prompt", os.path.join(ROOT, "examples", "shared_prompt.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompt", [200, 192])
def test_graph_and_eager_steps_agree(prompt):
    """The same kernels on the same inputs, in the same order: the same bits."""
    m = example()
    kw = dict(answers=5, prompt=prompt, new=4, heads=8, kv_heads=2)
    eager, a, _ = m.run(graph=False, **kw)
    graph, b, _ = m.run(graph=True, **kw)
    assert bool(eager.isfinite().all()) and torch.equal(eager, graph)
    assert torch.equal(a.cache.k.view(torch.uint8), b.cache.k.view(torch.uint8)) and torch.equal(a.pool.state, b.pool.state)


def test_a_step_is_what_the_statements_say():
    """The next step's attention and states, from what the cache and the pool hold after some."""
    from tensor_layout_amd import kv, linear
    m = example()
    _, layers, _ = m.run(answers=3, prompt=150, new=2, heads=4, kv_heads=2)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((3, 4, 64), generator=g).to(torch.bfloat16)
    c, lengths = layers.cache, layers.lengths
    assert lengths.tolist() == [152] * 3
    lse = torch.empty((3, 4), device="cuda")
    got = kv.attend_shared(q.cuda(), c, layers.table, layers.starts, lengths, layers.groups, layers.shared, lse=lse)
    pools = [x.cpu() for x in (c.k, c.v, c.k_scale, c.v_scale)]
    want = kv_oracle.attend(q, *pools, layers.table.tolist(), [0, 1, 2, 3], [152] * 3, 0.125, groups=[0, 3], shared=[150])
    compare_attend(got.cpu(), lse.cpu(), *want, pools[1], pools[3], torch.bfloat16, True, 64, 152)
    # An answer's own copy of the prompt's last tokens holds the same: alone, each sees what it sees with its group.
    alone = kv_oracle.attend(q, *pools, layers.table.tolist(), [0, 1, 2, 3], [152] * 3, 0.125)
    assert torch.equal(alone[0], want[0])
    k, v = (torch.randn((3, 4, 64), generator=g).to(torch.bfloat16) for _ in range(2))
    state, decay = layers.pool.state.cpu(), layers.pool.decay.cpu()
    out = linear.attend(q.cuda(), k.cuda(), v.cuda(), layers.pool, layers.slots, layers.starts)
    w = linear_oracle.attend(q, k, v, state, decay, [1, 2, 3], [0, 1, 2, 3], None, 0.125)
    # One token: two products and a sum a number in 32 bits, 64 of them an output, rounded to bf16.
    assert bool(((out.cpu().double() - w[0]).abs() <= 72 * 2.0 ** -24 * w[2] + 2.0 ** -8 * w[0].abs()).all())
    assert bool(((layers.pool.state.cpu().double() - w[1]).abs() <= 2.0 ** -21 * w[3]).all())
