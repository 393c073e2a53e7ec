"""The serving example: append and attend together, in chunks, eagerly and in a graph."""

from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from oracle import kv_oracle

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("paged_decode", os.path.join(ROOT, "examples", "paged_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("e4m3", [True, False])
def test_graph_and_eager_steps_agree(e4m3):
    """The same kernels on the same inputs, in the same order: the same bits."""
    m = example()
    kw = dict(batch=3, prompt=150, new=5, chunk=40, e4m3=e4m3, heads=8, kv_heads=2)
    eager, a, _ = m.run(graph=False, **kw)
    graph, b, _ = m.run(graph=True, **kw)
    assert torch.equal(a.lengths, b.lengths) and torch.equal(a.table, b.table)
    assert torch.equal(a.cache.k.view(torch.uint8), b.cache.k.view(torch.uint8))
    assert torch.equal(eager, graph)


def test_chunks_hold_what_the_whole_prompt_holds():
    """A 16-bit cache holds the same however the prompt is cut (up to the projections' own rounding)."""
    m = example()
    kw = dict(batch=2, prompt=130, new=0, e4m3=False, heads=4, kv_heads=2)
    _, a, _ = m.run(chunk=130, **kw)
    _, b, _ = m.run(chunk=33, **kw)
    for x, y in ((a.cache.k, b.cache.k), (a.cache.v, b.cache.v)):
        table = a.table.tolist()
        for row_a, row_b, n in zip(table, b.table.tolist(), a.lengths.tolist()):
            for j in range(n):
                u, w = x[row_a[j // a.page], j % a.page].float(), y[row_b[j // b.page], j % b.page].float()
                # Products of other shapes may sum in another order: each of a pair a rounding apart at most (2^-7 of
                # it), which the rotation adds up, and one rounding of the result more.
                assert bool(((u - w).abs() <= 3 * 2.0 ** -7 * u.abs().amax(-1, keepdim=True)).all())


def test_a_step_is_what_the_statement_says():
    m = example()
    _, layer, _ = m.run(batch=2, prompt=70, new=0, chunk=25, heads=4, kv_heads=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn((2, 4, 64), generator=g, device="cuda").to(torch.bfloat16)
    starts = torch.arange(3, dtype=torch.int32, device="cuda")
    from tensor_layout_amd import kv
    got = kv.attend(q, layer.cache, layer.table, starts, layer.lengths).cpu().double()
    c = layer.cache
    out, _, size, score = kv_oracle.attend(q.cpu(), c.k.cpu(), c.v.cpu(), c.k_scale.cpu(), c.v_scale.cpu(), layer.table.tolist(),
                                           [0, 1, 2], layer.lengths.tolist(), 0.125)
    # Weights and output are rounded to bf16, scores summed in 32 bits.
    err = 2 * torch.expm1(72 * 2.0 ** -24 * score)[..., None] + 2.0 ** -8 + 2.0 ** -19
    assert bool(((got - out).abs() <= err * size + 2.0 ** -8 * out.abs()).all())
