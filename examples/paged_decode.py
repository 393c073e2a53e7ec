"""One attention layer served over a paged key/value cache.

    python examples/paged_decode.py            # 8 prompts of up to 2048 tokens, 32 tokens each

Prompts go through in chunks; then every sequence gets a token at a time, the
step (projections, append, attend) captured once in a HIP graph and replayed
on new lengths.  Weights are random: the point is how the calls fit together.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tensor_layout_amd import kv  # noqa: E402


class Layer:
    """Projections, a cache and the pages of its sequences."""

    def __init__(self, batch, capacity, heads=16, kv_heads=4, dim=64, page=64, block=16, dtype=torch.bfloat16, e4m3=True,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.batch, self.heads, self.kv_heads, self.dim, self.page, self.dtype = batch, heads, kv_heads, dim, page, dtype
        self.hidden = heads * dim

        def weight(n, m):
            return (torch.randn((n, m), generator=g, device="cuda") * n ** -0.5).to(dtype)

        self.w_qkv = weight(self.hidden, (heads + 2 * kv_heads) * dim)
        self.w_out = weight(heads * dim, self.hidden)
        self.inv_freq = (10_000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)).float()
        self.width = -(-capacity // page)
        pages = batch * self.width
        held = torch.float8_e4m3fn if e4m3 else dtype
        pools = [torch.zeros((pages, page, kv_heads, dim), dtype=torch.float32, device="cuda").to(held) for _ in range(2)]
        scales = [torch.ones((pages, kv_heads, page // block), device="cuda") for _ in range(2)] if e4m3 else [None, None]
        self.cache = kv.PagedCache(*pools, *scales)
        # Pages are handed out as sequences grow; -1: not there yet.
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = torch.full((batch, self.width), -1, dtype=torch.int32, device="cuda")
        self.rows = [[] for _ in range(batch)]
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def grow(self, b, length):
        """Pages for `length` tokens of sequence b."""
        while len(self.rows[b]) * self.page < length:
            self.rows[b].append(self.free.pop())
            self.table[b, len(self.rows[b]) - 1] = self.rows[b][-1]

    def step(self, x, starts):
        """x [tokens, hidden] of all sequences, packed; lengths already count them."""
        n = x.shape[0]
        qkv = (x @ self.w_qkv).view(n, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = kv.append(self.cache, k, v, self.table, starts, self.lengths, q=q, inv_freq=self.inv_freq)
        return kv.attend(q, self.cache, self.table, starts, self.lengths).view(n, -1) @ self.w_out

    def prefill(self, prompts, chunk):
        """Each prompt [tokens, hidden] in chunks, all sequences together; every sequence's last output."""
        done, last = [0] * self.batch, [None] * self.batch
        while any(d < p.shape[0] for d, p in zip(done, prompts)):
            parts = [p[d:d + chunk] for d, p in zip(done, prompts)]
            counts = [p.shape[0] for p in parts]
            for b, n in enumerate(counts):
                self.grow(b, done[b] + n)
            starts = torch.tensor([sum(counts[:b]) for b in range(self.batch + 1)], dtype=torch.int32, device="cuda")
            self.lengths += torch.tensor(counts, dtype=torch.int32, device="cuda")
            y = self.step(torch.cat(parts), starts)
            at = 0
            for b, n in enumerate(counts):
                at += n
                done[b] += n
                if n:
                    last[b] = y[at - 1]
        return torch.stack(last)

    def capture(self):
        """A decoding step as a graph: input, output, replay."""
        x = torch.zeros((self.batch, self.hidden), dtype=self.dtype, device="cuda")
        # What the graph reads has to live as long as it does.
        self.starts = torch.arange(self.batch + 1, dtype=torch.int32, device="cuda")
        _ = (x @ self.w_qkv)[:, :self.heads * self.dim] @ self.w_out   # the libraries load what they need before
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.step(x, self.starts)
        return x, y, graph


def run(batch=8, prompt=2048, new=32, chunk=512, graph=True, seed=0, **kw):
    """Last outputs of the prompts and of every decoded token [new + 1, batch, hidden], the layer, and seconds a token."""
    layer = Layer(batch, prompt + new, seed=seed, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    lengths = [max(1, prompt * (b + 2) // (batch + 1)) for b in range(batch)]
    prompts = [torch.randn((n, layer.hidden), generator=g, device="cuda").to(layer.dtype) for n in lengths]
    y = layer.prefill(prompts, chunk)
    outs = [y.clone()]
    lengths = [p.shape[0] for p in prompts]
    starts = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    if graph:
        x_in, y_out, captured = layer.capture()
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(new):
        for b in range(batch):
            lengths[b] += 1
            layer.grow(b, lengths[b])
        layer.lengths += 1
        if graph:
            x_in.copy_(outs[-1])
            captured.replay()
            outs.append(y_out.clone())
        else:
            outs.append(layer.step(outs[-1], starts))
    torch.cuda.synchronize()
    return torch.stack(outs), layer, (time.perf_counter() - began) / max(1, new)


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=2048)
    p.add_argument("--new", type=int, default=32)
    p.add_argument("--chunk", type=int, default=512)
    a = p.parse_args()
    for graph in (False, True):
        outs, layer, s = run(a.batch, a.prompt, a.new, a.chunk, graph=graph)
        print("%s: %.0f us a step, %d sequences, longest %d tokens, outputs' mean square %.4f"
              % ("graph" if graph else "eager", s * 1e6, a.batch, int(layer.lengths.max()), float(outs.float().square().mean())))


if __name__ == "__main__":
    main()
