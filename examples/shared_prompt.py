"""Many answers to one prompt, through a layer of attention and one of linear attention.

    python examples/shared_prompt.py           # 16 answers of 32 tokens to a prompt of 3001

The prompt goes through once.  Then every answer gets a row of the page table
that names the prompt's whole pages, a copy of its last, partly filled one
(read, append), and a slot of its own for the linear layer's state, which its
first step reads from the prompt's slot.  A step (projections, append,
attention to the shared tokens and the answer's own, linear attention) is
captured once in a HIP graph and replayed.  Weights are random: the point is
how the calls fit together.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tensor_layout_amd import kv, linear  # noqa: E402


class Layers:
    """Projections, a paged cache and a pool of states for a prompt and its answers."""

    def __init__(self, answers, capacity, heads=16, kv_heads=4, dim=64, page=64, block=16, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.answers, self.heads, self.kv_heads, self.dim, self.page = answers, heads, kv_heads, dim, page
        self.hidden = heads * dim

        def weight(n, m):
            return (torch.randn((n, m), generator=g, device="cuda") * n ** -0.5).to(dtype)

        self.w_qkv, self.w_out = weight(self.hidden, (heads + 2 * kv_heads) * dim), weight(self.hidden, self.hidden)
        self.w_linear, self.w_back = weight(self.hidden, 3 * self.hidden), weight(self.hidden, self.hidden)
        self.inv_freq = (10_000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)).float()
        self.width = -(-capacity // page)
        pages = (answers + 1) * self.width
        pools = [torch.zeros((pages, page, kv_heads, dim), device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.ones((pages, kv_heads, page // block), device="cuda") for _ in range(2)]
        self.cache = kv.PagedCache(*pools, *scales)
        decay = -torch.exp2(-8.0 * torch.arange(1, heads + 1, device="cuda", dtype=torch.float32) / heads)
        # Slot 0: the prompt's; the others: an answer each.
        self.pool = linear.StatePool(torch.zeros((answers + 1, heads, dim, dim), device="cuda"), decay)
        self.rows = [list(range(self.width))]   # row 0: the prompt's pages

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def prefill(self, x):
        """The prompt [tokens, hidden], once; its last output."""
        n = x.shape[0]
        self.prompt = n
        table, starts, lengths = self.ints(self.rows), self.ints([0, n]), self.ints([n])
        q, k, v = self.project(x)
        q = kv.append(self.cache, k, v, table, starts, lengths, q=q, inv_freq=self.inv_freq)
        y = kv.attend(q, self.cache, table, starts, lengths).view(n, -1) @ self.w_out + x
        a, b, c = (y @ self.w_linear).view(n, 3, self.heads, self.dim).unbind(1)
        z = linear.attend(a, b, c, self.pool, self.ints([0]), starts, sources=self.ints([-1]))
        return (z.view(n, -1) @ self.w_back + y)[-1]

    def fork(self):
        """A row, a copy of the last page's tokens and a slot for every answer."""
        whole, rest = divmod(self.prompt, self.page)
        free = iter(range(self.width, (self.answers + 1) * self.width))
        own = [[next(free) for _ in range(self.width - whole)] for _ in range(self.answers)]
        self.table = self.ints([self.rows[0][:whole] + pages for pages in own])
        if rest:
            part = [torch.empty((rest, self.kv_heads, self.dim), dtype=self.w_out.dtype, device="cuda") for _ in range(2)]
            kv.read(self.cache, self.ints(self.rows), self.ints([0, rest]), self.ints([self.prompt]), *part)
            copies = [p.expand(self.answers, *p.shape).reshape(-1, *p.shape[1:]) for p in part]
            kv.append(self.cache, *copies, self.table, self.ints([rest * i for i in range(self.answers + 1)]),
                      self.ints([self.prompt] * self.answers))
        # The row of a group's first sequence names the shared tokens; all of them, whole pages or not.
        self.groups, self.shared = self.ints([0, self.answers]), self.ints([self.prompt])
        self.starts = self.ints(list(range(self.answers + 1)))
        self.lengths = self.ints([self.prompt] * self.answers)
        self.slots = self.ints(list(range(1, self.answers + 1)))
        self.sources = self.ints([0] * self.answers)   # the first step reads the prompt's state

    def project(self, x):
        qkv = (x @ self.w_qkv).view(x.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        return qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)

    def step(self, x):
        """A token [answers, hidden] of every answer; lengths already count it."""
        q, k, v = self.project(x)
        batch = (self.table, self.starts, self.lengths)
        q = kv.append(self.cache, k, v, *batch, q=q, inv_freq=self.inv_freq)
        y = kv.attend_shared(q, self.cache, *batch, self.groups, self.shared).view(x.shape[0], -1) @ self.w_out + x
        a, b, c = (y @ self.w_linear).view(x.shape[0], 3, self.heads, self.dim).unbind(1)
        z = linear.attend(a, b, c, self.pool, self.slots, self.starts, sources=self.sources)
        return z.view(x.shape[0], -1) @ self.w_back + y

    def capture(self):
        x = torch.zeros((self.answers, self.hidden), dtype=self.w_out.dtype, device="cuda")
        _ = ((x @ self.w_qkv)[:, :self.hidden] @ self.w_out @ self.w_linear)[:, :self.hidden] @ self.w_back   # the libraries load what they need before
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.step(x)
        return x, y, graph


def run(answers=16, prompt=3001, new=32, graph=True, seed=0, **kw):
    """Every step's outputs [new + 1, answers, hidden], the layers, and seconds a step."""
    layers = Layers(answers, prompt + new, seed=seed, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    last = layers.prefill(torch.randn((prompt, layers.hidden), generator=g, device="cuda").to(layers.w_out.dtype))
    layers.fork()
    # Every answer begins in its own way.
    outs = [(last + torch.randn((answers, layers.hidden), generator=g, device="cuda")).to(last.dtype)]
    if graph:
        x_in, y_out, captured = layers.capture()
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(new):
        layers.lengths += 1
        x = torch.nn.functional.normalize(outs[-1].float(), dim=-1).mul_(layers.hidden ** 0.5).to(last.dtype)
        if graph:
            x_in.copy_(x)
            captured.replay()
            outs.append(y_out.clone())
        else:
            outs.append(layers.step(x))
        layers.sources.copy_(layers.slots)
    torch.cuda.synchronize()
    return torch.stack(outs), layers, (time.perf_counter() - began) / max(1, new)


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--answers", type=int, default=16)
    p.add_argument("--prompt", type=int, default=3001)
    p.add_argument("--new", type=int, default=32)
    a = p.parse_args()
    for graph in (False, True):
        outs, layers, s = run(a.answers, a.prompt, a.new, graph=graph)
        print("%s: %.0f us a step, %d answers to a prompt of %d tokens, outputs' mean square %.4f"
              % ("graph" if graph else "eager", s * 1e6, a.answers, a.prompt, float(outs.float().square().mean())))


if __name__ == "__main__":
    main()
