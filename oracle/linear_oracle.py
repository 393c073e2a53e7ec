"""Plain statement in 64 bits, on the CPU, of linear attention with a decay for each head: the recurrence, token by token.

Takes torch CPU tensors and plain lists, shares no code with the library."""

from __future__ import annotations

import torch


def attend(q, k, v, state, decay, slots, starts, sources=None, scale=1.0, fill=0.0):
    """(out, state, size, states): the outputs and the pool afterwards, the sums of magnitudes behind each output, and behind
    each number of the pool.  Rows of no sequence keep `fill`."""
    tokens, heads, value_dim = v.shape
    share = heads // q.shape[1]
    q, k = (x.double().repeat_interleave(share, 1) for x in (q, k))
    v, old = v.double(), state.double()
    out = torch.full(v.shape, fill, dtype=torch.float64)
    size = torch.zeros_like(out)
    new, sizes = old.clone(), old.abs()
    keep = torch.exp(decay.double().clamp(max=0.0))[:, None, None]
    for b, to in enumerate(slots):
        r, e = starts[b], starts[b + 1]
        if not 0 <= r < e <= tokens:
            continue
        at = to if sources is None else sources[b]
        s = old[at].clone() if 0 <= at < len(old) else torch.zeros_like(old[0])
        a = s.abs()
        for t in range(r, e):
            s = s * keep + k[t][:, :, None] * v[t][:, None]
            a = a * keep + (k[t][:, :, None] * v[t][:, None]).abs()
            out[t] = scale * (q[t][:, :, None] * s).sum(1)
            size[t] = abs(scale) * (q[t].abs()[:, :, None] * a).sum(1)
        if 0 <= to < len(old):
            new[to], sizes[to] = s, a
    return out, new, size, sizes
