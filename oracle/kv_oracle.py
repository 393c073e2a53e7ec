"""Plain statement in 64 bits, on the CPU, of the paged key/value cache operators.

Loops over sequences, tokens and blocks; takes torch CPU tensors and plain
lists, shares no code with the library."""

from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn


def values(pool, scale):
    """A pool's values in 64 bits: [pages, page, kv_heads, dim]."""
    x = pool.to(torch.float32).double()
    if scale is None:
        return x
    block = pool.shape[1] // scale.shape[2]
    return x * scale.double().repeat_interleave(block, 2).transpose(1, 2)[..., None]


def ordered(starts, lengths, tokens, b):
    """(first row, new tokens, length) of a sequence; no new tokens where the arrays are out of order."""
    r, e, n = starts[b], starts[b + 1], lengths[b]
    return (r, e - r, n) if 0 <= r < e <= tokens and e - r <= n <= 1 << 30 else (0, 0, 0)


def attend(q, k_pool, v_pool, k_scale, v_scale, table, starts, lengths, scale, window=0, sinks=0, fill=None):
    """(out, lse, size, score): size is each output's sum of |weight * value|, score each row's largest sum of
    |scale * q * k| over what it sees.  Rows of no sequence keep `fill`."""
    tokens, heads, dim = q.shape
    k_all, v_all = values(k_pool, k_scale), values(v_pool, v_scale)
    page, kv_heads = k_pool.shape[1], k_pool.shape[2]
    group = heads // kv_heads
    nan = float("nan") if fill is None else fill
    out = torch.full(q.shape, nan, dtype=torch.float64)
    lse = torch.full((tokens, heads), nan, dtype=torch.float64)
    size, score = torch.zeros_like(out), torch.zeros_like(lse)
    qd = q.double()
    for b in range(len(lengths)):
        r0, n, length = ordered(starts, lengths, tokens, b)
        there = [j for j in range(min(length, len(table[b]) * page)) if 0 <= table[b][j // page] < k_pool.shape[0]]
        js = torch.tensor(there, dtype=torch.long)
        pg = torch.tensor([table[b][j // page] for j in there], dtype=torch.long)
        for i in range(n):
            pos = length - n + i
            see = js <= pos
            if window:
                see &= (pos - js < window) | (js < sinks)
            if not bool(see.any()):
                out[r0 + i], lse[r0 + i] = 0.0, -math.inf
                continue
            w, s = pg[see], js[see] % page
            for h in range(kv_heads):
                hs = slice(h * group, (h + 1) * group)
                k, v = k_all[w, s, h], v_all[w, s, h]
                x = qd[r0 + i, hs] @ k.t() * scale
                top = x.amax(-1, keepdim=True)
                p = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
                total = p.sum(-1, keepdim=True)
                pn = p / total.masked_fill(total == 0, 1.0)
                out[r0 + i, hs] = pn @ v
                lse[r0 + i, hs] = (top + total.log()).squeeze(-1)
                size[r0 + i, hs] = pn @ v.abs()
                score[r0 + i, hs] = (qd[r0 + i, hs].abs() @ k.abs().t() * scale).amax(-1)
    return out, lse, size, score


def rotated(x, place, inv_freq, sections, interleaved):
    """[tokens, heads, dim] in 64 bits, turned; place: [axes][tokens] positions."""
    y = x.double().clone()
    pairs = len(inv_freq)
    for c in range(pairs):
        axis, end = 0, 0
        if sections:
            for axis, n in enumerate(sections):
                end += n
                if c < end:
                    break
        i, j = (2 * c, 2 * c + 1) if interleaved else (c, c + pairs)
        a = torch.tensor([float(t) * float(inv_freq[c]) for t in place[axis]], dtype=torch.float64)[:, None]
        u, w = x[..., i].double(), x[..., j].double()
        y[..., i], y[..., j] = u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()
    return y


def block_scale(amax):
    """The least power of two, of 2^-126 at least, with amax <= 448 of it."""
    s = 2.0 ** -126
    while amax > 448.0 * s:
        s *= 2.0
    return s


def append(q, k, v, k_pool, v_pool, k_scale, v_scale, table, starts, lengths, inv_freq=None, positions=None,
           sections=None, interleaved=False):
    """q rotated and the pools and scales afterwards, in 64 bits; an e4m3 pool as value over scale before its
    rounding.  Also a mask of the pool's tokens that are written."""
    tokens = k.shape[0]
    place = positions
    if place is None:
        place = [[0] * tokens]
        for b in range(len(lengths)):
            r0, n, length = ordered(starts, lengths, tokens, b)
            for i in range(n):
                place[0][r0 + i] = length - n + i
    f = [] if inv_freq is None else inv_freq.tolist()
    qr = None if q is None else rotated(q, place, f, sections, interleaved)
    res = [qr]
    page = k_pool.shape[1]
    touched = torch.zeros(k_pool.shape[:2], dtype=torch.bool)
    for x, pool, scale in ((rotated(k, place, f, sections, interleaved), k_pool, k_scale),
                           (v.double(), v_pool, v_scale)):
        new = pool.to(torch.float32).double()
        sc = None if scale is None else scale.double().clone()
        block = page if scale is None else page // scale.shape[2]
        for b in range(len(lengths)):
            r0, n, length = ordered(starts, lengths, tokens, b)
            at = length - n
            while at < length:
                end = min(length, (at // block + 1) * block)
                pg = table[b][at // page] if at // page < len(table[b]) else -1
                if 0 <= pg < k_pool.shape[0]:
                    j, had, rows = at % page, at % block, slice(r0 + at - (length - n), r0 + end - (length - n))
                    part = x[rows]
                    if scale is not None:
                        fine = torch.where(part.isfinite(), part.abs(), 0.0)
                        for h in range(k_pool.shape[2]):
                            s = block_scale(float(fine[:, h].max()))
                            old = float(sc[pg, h, j // block])
                            if had:
                                s = max(s, old)
                                new[pg, j - had:j, h] *= old / s
                            sc[pg, h, j // block] = s
                        part = part / sc[pg, :, j // block][:, None]
                    new[pg, j:j + end - at] = part
                    touched[pg, (j - had if scale is not None else j):j + end - at] = True
                at = end
        res += [new, sc]
    return (*res, touched)
