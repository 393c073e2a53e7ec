"""Small batches over a paged cache for the key/value tests."""

from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn


def half_step(dtype) -> float:
    """A rounding's largest error relative to the value."""
    return torch.finfo(dtype).eps / 2


def batch(g, news, lengths, page, *, spare=3, width=None, drop=()):
    """starts, lengths and a table of shuffled pages; `drop`: (sequence, page) entries that are not there."""
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    used = [-(-n // page) for n in lengths]
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=g).tolist()
    width = max(used + [1]) if width is None else width
    table, at = [], 0
    for u in used:
        row = order[at:at + u][:width]
        table.append(row + [-1] * (width - len(row)))
        at += u
    for b, p in drop:
        table[b][p] = -1
    return starts, list(lengths), table, pages


def pools(g, pages, page, kv_heads, dim, dtype, held8, block, by_head):
    """Two pools and their scales, with a NaN in every place; the caller overwrites what it means to hold."""
    out = []
    for _ in range(2):
        x = torch.randn((pages, page, kv_heads, dim), generator=g)
        x = (x * 96).clamp(-448, 448).to(E4M3) if held8 else x.to(dtype)
        if by_head:
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        s = torch.exp2(torch.randint(-8, -5, (pages, kv_heads, page // block), generator=g).float()) if held8 else None
        out += [x, s]
    return out


def poison(pool, table, lengths, page, to=None):
    """NaN wherever the batch holds no token: unused pages and the ends of last ones."""
    keep = torch.zeros(pool.shape[:2], dtype=torch.bool)
    for row, n in zip(table, lengths):
        for j in range(min(n, len(row) * page)):
            if 0 <= row[j // page] < pool.shape[0]:
                keep[row[j // page], j % page] = True
    if pool.dtype == E4M3:
        pool.view(torch.uint8)[~keep] = 0x7F
    else:
        pool[~keep] = float("nan")
