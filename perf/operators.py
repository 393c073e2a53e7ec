"""The paged key/value cache operators as they are measured: their cases, inputs, plain forms and exact values.

Two operators of a serving step:

* ``append``: the new tokens' keys are rotated to their positions and written, with the values, into the pages of a
  cache that is held in e4m3 with one scale for each block of tokens and head, or in the inputs' own 16-bit type; the
  queries are rotated in the same pass;
* ``attend``: each query row attends to the tokens of its own sequence that the cache holds, up to its own position,
  or to the last ``window`` of them and the first ``sinks``.

A case fixes the sizes and every sequence's length; the values and the pages' order come from the seed.
"""

import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", cache="e4m3", batch=1, prompts=0, new=1, length=1, ragged=False, heads=32,
             kv_heads=8, dim=128, page=16, block=16, order="token")
    if op == "append":
        c.update(rot=c["dim"], interleaved=False, sections="", far=0)
    else:
        c.update(window=0, sinks=0)
    c.update(kw)
    return c


def listed():
    return [
        # One user's next token: the call's own latency.
        _case("append one token", "append", length=41, far=100_000),
        # A full decode batch: one token a sequence, most of them into a block that holds some already.
        _case("append decode batch", "append", batch=256, length=80, ragged=True, page=32, far=30_000),
        # Three long prompts with image tokens: positions of three axes (time, height, width), large pages and blocks.
        _case("append prompts three axes", "append", dtype="fp16", batch=3, prompts=3, new=4093, length=4109, ragged=True,
              heads=28, kv_heads=4, page=64, block=64, order="head", sections="16,24,24"),
        # Eight prompts of a model with small heads, half of each rotated in interleaved pairs, into a 16-bit cache.
        _case("append prompts 16 bit", "append", cache="same", batch=8, prompts=8, new=8192, length=8192, heads=16,
              kv_heads=16, dim=64, page=64, rot=32, interleaved=True),
        # One user's next token after a short conversation: latency.
        _case("decode one", "attend", length=777),
        # A decode batch of ragged conversations: the bandwidth that the cache is read with.
        _case("decode batch", "attend", batch=64, length=8192, ragged=True, page=32),
        # Two users with whole books in the cache: few rows, a long axis to split.
        _case("decode long", "attend", dtype="fp16", batch=2, length=131_009, heads=64, page=64, block=64, order="head"),
        # A layer with a window and four first tokens that stay visible, deep in long conversations.
        _case("decode window", "attend", batch=64, length=16_384, ragged=True, heads=64, dim=64, window=1024, sinks=4),
        # Four drafted tokens a sequence to be checked; three query heads share one of the cache.
        _case("verify drafts", "attend", batch=32, prompts=32, new=4, length=4096, ragged=True, heads=24, dim=96),
        # A whole prompt at once: the largest product.
        _case("prompt", "attend", prompts=1, new=8192, length=8192, page=64),
        # Two prompts through a windowed layer with a 16-bit cache and no shared heads.
        _case("prompt window 16 bit", "attend", dtype="fp16", cache="same", batch=2, prompts=2, new=8000, length=8000,
              ragged=True, heads=16, kv_heads=16, dim=64, page=32, order="head", window=1024, sinks=4),
        # A chunk of one prompt among eight decoding sequences.
        _case("mixed", "attend", batch=9, prompts=1, new=1024, length=4096, ragged=True, kv_heads=4, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        block = rng.choice([16, 16, 32, 64])
        kw = dict(dtype=rng.choice(["bf16", "fp16"]), cache=rng.choice(["e4m3", "e4m3", "same"]), ragged=rng.random() < 0.7,
                  kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]),
                  dim=rng.choice([64, 64, 80, 96, 112, 128, 128, 128, 192, 256]), block=block,
                  page=block * rng.choice([1, 1, 2, 4]), order=rng.choice(["token", "head"]))
        kind = rng.choice(["decode", "prompts", "few"])
        kw["batch"] = _log(rng, 1, 256 if kind == "decode" else 8 if kind == "prompts" else 64)
        if kind == "prompts":
            kw["new"] = _log(rng, 33, 8192)
            kw["prompts"] = rng.randint(1, kw["batch"])
        elif kind == "few":
            kw["new"] = rng.randint(2, 32)
            kw["prompts"] = kw["batch"]
        if rng.random() < 0.4:
            kw["length"] = kw.get("new", 1) + rng.randint(0, 100)
            c = _case("", "append", **kw)
            c["rot"] = c["dim"] if rng.random() < 0.6 else c["dim"] // 2
            c["interleaved"] = rng.random() < 0.4
            c["far"] = rng.choice([0, 4000, 1_000_000])
            if rng.random() < 0.3:
                half = c["rot"] // 2
                a = rng.randint(1, half - 2)
                b = rng.randint(1, half - a - 1)
                c["sections"] = "%d,%d,%d" % (a, b, half - a - b)
            fits = sum(_shape(c)[0]) * (c["heads"] + 4 * c["kv_heads"]) * c["dim"] <= 3.3e8
        else:
            kw["length"] = max(kw.get("new", 1), _log(rng, 1, 131_072))
            c = _case("", "attend", **kw)
            if rng.random() < 0.4:
                c["window"] = _log(rng, 16, 4096)
                c["sinks"] = rng.choice([0, 1, 4, 16, 65])
            # No more than the largest listed ones, for the kernels (work) and for the plain form (padded scores, gathered cache).
            w = work(c)
            fits = (c["batch"] * c["heads"] * c["new"] * c["length"] <= 2.1e9 and w["bytes"] <= 5.4e8 and w["flops"] <= 5.4e11
                    and c["batch"] * c["kv_heads"] * c["length"] * c["dim"] <= 5.4e8)
        if fits:
            del c["name"]
            return c


def _shape(case):
    """(new tokens, length with them) of every sequence: of the case alone."""
    r = random.Random("%d %d %d" % (case["batch"], case["new"], case["length"]))
    news, lengths = [], []
    for b in range(case["batch"]):
        n = 1
        if b < case["prompts"]:
            n = r.randint(max(1, case["new"] // 2), case["new"]) if case["ragged"] and b and case["new"] > 32 else case["new"]
        news.append(n)
        lengths.append(r.randint(max(n, case["length"] // 4), case["length"]) if case["ragged"] and b else case["length"])
    return news, lengths


def _sections(case):
    return tuple(int(x) for x in case["sections"].split(",")) if case["sections"] else None


def _pool(case, pages, heads, dim, dtype, device):
    """Storage of [pages, page, heads, dim], in memory by token or by head."""
    if case["order"] == "token":
        return torch.empty((pages, case["page"], heads, dim), dtype=dtype, device=device)
    return torch.empty((pages, heads, case["page"], dim), dtype=dtype, device=device).transpose(1, 2)


def prepare(case, seed):
    device = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=device).manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    held = E4M3 if case["cache"] == "e4m3" else dtype
    news, lengths = _shape(case)
    batch, page, block, heads, kv_heads, dim = (case[x] for x in ("batch", "page", "block", "heads", "kv_heads", "dim"))
    tokens, width = sum(news), -(-max(lengths) // page)
    used = [-(-n // page) for n in lengths]
    pages = sum(used) + 3

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device, dtype=torch.float32)

    order = torch.randperm(pages, generator=g, device=device).to(torch.int32)
    at = torch.tensor([sum(used[:b]) for b in range(batch)], device=device)[:, None] + torch.arange(width, device=device)[None]
    there = torch.arange(width, device=device)[None] < torch.tensor(used, device=device)[:, None]
    if case["op"] == "attend" and case["window"]:  # what lies between the first tokens and the window has been given back
        lo = torch.tensor([n - m - case["window"] for m, n in zip(news, lengths)], device=device)[:, None]
        p = torch.arange(width, device=device)[None] * page
        there = there & ((p < case["sinks"]) | (p + page > lo))
    table = torch.where(there, order[at.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    starts = torch.tensor([sum(news[:b]) for b in range(batch + 1)], dtype=torch.int32, device=device)
    lengths_ = torch.tensor(lengths, dtype=torch.int32, device=device)

    caches, scales = [], []
    for _ in range(2):
        c = _pool(case, pages, kv_heads, dim, held, device)
        for a in range(0, pages, 4096):  # values near one; a block's largest uses most of e4m3's range
            x = normal(min(4096, pages - a), page, kv_heads, dim)
            if held == E4M3:
                c[a:a + 4096].view(torch.uint8).copy_((x * 96).clamp_(-448, 448).to(E4M3).view(torch.uint8))
            else:
                c[a:a + 4096].copy_(x)
        caches.append(c)
        scales.append(torch.exp2(torch.randint(-8, -5, (pages, kv_heads, page // block), generator=g, device=device).float()) if held == E4M3 else None)
    s = {"op": case["op"], "table": table, "starts": starts, "lengths": lengths_, "block": block, "most": max(news),
         "k_cache": caches[0], "v_cache": caches[1], "k_scale": scales[0], "v_scale": scales[1],
         "q": normal(tokens, heads, dim).to(dtype)}
    if case["op"] == "append":
        # Some channels of keys are several times as large as the others, as they are in models.
        s["k"] = (normal(tokens, kv_heads, dim) * torch.exp(normal(1, kv_heads, dim))).to(dtype)
        s["v"] = normal(tokens, kv_heads, dim).to(dtype)
        rot, sections = case["rot"], _sections(case)
        s["inv_freq"] = (10_000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)).float()
        seq = torch.repeat_interleave(torch.arange(batch, device=device), torch.tensor(news, device=device))
        index = torch.arange(tokens, device=device) - starts[seq] + lengths_[seq] - torch.tensor(news, device=device)[seq]
        s["positions"] = None
        if sections:  # image patches: a time for each group of tokens, a height and a width within it
            s["positions"] = torch.stack([index // 256 + case["far"], index // 16 % 16, index % 16]).to(torch.int32).contiguous()
        elif case["far"]:
            s["positions"] = (index + case["far"]).to(torch.int32)[None].contiguous()
        s["sections"], s["interleaved"] = sections, case["interleaved"]
        s["q_out"] = torch.empty_like(s["q"])
    else:
        s["q"] = (s["q"].float() * 2).to(dtype)  # scores that spread: some tokens matter much more than others
        s["scale"], s["window"], s["sinks"] = dim ** -0.5, case["window"], case["sinks"]
        s["lse"] = torch.empty((tokens, heads), dtype=torch.float32, device=device)
        s["out"] = torch.empty_like(s["q"])
    if own:
        from tensor_layout_amd import kv
        s["cache"] = kv.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return s


def run(s):
    if s["op"] == "append":
        if own:
            from tensor_layout_amd import kv
            kv.append(s["cache"], s["k"], s["v"], s["table"], s["starts"], s["lengths"], q=s["q"], q_out=s["q_out"],
                      inv_freq=s["inv_freq"], positions=s["positions"], sections=s["sections"], interleaved=s["interleaved"])
        else:
            _plain_append(s)
        out = {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
        if s["k_scale"] is not None:
            out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
        return out
    if own:
        from tensor_layout_amd import kv
        kv.attend(s["q"], s["cache"], s["table"], s["starts"], s["lengths"], scale=s["scale"], window=s["window"],
                  sinks=s["sinks"], out=s["out"], lse=s["lse"])
    else:
        _plain_attend(s)
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the plain forms


def _rows(s, tokens):
    """Each packed row's sequence, and its token's index in that sequence."""
    starts = s["starts"].long()
    row = torch.arange(tokens, device=starts.device)
    seq = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    return seq, row - starts[seq + 1] + s["lengths"].long()[seq]


def _rotated(x, cos, sin, interleaved):
    """x [tokens, heads, dim] in 32 bits with its first 2 * cos.shape[-1] channels rotated."""
    x, half = x.float(), cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _plain_append(s):
    tokens = s["k"].shape[0]
    seq, index = _rows(s, tokens)
    pos = index[None] if s["positions"] is None else s["positions"]
    f = s["inv_freq"].double()
    if s["sections"] is None:
        axis = torch.zeros(f.numel(), dtype=torch.long, device=f.device)
    else:
        axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=f.device), torch.tensor(s["sections"], device=f.device))
    angle = pos.double()[axis].t() * f
    cos, sin = angle.cos().float(), angle.sin().float()
    s["q_out"].copy_(_rotated(s["q"], cos, sin, s["interleaved"]))
    page, block = s["k_cache"].shape[1], s["block"]
    where = s["table"].long()[seq, index // page]
    slot = index % page
    for x, cache, scale in ((_rotated(s["k"], cos, sin, s["interleaved"]), s["k_cache"], s["k_scale"]), (s["v"].float(), s["v_cache"], s["v_scale"])):
        if scale is None:
            cache[where, slot] = x.to(cache.dtype)
            continue
        held = cache.view(torch.uint8)
        # Each touched block's number: a sequence's blocks follow one another.
        starts, lengths = s["starts"].long(), s["lengths"].long()
        first = (lengths - (starts[1:] - starts[:-1])) // block
        ids = (starts[:-1] // block + 2 * torch.arange(len(lengths), device=x.device) - first)[seq] + index // block
        count = tokens // block + 2 * len(lengths)
        amax = torch.zeros((count, x.shape[1]), device=x.device)
        amax.scatter_reduce_(0, ids[:, None].expand(-1, x.shape[1]), torch.where(x.isfinite(), x.abs(), 0.0).amax(-1), "amax")
        part, exponent = torch.frexp(amax)  # the least power of two that brings amax to 448 = 0.875 * 2^9 or under
        new = torch.exp2((exponent - 9 + (part > 0.875)).clamp(-126, 127).float()).masked_fill_(amax == 0, 2.0 ** -126)
        # Tokens that a sequence's first touched block holds already keep their values under the larger scale.
        b0 = (lengths - (starts[1:] - starts[:-1])) // block
        had = (lengths - (starts[1:] - starts[:-1])) % block
        row0 = starts[:-1].clamp(max=tokens - 1)
        some = (had > 0) & (starts[1:] > starts[:-1])
        where0 = s["table"].long()[torch.arange(len(b0), device=x.device), (b0 * block // page).clamp(max=s["table"].shape[1] - 1)].clamp(min=0)
        old = scale[where0, :, b0 % (page // block)]
        grown = torch.where(some[:, None], torch.maximum(old, new[ids[row0]]), new[ids[row0]])
        new[ids[row0]] = grown
        inside = torch.arange(block, device=x.device)
        at = (where0[:, None], (b0 * block % page)[:, None] + inside)
        was = held[at].view(E4M3).float()
        now = (was * (old / grown)[:, None, :, None]).to(E4M3).view(torch.uint8)
        change = some[:, None] & (inside < had[:, None])
        held[at[0].expand_as(change)[change], at[1][change]] = now[change]
        mine = new[ids]
        scale[where, :, slot // block] = mine
        held[where, slot] = (x / mine[..., None]).to(E4M3).view(torch.uint8)


def _gathered(cache, scale, table, block):
    """[batch, kv_heads, width * page, dim] in 32 bits."""
    t = table.clamp(min=0).long()
    if scale is None:
        x = cache[t].float()
    else:
        x = cache.view(torch.uint8)[t].view(E4M3).float()
        x = x * scale[t].repeat_interleave(block, -1).transpose(2, 3)[..., None]
    return x.permute(0, 3, 1, 2, 4).flatten(2, 3).contiguous()


def _visible(s, most, length):
    """[batch, most, length]: which tokens each of a sequence's rows sees."""
    lengths = s["lengths"].long()
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(most, device=lengths.device)
    j = torch.arange(length, device=lengths.device)
    pos = (lengths - count)[:, None] + i
    see = (j <= pos[..., None]) & (i < count[:, None])[..., None]
    if s["window"]:
        see &= (j > pos[..., None] - s["window"]) | (j < s["sinks"])
    ok = (s["table"] >= 0) & (s["table"] < s["k_cache"].shape[0])
    return see & ok.repeat_interleave(s["k_cache"].shape[1], 1)[:, None]


def _plain_attend(s):
    tokens, heads, dim = s["q"].shape
    batch, most = s["table"].shape[0], s["most"]
    k = _gathered(s["k_cache"], s["k_scale"], s["table"], s["block"])
    v = _gathered(s["v_cache"], s["v_scale"], s["table"], s["block"])
    kv_heads, length = k.shape[1], k.shape[2]
    row = s["starts"][:-1].long()[:, None] + torch.arange(most, device=k.device)
    q = s["q"][row.clamp(max=tokens - 1)].float().reshape(batch, most, kv_heads, heads // kv_heads, dim)
    q = q.permute(0, 2, 3, 1, 4).reshape(batch * kv_heads, -1, dim)
    score = torch.bmm(q, k.flatten(0, 1).transpose(1, 2).contiguous()).mul_(s["scale"])
    score = score.view(batch, kv_heads, heads // kv_heads, most, length)
    score.masked_fill_(~_visible(s, most, length)[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p.view(batch * kv_heads, -1, length), v.flatten(0, 1)).view(batch, kv_heads, -1, most, dim)
    out = (out / total.masked_fill(total == 0, 1.0)).permute(0, 3, 1, 2, 4).reshape(batch, most, heads, dim)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(batch, most, heads)
    seq, _ = _rows(s, tokens)
    i = torch.arange(tokens, device=k.device) - s["starts"].long()[seq]
    s["out"].copy_(out[seq, i])
    s["lse"].copy_(lse[seq, i])


# ---------------------------------------------------------------- what the paths cannot do without


def work(case):
    news, lengths = _shape(case)
    tokens = sum(news)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    held = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        moved = tokens * (heads * dim * 4 + 2 * kv_heads * dim * (2 + held))
        if held == 1:
            moved += 2 * 4 * kv_heads * sum(-(-n // case["block"]) for n in news)
        return {"bytes": moved + 4 * case["batch"] * 3, "flops": 3 * tokens * (heads + kv_heads) * case["rot"]}
    seen = pairs = 0
    for n, length in zip(news, lengths):
        first = length - n
        if not case["window"]:
            pairs += n * first + n * (n + 1) // 2
            seen += length
            continue
        w, sinks = case["window"], case["sinks"]
        lo = max(0, first - w + 1)
        seen += length - lo + min(sinks, lo)
        for p in (first, length - 1) if n > 64 else range(first, length):  # the ends' mean stands for a long prompt
            a = max(0, p - w + 1)
            pairs += (p + 1 - a + min(sinks, a)) * (n / 2 if n > 64 else 1)
    moved = 2 * seen * kv_heads * (dim * held + (4 / case["block"] if held == 1 else 0))
    return {"bytes": moved + tokens * heads * (dim * 4 + 4), "flops": 4 * pairs * heads * dim}


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if s["op"] == "append" else _exact_attend(s)


def _exact_append(s):
    """Sequence by sequence and block by block. What the cache holds is given before its last rounding: the value over its block's scale."""
    def turned(x):
        n = s["inv_freq"].numel()
        y = x.double().clone()
        for c in range(n):
            a, b = (2 * c, 2 * c + 1) if s["interleaved"] else (c, c + n)
            axis = 0
            if s["sections"]:
                while c >= sum(s["sections"][:axis + 1]):
                    axis += 1
            z = torch.polar(torch.ones_like(place[axis]), place[axis] * s["inv_freq"][c].double())[:, None]
            z = torch.complex(x[..., a].double(), x[..., b].double()) * z
            y[..., a], y[..., b] = z.real, z.imag
        return y

    starts, lengths, table = (s[k].tolist() for k in ("starts", "lengths", "table"))
    page, block = s["k_cache"].shape[1], s["block"]
    if s["positions"] is None:
        index = [lengths[b] - starts[b + 1] + t for b in range(len(lengths)) for t in range(starts[b], starts[b + 1])]
        place = torch.tensor([index], dtype=torch.float64, device=s["q"].device)
    else:
        place = s["positions"].double()
    out = {"q": turned(s["q"])}
    for name, x in (("k", turned(s["k"])), ("v", s["v"].double())):
        cache, scale = s[name + "_cache"].double(), s[name + "_scale"]
        scale = None if scale is None else scale.double().cpu()
        for b, length in enumerate(lengths):
            at = length - (starts[b + 1] - starts[b])
            while at < length:
                end = min(length, at // block * block + block)
                p, j = table[b][at // page], at % page
                new = x[starts[b + 1] - length + at:starts[b + 1] - length + end]
                if scale is not None:
                    had = at % block
                    for h, a in enumerate(new.abs().amax((0, 2)).tolist()):
                        e = -126 if a == 0 else math.ceil(math.log2(a / 448))
                        e += (448 * 2.0 ** e < a) - (448 * 2.0 ** (e - 1) >= a > 0)
                        old = float(scale[p, h, j // block])
                        now = max(2.0 ** max(e, -126), old if had else 0.0)
                        if had:
                            cache[p, j - had:j, h] *= old / now
                        scale[p, h, j // block] = now
                    new = new / scale[p, :, j // block].to(new.device)[:, None]
                cache[p, j:j + end - at] = new
                at = end
        out[name] = cache
        if scale is not None:
            out[name + "_scale"] = scale
    return out


def _exact_attend(s):
    """Sequence by sequence, a few heads and rows at a time."""
    starts, lengths, table = (s[k].tolist() for k in ("starts", "lengths", "table"))
    q, pool, page = s["q"], s["k_cache"], s["k_cache"].shape[1]
    heads, dim, kv_heads = q.shape[1], q.shape[2], pool.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for b, length in enumerate(lengths):
        n = starts[b + 1] - starts[b]
        j = torch.tensor([t for t in range(length) if 0 <= table[b][t // page] < pool.shape[0]], device=q.device)
        where = s["table"][b].long()[j // page]
        for h in range(kv_heads):
            k, v = s["k_cache"][where, j % page, h] if s["k_scale"] is None else None, None
            if k is None:
                k = s["k_cache"].view(torch.uint8)[where, j % page, h].view(E4M3).double() * s["k_scale"][where, h, j % page // s["block"]].double()[:, None]
                v = s["v_cache"].view(torch.uint8)[where, j % page, h].view(E4M3).double() * s["v_scale"][where, h, j % page // s["block"]].double()[:, None]
            else:
                k, v = k.double(), s["v_cache"][where, j % page, h].double()
            for i in range(0, n, 2048):
                rows = slice(starts[b] + i, starts[b] + min(n, i + 2048))
                pos = torch.arange(length - n + i, length - n + min(n, i + 2048), device=q.device)[:, None]
                see = j <= pos
                if s["window"]:
                    see = see & ((pos - j < s["window"]) | (j < s["sinks"]))
                share = slice(h * (heads // kv_heads), (h + 1) * (heads // kv_heads))
                x = q[rows, share].double().transpose(0, 1) @ k.t() * s["scale"]
                x = torch.where(see, x, -math.inf)
                total = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(total.isfinite(), total, 0.0)[..., None])
                out[rows, share] = (p @ v).transpose(0, 1)
                lse[rows, share] = total.transpose(0, 1)
    return {"out": out, "lse": lse}
