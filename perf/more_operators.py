"""Operators that serve many continuations of a prompt, as they are measured: cases, inputs, plain forms, exact values.

Three operators of a serving step:

* ``shared``: attention over a paged cache for a batch whose sequences share, group by group, their first tokens: those
  are read and multiplied once for all of a group's rows;
* ``read``: a sequence's tokens out of the pages of a cache that is held in e4m3 with one scale for each block of tokens
  and head, or in 16 bits, as packed rows of 16-bit keys and values;
* ``linear``: linear attention with a decay for each head, S_t = e^g S_(t-1) + k_t v_t^T and o_t = scale q_t S_t, whose
  past is one state a head in a pool of slots: whole prompts, drafts and single tokens.

A case fixes the sizes and every sequence's length; the values and the pages' order come from the seed.
"""

import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CHUNK = 128  # tokens that the plain form of linear attention takes together


def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", batch=1, new=1, ragged=False, heads=32)
    if op == "linear":
        c.update(key_heads=kw.get("heads", 32), key_dim=128, value_dim=128, fresh=False)
    else:
        c.update(cache="e4m3", kv_heads=8, dim=128, page=16, block=16, order="token", length=1)
    if op == "shared":
        c.update(groups=1, shared=1)
    c.update(kw)
    return c


def listed():
    return [
        # Four answers to one short prompt, a few tokens in: the call's latency.
        _case("shared four answers", "shared", batch=4, shared=500, length=530, ragged=True),
        # A decode batch behind one system prompt, each with a conversation of its own.
        _case("shared system prompt", "shared", batch=64, shared=4096, length=5120, ragged=True, page=32),
        # Many samples of one long prompt, a few hundred tokens in: the product over the prefix is what counts.
        _case("shared many samples", "shared", batch=256, shared=32_768, length=33_024, ragged=True, heads=64, page=64, block=64,
              order="head"),
        # Six prompts with eight samples each and three drafted tokens a sample to be checked; a 16-bit cache.
        _case("shared groups drafts", "shared", dtype="fp16", cache="same", batch=48, groups=6, shared=3001, length=3400, ragged=True,
              new=3, heads=24, dim=96, page=16),
        # Users' questions, of up to 400 tokens, behind a common instruction: prompts that continue a prefix.
        _case("shared questions", "shared", batch=16, shared=2048, length=2448, new=400, ragged=True, kv_heads=4, page=64),
        # The tokens of a partly filled page, to be written into another sequence's own: latency.
        _case("read a page", "read", new=41, length=553, page=64),
        # Conversations that leave for another machine, whole: the bandwidth that a cache is read back with.
        _case("read conversations", "read", batch=8, new=16_384, length=16_384, ragged=True, page=32),
        # The last tokens of many sequences out of a 16-bit cache with odd heads.
        _case("read 16 bit", "read", dtype="fp16", cache="same", batch=61, new=1021, length=1500, ragged=True, kv_heads=5, dim=80,
              page=48, order="head"),
        # One user's next token through one layer's states: latency.
        _case("linear one token", "linear", heads=16),
        # A full decode batch: every state is read and written once.
        _case("linear decode batch", "linear", batch=128),
        # A whole prompt of one user, from nothing.
        _case("linear prompt", "linear", new=8192, fresh=True),
        # Prompts of many users that continue, with keys shared by heads and odd sizes.
        _case("linear prompts", "linear", dtype="fp16", batch=24, new=2000, ragged=True, heads=12, key_heads=4, key_dim=64, value_dim=96),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["shared", "shared", "read", "linear", "linear"])
        kw = dict(dtype=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.8)
        kind = rng.choice(["one", "few", "many"])
        if op == "linear":
            key_heads = rng.choice([1, 2, 4, 8, 16])
            kw.update(heads=key_heads * rng.choice([1, 1, 1, 2, 3, 4]), key_heads=key_heads, fresh=rng.random() < 0.3,
                      key_dim=rng.choice([32, 64, 64, 80, 128, 128, 128, 192, 256]),
                      value_dim=rng.choice([32, 64, 64, 96, 128, 128, 128, 192, 256]),
                      batch=_log(rng, 1, {"one": 256, "few": 128, "many": 32}[kind]),
                      new={"one": 1, "few": rng.randint(2, 16), "many": _log(rng, 17, 16_384)}[kind])
            c = _case("", op, **kw)
            rows = sum(_shape(c)[0])
            fits = (work(c)["bytes"] <= 5.4e8 and c["batch"] * c["new"] * c["heads"] * max(c["key_dim"], c["value_dim"]) <= 8e7
                    and rows * c["heads"] * c["key_dim"] * c["value_dim"] <= 4.4e9)
        else:
            kv_heads = rng.choice([1, 2, 4, 8, 16])
            block = rng.choice([16, 16, 32, 64])
            kw.update(cache=rng.choice(["e4m3", "e4m3", "same"]), kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]),
                      dim=rng.choice([64, 64, 80, 96, 112, 128, 128, 128, 192, 256]), block=block, page=block * rng.choice([1, 1, 2, 4]),
                      order=rng.choice(["token", "head"]))
        if op == "read":
            kw["batch"], kw["new"] = _log(rng, 1, 64), _log(rng, 1, 16_384)
            kw["length"] = kw["new"] + rng.choice([0, rng.randint(0, 2000)])
            c = _case("", op, **kw)
            fits = work(c)["bytes"] <= 5.6e8 and c["batch"] * c["length"] * c["kv_heads"] * c["dim"] <= 4e8
        elif op == "shared":
            kw["batch"] = _log(rng, 2, {"one": 256, "few": 64, "many": 16}[kind])
            kw["groups"] = min(kw["batch"], rng.choice([1, 1, 1, 2, 5, 9]))
            kw["new"] = {"one": 1, "few": rng.randint(2, 16), "many": _log(rng, 17, 1000)}[kind]
            kw["shared"] = _log(rng, 16, 65_536)
            kw["length"] = kw["shared"] + kw["new"] + _log(rng, 1, 2000)
            c = _case("", op, **kw)
            w = work(c)
            # No more than the largest listed one, for the kernels and for the plain form (padded scores, gathered caches).
            fits = (w["flops"] <= 2.7e11 and w["bytes"] <= 5.4e8 and c["batch"] * c["heads"] * c["new"] * c["length"] <= 5.4e8
                    and (c["groups"] * c["shared"] + c["batch"] * (c["length"] - c["shared"])) * c["kv_heads"] * c["dim"] <= 4e8)
        if fits:
            del c["name"]
            return c


def _shape(case):
    """New tokens of every sequence, its length with them where it has one, and the sequences that groups begin at: of the case alone."""
    r = random.Random("%d %d %d" % (case["batch"], case["new"], case.get("length", 0)))
    news, lengths = [], []
    first = case.get("shared", 0)
    for b in range(case["batch"]):
        n = case["new"]
        if case["ragged"] and b and n > 16:
            n = r.randint(max(1, n // 2), n)
        news.append(n)
        length = case.get("length", n)
        lengths.append(r.randint(first + n, length) if case["ragged"] and b else length)
    groups = [0]
    n = case.get("groups", 1)
    for g in range(1, n):  # groups of several sizes, one sequence at least
        even = case["batch"] * g // n
        groups.append(min(max(groups[-1] + 1, even + (r.randint(-1, 1) if case["ragged"] else 0)), case["batch"] - (n - g)))
    return news, lengths, groups + [case["batch"]]


def _shares(case):
    """Each group's shared tokens: the first has all, the others up to a quarter less."""
    return [case["shared"] - (case["shared"] // 4 * g // case["groups"] if case["ragged"] else 0) for g in range(case["groups"])]


def _pool(case, pages, heads, dim, dtype, device):
    """Storage of [pages, page, heads, dim], in memory by token or by head."""
    if case["order"] == "token":
        return torch.empty((pages, case["page"], heads, dim), dtype=dtype, device=device)
    return torch.empty((pages, heads, case["page"], dim), dtype=dtype, device=device).transpose(1, 2)


def prepare(case, seed):
    device = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=device).manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    news, lengths, groups = _shape(case)
    tokens, batch, heads = sum(news), case["batch"], case["heads"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device, dtype=torch.float32)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=device)

    s = {"op": case["op"], "starts": ints([sum(news[:b]) for b in range(batch + 1)]), "most": max(news)}
    if case["op"] == "linear":
        dk, dv = case["key_dim"], case["value_dim"]
        # Decays as such models have them: from a few tokens' reach to some hundred.
        s["decay"] = -torch.exp2(-8.0 * torch.arange(1, heads + 1, device=device, dtype=torch.float32) / heads)
        s["q"], s["k"] = (normal(tokens, case["key_heads"], dk).to(dtype) for _ in range(2))
        s["v"] = normal(tokens, heads, dv).to(dtype)
        # A slot to read and another to write for each sequence: the step can be taken back.
        slots = torch.randperm(2 * batch, generator=g, device=device).to(torch.int32)
        s["slots"], s["sources"] = slots[:batch].contiguous(), slots[batch:].contiguous()
        if case["fresh"]:
            s["sources"].fill_(-1)
        s["state"] = normal(2 * batch, heads, dk, dv)
        s["out"] = torch.empty_like(s["v"])
        if own:
            from tensor_layout_amd import linear
            s["pool"] = linear.StatePool(s["state"], s["decay"])
        return s

    held = E4M3 if case["cache"] == "e4m3" else dtype
    page, block, kv_heads, dim = (case[x] for x in ("page", "block", "kv_heads", "dim"))
    width = -(-max(lengths) // page)
    # Whole pages of the shared tokens are the first sequence's of each group; the rest are a sequence's own.
    common = [0] * batch
    if case["op"] == "shared":
        for i, n in enumerate(_shares(case)):
            for b in range(groups[i] + 1, groups[i + 1]):
                common[b] = n // page
        s["groups"], s["shared"] = ints(groups), ints(_shares(case))
        s["widest"] = max(n - c for n, c in zip(lengths, sum(([n] * (groups[i + 1] - groups[i]) for i, n in enumerate(_shares(case))), [])))
        s["most_rows"] = max(sum(news[groups[i]:groups[i + 1]]) for i in range(case["groups"]))
        s["most_shared"] = max(_shares(case))
    used = [-(-n // page) - c for n, c in zip(lengths, common)]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device=device).tolist()
    rows, at = [], 0
    for b in range(batch):
        leader = max(x for x in groups if x <= b)
        row = (rows[leader][:common[b]] if common[b] else []) + order[at:at + used[b]]
        at += used[b]
        rows.append(row + [-1] * (width - len(row)))
    s["table"], s["lengths"], s["block"] = ints(rows), ints(lengths), block
    for name in ("k", "v"):
        c = _pool(case, pages, kv_heads, dim, held, device)
        for a in range(0, pages, 4096):  # values near one; a block's largest uses most of e4m3's range
            x = normal(min(4096, pages - a), page, kv_heads, dim)
            if held == E4M3:
                c[a:a + 4096].view(torch.uint8).copy_((x * 96).clamp_(-448, 448).to(E4M3).view(torch.uint8))
            else:
                c[a:a + 4096].copy_(x)
        s[name + "_cache"] = c
        s[name + "_scale"] = torch.exp2(torch.randint(-8, -5, (pages, kv_heads, page // block), generator=g, device=device).float()) if held == E4M3 else None
    if case["op"] == "shared":
        s["q"] = (normal(tokens, heads, dim) * 2).to(dtype)  # scores that spread: some tokens matter much more than others
        s["scale"] = dim ** -0.5
        s["lse"] = torch.empty((tokens, heads), dtype=torch.float32, device=device)
        s["out"] = torch.empty_like(s["q"])
    else:
        s["k"], s["v"] = (torch.empty((tokens, kv_heads, dim), dtype=dtype, device=device) for _ in range(2))
    if own:
        from tensor_layout_amd import kv
        s["cache"] = kv.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return s


def run(s):
    if s["op"] == "linear":
        if own:
            from tensor_layout_amd import linear
            linear.attend(s["q"], s["k"], s["v"], s["pool"], s["slots"], s["starts"], sources=s["sources"], out=s["out"])
        else:
            _plain_linear(s)
        return {"out": s["out"], "state": s["state"]}
    if s["op"] == "read":
        if own:
            from tensor_layout_amd import kv
            kv.read(s["cache"], s["table"], s["starts"], s["lengths"], s["k"], s["v"])
        else:
            _plain_read(s)
        return {"k": s["k"], "v": s["v"]}
    if own:
        from tensor_layout_amd import kv
        kv.attend_shared(s["q"], s["cache"], s["table"], s["starts"], s["lengths"], s["groups"], s["shared"], scale=s["scale"],
                         out=s["out"], lse=s["lse"])
    else:
        _plain_shared(s)
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the plain forms


def _rows(s, tokens):
    """Each packed row's sequence, and its place among the sequence's new tokens."""
    starts = s["starts"].long()
    row = torch.arange(tokens, device=starts.device)
    seq = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    return seq, row - starts[seq]


def _values(cache, scale, pages, block):
    """Pages [...] of a cache in 32 bits: [..., page, kv_heads, dim]."""
    if scale is None:
        return cache[pages].float()
    x = cache.view(torch.uint8)[pages].view(E4M3).float()
    return x * scale[pages].repeat_interleave(block, -1).transpose(-1, -2)[..., None]


def _plain_read(s):
    tokens = s["k"].shape[0]
    seq, i = _rows(s, tokens)
    lengths, starts, page = s["lengths"].long(), s["starts"].long(), s["k_cache"].shape[1]
    at = lengths[seq] - (starts[seq + 1] - starts[seq]) + i
    where, slot = s["table"].long()[seq, at // page], at % page
    for name in ("k", "v"):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        if scale is None:
            s[name].copy_(cache[where, slot])
        else:
            s[name].copy_(cache.view(torch.uint8)[where, slot].view(E4M3).float() * scale[where, :, slot // s["block"]][..., None])


def _scores(q, k, see, scale):
    """Scores [n, kv_heads, rows, tokens] in 32 bits of q [n, kv_heads, rows, dim] and k [n, kv_heads, tokens, dim]; see: [n, 1, rows, tokens]."""
    x = torch.bmm(q.flatten(0, 1), k.flatten(0, 1).transpose(1, 2).contiguous()).mul_(scale).view(*q.shape[:3], k.shape[2])
    return x.masked_fill_(~see, -math.inf)


def _weighed(x, top, v):
    """exp(x - top) v and the sums of exp(x - top)."""
    p = x.sub_(top).exp_()
    return torch.bmm(p.flatten(0, 1), v.flatten(0, 1)).view(*p.shape[:3], v.shape[3]), p.sum(-1, keepdim=True)


def _plain_shared(s):
    """Prefix scores for all rows of a group at once, then each sequence's own, under one maximum a row."""
    tokens, heads, dim = s["q"].shape
    kv_heads, page = s["k_cache"].shape[2], s["k_cache"].shape[1]
    group = heads // kv_heads
    starts, lengths, groups, shared = (s[x].long() for x in ("starts", "lengths", "groups", "shared"))
    device, most, rows, long_, widest = starts.device, s["most"], s["most_rows"], s["most_shared"], s["widest"]
    table = s["table"].clamp(min=0).long()
    seq, i = _rows(s, tokens)
    of = torch.searchsorted(groups[1:].contiguous(), seq, right=True)  # a row's group, and its place in it
    place = torch.arange(tokens, device=device) - starts[groups[of]]

    def padded(a, b, n, m):  # q's rows as [n, kv_heads, m * group, dim]
        x = torch.zeros((n, m, heads, dim), device=device)
        x[a, b] = s["q"].float()
        return x.view(n, m, kv_heads, group, dim).transpose(1, 2).reshape(n, kv_heads, m * group, dim)

    def back(x, a, b, n, m):  # and back to [tokens, heads, ...]
        return x.view(n, kv_heads, m, group, -1).transpose(1, 2).reshape(n, m, heads, -1)[a, b]

    # The prefix: its pages from each group's first sequence.
    pre = table[groups[:-1], :-(-long_ // page)]
    k, v = (_values(s[x + "_cache"], s[x + "_scale"], pre, s["block"]).flatten(1, 2)[:, :long_].transpose(1, 2).contiguous() for x in "kv")
    see = (torch.arange(long_, device=device) < shared[:, None])[:, None, None]
    n = groups.numel() - 1
    score_p = _scores(padded(of, place, n, rows), k, see, s["scale"])
    v_p = v
    # Each sequence's own tokens, from the shared ones on.
    batch = lengths.numel()
    first = shared[torch.searchsorted(groups[1:].contiguous(), torch.arange(batch, device=device), right=True)]
    at = first[:, None] + torch.arange(widest, device=device)
    there = at < lengths[:, None]
    where = table.gather(1, (at // page).clamp(max=table.shape[1] - 1))
    slot = at % page
    kvs = []
    for x in "kv":
        cache, scale = s[x + "_cache"], s[x + "_scale"]
        if scale is None:
            y = cache[where, slot].float()
        else:
            y = cache.view(torch.uint8)[where, slot].view(E4M3).float() * scale[where, :, slot // s["block"]][..., None]
        kvs.append(y.transpose(1, 2).contiguous())
    pos = (lengths - (starts[1:] - starts[:-1]))[:, None] + torch.arange(most, device=device)
    see = ((at[:, None] <= pos[..., None]) & there[:, None]).repeat_interleave(group, 1)[:, None]
    score_o = _scores(padded(seq, i, batch, most), kvs[0], see, s["scale"])
    # One maximum for both parts of a row.
    top_p, top_o = score_p.amax(-1, keepdim=True), score_o.amax(-1, keepdim=True)
    top = torch.maximum(back(top_p, of, place, n, rows), back(top_o, seq, i, batch, most))
    spread_p, spread_o = torch.zeros((n, rows, heads, 1), device=device), torch.zeros((batch, most, heads, 1), device=device)
    spread_p[of, place], spread_o[seq, i] = top, top
    out_p, sum_p = _weighed(score_p, spread_p.view(n, rows, kv_heads, group, 1).transpose(1, 2).reshape(n, kv_heads, -1, 1), v_p)
    out_o, sum_o = _weighed(score_o, spread_o.view(batch, most, kv_heads, group, 1).transpose(1, 2).reshape(batch, kv_heads, -1, 1), kvs[1])
    total = back(sum_p, of, place, n, rows) + back(sum_o, seq, i, batch, most)
    s["out"].copy_((back(out_p, of, place, n, rows) + back(out_o, seq, i, batch, most)) / total)
    s["lse"].copy_((top + total.log()).squeeze(-1))


def _plain_linear(s):
    """Chunks of tokens: masked products inside a chunk, and the state that each chunk begins with."""
    tokens, heads, dv = s["v"].shape
    dk, batch, most = s["q"].shape[2], s["slots"].numel(), s["most"]
    share = heads // s["q"].shape[1]
    seq, i = _rows(s, tokens)
    device = seq.device
    c = min(CHUNK, most)
    n = -(-most // c)
    g = s["decay"].double()[:, None]
    counts = (s["starts"][1:] - s["starts"][:-1]).long()

    def padded(x):  # [batch * heads, n * c, dim] in 32 bits
        y = torch.zeros((batch, n * c, heads, x.shape[2]), device=device)
        y[seq, i] = x.float().repeat_interleave(heads // x.shape[1], 1)
        return y.transpose(1, 2).contiguous().view(batch * heads, n * c, x.shape[2])

    def power(x):  # e^(g x) for each head, none where x is under zero; repeated for each sequence
        y = torch.exp(g.view(-1, *[1] * x.dim()) * x.clamp(min=0)).masked_fill_(x < 0, 0.0).float()
        return y.repeat(batch, *[1] * x.dim())

    q, k, v = padded(s["q"]), padded(s["k"]), padded(s["v"])
    source = s["sources"].long()
    old = s["state"][source.clamp(min=0)].masked_fill_((source < 0)[:, None, None, None], 0.0).view(batch * heads, dk, dv)
    j = torch.arange(c, device=device)
    inside = power(j[:, None] - j)  # [batch * heads, c, c]
    qc, kc, vc = (x.view(batch * heads * n, c, -1) for x in (q, k, v))
    p = torch.bmm(qc, kc.transpose(1, 2).contiguous()).view(-1, n, c, c).mul_(inside[:, None])
    out = torch.bmm(p.view(-1, c, c), vc).view(batch * heads, n, c, dv)
    # What each chunk adds, and the states before each.
    added = torch.bmm((kc.view(-1, n, c, dk) * power(c - 1 - j)[:, None, :, None]).view(-1, c, dk).transpose(1, 2).contiguous(), vc)
    at = torch.arange(n, device=device)
    ahead = at[:, None] - 1 - at
    begin = torch.bmm(power(torch.where(ahead < 0, -1, ahead * c)), added.view(batch * heads, n, dk * dv))
    begin = begin + power(at * c)[..., None] * old.reshape(batch * heads, 1, dk * dv)
    out = out + torch.bmm((qc.view(-1, n, c, dk) * power(j + 1)[:, None, :, None]).view(-1, c, dk), begin.view(-1, dk, dv)).view_as(out)
    out = out.view(batch, heads, n * c, dv).transpose(1, 2)[seq, i] * dk ** -0.5
    s["out"].copy_(out)
    # The last states: every token's weight by how far from its sequence's end it stands.
    left = (counts[:, None] - 1 - torch.arange(n * c, device=device))[:, None]
    w = torch.exp(g * left.clamp(min=0)).masked_fill_(left < 0, 0.0).float().view(batch * heads, n * c, 1)
    last = torch.bmm((k * w).transpose(1, 2).contiguous(), v)
    last = last + torch.exp(g[:, 0] * counts[:, None]).float().view(-1, 1, 1) * old
    s["state"][s["slots"].long()] = last.view(batch, heads, dk, dv)


# ---------------------------------------------------------------- what the paths cannot do without


def work(case):
    news, lengths, groups = _shape(case)
    tokens, heads = sum(news), case["heads"]
    if case["op"] == "linear":
        dk, dv = case["key_dim"], case["value_dim"]
        states = case["batch"] * heads * dk * dv * 4 * (1 if case["fresh"] else 2)
        return {"bytes": states + tokens * 2 * (2 * case["key_heads"] * dk + 2 * heads * dv), "flops": 4 * tokens * heads * dk * dv}
    held = 1 if case["cache"] == "e4m3" else 2
    token = 2 * case["kv_heads"] * (case["dim"] * held + (4 / case["block"] if held == 1 else 0))
    if case["op"] == "read":
        return {"bytes": tokens * (token + 4 * case["kv_heads"] * case["dim"]), "flops": 0}
    seen = pairs = 0
    for g, n in enumerate(_shares(case)):
        seen += n
        for b in range(groups[g], groups[g + 1]):
            seen += lengths[b] - n
            pairs += news[b] * (lengths[b] - news[b]) + news[b] * (news[b] + 1) // 2
    return {"bytes": seen * token + tokens * heads * (case["dim"] * 4 + 4), "flops": 4 * pairs * heads * case["dim"]}


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    if case["op"] == "linear":
        news = _shape(case)[0]
        if sum(news) * (8e-5 + case["heads"] * case["key_dim"] * case["value_dim"] * 2e-11) > 20:
            return None
        return _exact_linear(prepare(case, seed))
    return (_exact_read if case["op"] == "read" else _exact_shared)(prepare(case, seed))


def _token(s, name, page, slot):
    """Keys or values of tokens in 64 bits: [tokens, kv_heads, dim]."""
    if s[name + "_scale"] is None:
        return s[name + "_cache"][page, slot].double()
    return s[name + "_cache"].view(torch.uint8)[page, slot].view(E4M3).double() * s[name + "_scale"][page, :, slot // s["block"]].double()[..., None]


def _exact_read(s):
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    page, out = s["k_cache"].shape[1], {"k": [], "v": []}
    for b, n in enumerate(lengths):
        j = torch.arange(n - (starts[b + 1] - starts[b]), n, device=s["k"].device)
        for name in out:
            out[name].append(_token(s, name, s["table"][b].long()[j // page], j % page))
    return {name: torch.cat(x) for name, x in out.items()}


def _exact_shared(s):
    """Group by group and head by head; a row's tokens are the group's and its own."""
    starts, lengths, groups, shared = (s[x].tolist() for x in ("starts", "lengths", "groups", "shared"))
    q, page = s["q"], s["k_cache"].shape[1]
    kv_heads, heads = s["k_cache"].shape[2], q.shape[1]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    for g, common in enumerate(shared):
        def tokens(b, lo, hi):
            j = torch.arange(lo, hi, device=q.device)
            where = s["table"][b].long()[j // page]
            return [_token(s, name, where, j % page) for name in ("k", "v")]

        pre = tokens(groups[g], 0, common)
        rows = slice(starts[groups[g]], starts[groups[g + 1]])
        for h in range(kv_heads):
            part = slice(h * (heads // kv_heads), (h + 1) * (heads // kv_heads))
            x = q[rows, part].double()
            score = torch.matmul(x.flatten(0, 1), pre[0][:, h].t().contiguous()) * s["scale"]
            first = torch.logsumexp(score, -1)
            mean = torch.matmul(torch.exp(score - first[:, None]), pre[1][:, h].contiguous())
            lse[rows, part], out[rows, part] = first.view(x.shape[:2]), mean.view(x.shape)
        for b in range(groups[g], groups[g + 1]):
            k, v = tokens(b, common, lengths[b])
            rows, n = slice(starts[b], starts[b + 1]), starts[b + 1] - starts[b]
            pos = torch.arange(lengths[b] - n, lengths[b], device=q.device)
            k, v = (t.repeat_interleave(heads // kv_heads, 1).transpose(0, 1) for t in (k, v))
            x = torch.matmul(q[rows].double().transpose(0, 1), k.transpose(1, 2).contiguous()) * s["scale"]
            x = x.masked_fill(torch.arange(common, lengths[b], device=q.device) > pos[:, None], -math.inf)
            mine = torch.logsumexp(x, -1)
            mean = torch.matmul(torch.exp(x - mine[..., None]), v.contiguous()).transpose(0, 1)
            mine = mine.t()
            total = torch.logaddexp(lse[rows], mine)
            out[rows] = out[rows] * torch.exp(lse[rows] - total)[..., None] + mean * torch.exp(mine - total)[..., None]
            lse[rows] = total
    return {"out": out, "lse": lse}


def _exact_linear(s):
    """The recurrence itself, token by token."""
    starts, slots, sources = (s[x].tolist() for x in ("starts", "slots", "sources"))
    state, share = s["state"].double(), s["v"].shape[1] // s["q"].shape[1]
    q, k, v = s["q"].double().repeat_interleave(share, 1), s["k"].double().repeat_interleave(share, 1), s["v"].double()
    out, keep = torch.empty_like(v), torch.exp(s["decay"].double())[:, None, None]
    for b in range(len(slots)):
        x = state[sources[b]].clone() if sources[b] >= 0 else torch.zeros_like(state[0])
        for t in range(starts[b], starts[b + 1]):
            x.mul_(keep).addcmul_(k[t][:, :, None], v[t][:, None])
            out[t] = (q[t][:, :, None] * x).sum(1)
        state[slots[b]] = x
    return {"out": out * s["q"].shape[2] ** -0.5, "state": state}
