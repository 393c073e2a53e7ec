"""Paged key/value cache operators where calls meet each other or their limits, against the statement in 64 bits.

Tolerances are those of tests/test_gpu_kv.py, whose checks these tests use."""

from __future__ import annotations

import math

import pytest
import torch

from oracle import kv_oracle
from tests import kv_cases
from tests.kv_cases import half_step
from tests.test_gpu_kv import TYPES, check_append, check_attend, compare_attend, dev, on_gpu

pytestmark = pytest.mark.gpu


def attend_on(cache, host, g, news, lengths, table, heads, dtype, held8, scale=0.125):
    """One call on a cache that lives on, against the statement."""
    from tensor_layout_amd import kv
    k, ks, v, vs = host
    starts = [sum(news[:b]) for b in range(len(news) + 1)]
    q = torch.randn((starts[-1], heads, k.shape[3]), generator=g).to(dtype)
    want = kv_oracle.attend(q, k, v, ks, vs, table, starts, lengths, scale)
    got, lse = torch.full(q.shape, 7.0, dtype=dtype, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    kv.attend(dev(q), cache, dev(table), dev(starts), dev(lengths), scale=scale, out=got, lse=lse)
    compare_attend(got.cpu(), lse.cpu(), *want, v, vs, dtype, held8, k.shape[3], max(lengths))


@pytest.mark.parametrize("dtype,held8", TYPES)
def test_one_cache_for_a_prompt_and_the_tokens_after_it(dtype, held8):
    """Calls of every kind in turn on one cache and stream: none leaves anything in the workspace that the next one meets."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(41)
    page, kv_heads, heads, dim, tokens = 32, 2, 8, 64, 2600
    _, _, table, pages = kv_cases.batch(g, [1, 1], [tokens, 700], page)
    host = kv_cases.pools(g, pages, page, kv_heads, dim, dtype, held8, 16, False)
    cache = kv.PagedCache(on_gpu(host[0]), on_gpu(host[2]), dev(host[1]), dev(host[3]))
    for _ in range(2):
        attend_on(cache, host, g, [100], [2000], table[:1], heads, dtype, held8)   # one prompt's chunk, its tokens split
        attend_on(cache, host, g, [1], [2001], table[:1], heads, dtype, held8)     # the token after it
        attend_on(cache, host, g, [1, 1], [2002, 650], table, heads, dtype, held8)
        attend_on(cache, host, g, [1, 90], [2003, 690], table, heads, dtype, held8)
        torch.cuda.synchronize()
        assert all(not bool(t[:kv.COUNTERS].any()) for _, _, t in cache._work.values())


@pytest.mark.parametrize("dim", range(16, 257, 16))
@pytest.mark.parametrize("dtype,held8", TYPES)
def test_every_length_of_a_head(dim, dtype, held8):
    """Single tokens, drafts and a chunk together, and a prompt by itself."""
    check_attend(42, [1, 5, 70], [150, 60, 200], heads=8, kv_heads=2, dim=dim, dtype=dtype, held8=held8)
    check_attend(43, [70], [130], heads=4, kv_heads=2, dim=dim, dtype=dtype, held8=held8)
    check_attend(44, [4, 4], [90, 300], heads=8, kv_heads=2, dim=dim, dtype=dtype, held8=held8)


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("news,lengths", [([1], [700]), ([1, 4], [33, 150]), ([100], [2000]), ([90, 1], [300, 40]), ([75], [203])])
def test_queries_that_are_no_numbers(news, lengths, dtype, held8):
    """A row whose scores are no numbers has no number for its output: it does not pass for one that sees nothing."""
    def put(q, **_):
        q[0, 0, 3] = math.nan
        q[-1, 5] = math.nan
    check_attend(45, news, lengths, heads=8, kv_heads=2, dim=64, dtype=dtype, held8=held8, tweak=put)


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("news,lengths,at", [([1], [33], 32), ([1], [1], 0), ([1, 1], [640, 129], 128), ([4], [161], 157),
                                             ([100], [2000], 1999), ([100], [2000], 512), ([90, 1], [300, 33], 32)])
def test_a_key_that_is_no_number_shows_wherever_it_stands(news, lengths, at, dtype, held8):
    """Also where no other token is taken by the same wave, or the same part of a split sequence."""
    def put(k, table, **_):
        b = len(table) - 1
        k[table[b][at // 32], at % 32, 1, 7] = math.nan
    check_attend(46, news, lengths, heads=8, kv_heads=2, dim=64, dtype=dtype, held8=held8, tweak=put)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("news,lengths,at", [([1], [33], 32), ([1], [640], 128), ([4], [161], 157), ([100], [2000], 512)])
def test_a_key_without_end(news, lengths, at, dtype):
    """Scores of plus and minus infinity, as the queries' signs have it."""
    def put(k, table, **_):
        k[table[0][at // 32], at % 32, 1, 7] = math.inf
    check_attend(47, news, lengths, heads=8, kv_heads=2, dim=64, dtype=dtype, held8=False, tweak=put)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("news", [[1, 1, 1], [5, 2, 3], [90, 70, 1], [100]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_scales_of_pages_that_hold_nothing(news, window, sinks, bad, dtype):
    """Pools and scales fresh from the allocator: what no token stands under is read by no row, page 0's among it."""
    from tensor_layout_amd import kv
    page, block, kv_heads, dim = 32, 16, 2, 64
    g = torch.Generator().manual_seed(48)
    lengths = [400, 500, 100][:len(news)]
    starts, lengths, table, pages = kv_cases.batch(g, news, lengths, page)
    spare = next(p for p in range(pages) if not any(p in row for row in table))
    table = [[spare if p == 0 else p for p in row] for row in table]
    for b, p in ((0, 0), (0, 3), (1, 1), (1, 11)):
        if b < len(table):
            table[b][p] = -1
    k, ks, v, vs = kv_cases.pools(g, pages, page, kv_heads, dim, dtype, True, block, False)
    for x in (k, v):
        kv_cases.poison(x, table, lengths, page)
    held = torch.zeros((pages, page // block), dtype=torch.bool)
    for row, n in zip(table, lengths):
        for j in range(0, n, block):
            if row[j // page] >= 0:
                held[row[j // page], j % page // block] = True
    for x in (ks, vs):
        x.copy_(torch.where(held[:, None], x, bad))
    q = torch.randn((starts[-1], 4, dim), generator=g).to(dtype)
    want = kv_oracle.attend(q, k, v, ks, vs, table, starts, lengths, 0.125, window, sinks)
    got, lse = torch.empty_like(q, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    kv.attend(dev(q), kv.PagedCache(on_gpu(k), on_gpu(v), dev(ks), dev(vs)), dev(table), dev(starts), dev(lengths), scale=0.125,
              window=window, sinks=sinks, out=got, lse=lse)
    compare_attend(got.cpu(), lse.cpu(), *want, v, vs, dtype, True, dim, 500)


def out_of_order(*changes):
    """starts[b] = x for each (b, x): the sequences on both sides of it are out of order, all others stay as they are."""
    def put(starts, **_):
        for b, x in changes:
            starts[b] = x
    return put


BAD_STARTS = [((1, 10_000),), ((2, -50),), ((1, 1 << 30), (4, -(1 << 30))), ((5, 0),), ((3, 10_000), (4, 5))]


@pytest.mark.parametrize("changes", BAD_STARTS)
@pytest.mark.parametrize("news", [[40, 40, 150, 1, 130, 90], [80] * 6, [3, 1, 2, 5, 1, 2]])
def test_prompts_beside_a_sequence_that_is_skipped(news, changes):
    check_attend(49, news, [n + (60 if n > 8 else 1) for n in news], heads=8, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True,
                 tweak=out_of_order(*changes))


def test_split_prompts_beside_a_sequence_that_is_skipped():
    check_attend(50, [10, 60, 90], [70, 1500, 1200], heads=4, kv_heads=1, dim=64, dtype=torch.float16, held8=False,
                 tweak=out_of_order((1, 500), (0, -3)))
    def long(lengths, **_):
        lengths[0] = (1 << 30) + 1
    check_attend(51, [80, 60, 90], [90, 1500, 1200], heads=4, kv_heads=1, dim=64, dtype=torch.bfloat16, held8=False, width=60,
                 tweak=long)


def test_prompts_of_many_sequences_some_of_which_are_skipped():
    """Over 64 sequences: they are looked through 64 at a time."""
    n = [1 + 37 * i % 60 for i in range(150)]
    check_attend(52, n, [x + 5 for x in n], heads=4, kv_heads=1, dim=16, dtype=torch.bfloat16, held8=True, page=16,
                 tweak=out_of_order((3, 1 << 20), (70, -4), (149, 0)))


@pytest.mark.parametrize("changes", BAD_STARTS)
@pytest.mark.parametrize("news", [[40, 40, 150, 1, 130, 90], [80] * 6, [1] * 6, [2, 1, 3, 1, 1, 2]])
@pytest.mark.parametrize("held8", [True, False])
def test_append_beside_a_sequence_that_is_skipped(news, changes, held8):
    check_append(53, news, [n + (60 if n > 8 else 1) for n in news], heads=4, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=held8,
                 tweak=out_of_order(*changes))


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("held8", [True, False])
def test_append_of_many_sequences_some_of_which_are_skipped(n, held8):
    check_append(54, [n] * 150, [n + 7 * i % 30 for i in range(150)], heads=2, kv_heads=1, dim=16, dtype=torch.bfloat16, held8=held8,
                 page=16, tweak=out_of_order((3, 1 << 20), (70, -4), (100, 9), (140, 1 << 30)))


# ---------------------------------------------------------------- streams


def step_on(cache, g, new=1, length=1500, heads=8, kv_heads=2, dim=64):
    """Arguments of one attend call of a sequence on pages in order, and its queries on the GPU."""
    table = dev([list(range(cache.k.shape[0]))])
    return torch.randn((new, heads, dim), generator=g).to(cache.k.dtype).cuda(), table, dev([0, new]), dev([length])


def small_cache(g, pages=60, page=32, kv_heads=2, dim=64, dtype=torch.bfloat16):
    from tensor_layout_amd import kv
    k, _, v, _ = kv_cases.pools(g, pages, page, kv_heads, dim, dtype, False, 16, False)
    return kv.PagedCache(k.cuda(), v.cuda())


def test_a_graph_captured_on_a_named_stream_has_its_own_workspace():
    """The named stream is the one that captures, whatever torch's current one is: replays leave the eager calls' memory alone."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(55)
    cache = small_cache(g)
    q, table, starts, lengths = step_on(cache, g)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    name = side.cuda_stream
    want = kv.attend(q, cache, table, starts, lengths)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    out = torch.empty_like(q)
    kv.attend(q, cache, table, starts, lengths, out=out, stream=name)   # an eager call first: the stream has a workspace
    torch.cuda.synchronize()
    before = dict(cache._work)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            kv.attend(q, cache, table, starts, lengths, out=out, stream=name)
    assert cache._work == before
    mine = cache._work[name][2]
    mine[kv.COUNTERS:].fill_(0x5A)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert bool((mine[kv.COUNTERS:] == 0x5A).all()) and not bool(mine[:kv.COUNTERS].any())
    kv.attend(q, cache, table, starts, lengths, out=out.zero_(), stream=name)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_the_default_stream_by_its_name():
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(64)
    cache = small_cache(g)
    q, table, starts, lengths = step_on(cache, g, new=3)
    want = kv.attend(q, cache, table, starts, lengths)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(2):
            out = kv.attend(q, cache, table, starts, lengths, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_result_made_for_a_named_stream_is_that_streams():
    """Memory that the current stream has just given back may still be at work there: it is not what a call on another
    stream gets for its result."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(56)
    cache = small_cache(g)
    q, table, starts, lengths = step_on(cache, g, new=40)
    k = torch.randn((40, 2, 64), generator=g).to(cache.k.dtype).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda: kv.attend(q, cache, table, starts, lengths, stream=side.cuda_stream),
                 lambda: kv.append(cache, k, k, table, starts, lengths, q=q, stream=side.cuda_stream)):
        freed = torch.empty_like(q)
        at = freed.data_ptr()
        del freed
        out = call()
        assert out.data_ptr() != at
        assert torch.empty_like(q).data_ptr() == at
        torch.cuda.synchronize()


@pytest.mark.parametrize("n,length", [(1, 31), (5, 36), (100, 400)])
def test_many_small_weights_of_an_fp16_cache(n, length):
    """Weights 2^-26 of the largest: together they are most of an output, and none may be lost for being small.

    Token 0 has a score of 26 log 2 and a value of zero, all others a score of zero and a value of 30000.  Row i's
    output is c 30000 2^-26 / (1 + c 2^-26) with c other tokens, off by the scores' rounding (2^-20 of it at most) and
    by its own rounding in fp16, at outputs under 2^-14 by half of the smallest number."""
    from tensor_layout_amd import kv
    k, v = torch.zeros((16, 32, 1, 64)).half(), torch.full((16, 32, 1, 64), 30000.0).half()
    k[0, 0, 0, 0], v[0, 0] = 26.0, 0.0
    q = torch.zeros((n, 2, 64)).half()
    q[:, :, 0] = 1.0
    got = kv.attend(dev(q), kv.PagedCache(dev(k), dev(v)), dev([list(range(16))]), dev([0, n]), dev([length]), scale=math.log(2.0))
    c = torch.arange(length - n, length, dtype=torch.float64)[:, None, None]
    want = c * 30000 * 2.0 ** -26 / (1 + c * 2.0 ** -26)
    assert bool(((got.cpu().double() - want).abs() <= (2.0 ** -11 + 2.0 ** -20) * want + 2.0 ** -25).all())


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("news,lengths", [([1, 1, 1], [2, 150, 700]), ([4, 3], [9, 400]), ([8], [300])])
def test_weights_of_few_rows_keep_16_bits(news, lengths, dtype, held8):
    """Values that cancel: an output far under the sum of |weight * value| shows its weights' rounding.

    Over e4m3 a weight is two bf16 numbers, each off by half a step (2^-8) of what it holds: 2^-16.  Over bf16 the first
    is cut off, a step (2^-7) at most, and the second is off by half a step of that and 2^-20 of the weight.  Over fp16
    it is one number, half a step of 2^-11, and 2^-32 of the largest at least.  The exponential and the sum: 2^-19."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(57)
    starts, lengths, table, pages = kv_cases.batch(g, news, lengths, 32)
    k, ks, v, vs = kv_cases.pools(g, pages, 32, 2, 64, dtype, held8, 16, False)
    q = torch.randn((starts[-1], 8, 64), generator=g).to(dtype)
    out, _, size, score = kv_oracle.attend(q, k, v, ks, vs, table, starts, lengths, 0.125)
    got = kv.attend(dev(q), kv.PagedCache(on_gpu(k), on_gpu(v), dev(ks), dev(vs)), dev(table), dev(starts), dev(lengths)).cpu()
    u_w = 2.0 ** -16 if held8 else 2.0 ** -15 + 2.0 ** -20 if dtype == torch.bfloat16 else 2.0 ** -11
    tol = (2 * torch.expm1((64 + 8) * 2.0 ** -24 * score)[..., None] + u_w + 2.0 ** -19) * size + half_step(dtype) * out.abs()
    if dtype == torch.float16:
        tol += 2.0 ** -25   # an output under fp16's normal numbers
        tol += 0.0 if held8 else max(lengths) * 2.0 ** -32 * float(v.float().abs().max())
    assert bool(((got.double() - out).abs() <= tol).all())


@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("news,lengths", [([1, 1], [40, 900]), ([4, 2], [40, 900]), ([8], [300]), ([70], [200])])
def test_infinite_values_that_all_rows_see(news, lengths, dtype, value):
    """They come out as they are, whatever their weights' bits."""
    def put(v, table, **_):
        for j in range(0, 33, 3):
            v[table[-1][j // 32], j % 32, j % 2, j] = value
    check_attend(65, news, lengths, heads=16, kv_heads=2, dim=64, dtype=dtype, held8=False, tweak=put, spread=1.0)


@pytest.mark.parametrize("page,block,dim,rot,interleaved", [(256, 256, 128, 128, False), (256, 128, 256, 256, True), (1024, 512, 64, 64, False),
                                                            (512, 512, 128, 36, False), (512, 256, 256, 130, True)])
@pytest.mark.parametrize("news,lengths", [([700, 1, 300], [900, 77, 300]), ([1] * 150, [1 + 37 * i % 400 for i in range(150)]), ([140], [530])])
def test_append_to_long_blocks(page, block, dim, rot, interleaved, news, lengths):
    """One scale for so many tokens that their angles do not fit a workgroup's memory."""
    sections = (rot // 8, rot // 2 - rot // 8) if interleaved else None
    far = 100_000 if interleaved else None
    check_append(66, news, lengths, heads=3, kv_heads=2, dim=dim, dtype=torch.bfloat16 if interleaved else torch.float16, held8=True, rot=rot,
                 interleaved=interleaved, sections=sections, far=far, page=page, block=block, in_place=True, old=2.0 ** -9)


def test_append_to_a_block_of_half_a_million_tokens():
    """The queries are dealt as for any other block: the same bits, and the same scale and values at the sequence's end."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(67)
    k, q = (torch.randn((40, n, 16), generator=g).to(torch.bfloat16).cuda() for n in (1, 3))
    inv = (10_000.0 ** (-torch.arange(0, 16, 2) / 16)).float().cuda()
    got = []
    for page, length in ((1 << 19, 300_000), (64, 64)):
        pool = [torch.zeros((2, page, 1, 16), dtype=torch.uint8, device="cuda").view(kv_cases.E4M3) for _ in range(2)]
        scale = [torch.full((2, 1, 1), 2.0 ** -20, device="cuda") for _ in range(2)]
        at = torch.arange(1000, 1040, dtype=torch.int32, device="cuda")[None]
        out = kv.append(kv.PagedCache(*pool, *scale), k, k, dev([[1]]), dev([0, 40]), dev([length]), q=q, inv_freq=inv, positions=at)
        got.append((out, scale[0][1], *(x.view(torch.uint8)[1, length - 40:length].clone() for x in pool)))
        assert not bool(pool[0].view(torch.uint8)[:, :length - 40].any())
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_caches_share_a_streams_workspace():
    """A model has a cache a layer; only the first call on a stream, and a larger one, takes memory."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(68)
    caches = [small_cache(g) for _ in range(5)]
    q, table, starts, lengths = step_on(caches[0], g)
    outs = [torch.empty_like(q) for _ in caches]
    first = [kv.attend(q, c, table, starts, lengths).clone() for c in caches]
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            kv.attend(q, caches[0], table, starts, lengths, out=outs[0])
            held = torch.cuda.memory_allocated()
            for c, out in zip(caches, outs):
                kv.attend(q, c, table, starts, lengths, out=out)
            assert torch.cuda.memory_allocated() == held
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, outs))


# ---------------------------------------------------------------- sizes that choose other kernels


def values64(pool, scale):
    """A pool's values in 64 bits, on the GPU."""
    x = pool.float().double()
    return x if scale is None else x * scale.double().repeat_interleave(pool.shape[1] // scale.shape[2], 2).transpose(1, 2)[..., None]


def attend64(q, k, v, ks, vs, table, starts, lengths, scale, window=0, sinks=0):
    """The statement's out, lse, size and score on the GPU, a cache head and 1024 rows at a time, for batches too large for its loops."""
    kx, vx = values64(k, ks), values64(v, vs)
    page, kv_heads, group = k.shape[1], k.shape[2], q.shape[1] // k.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    size, score = torch.zeros_like(out), torch.zeros_like(lse)
    for b, length in enumerate(lengths):
        n = starts[b + 1] - starts[b]
        if n == 0:
            continue
        j = torch.tensor([j for j in range(length) if table[b][j // page] >= 0], device="cuda")
        where = torch.tensor(table[b], device="cuda")[j // page]
        for i in range(0, n, 1024):
            rows = slice(starts[b] + i, starts[b] + min(n, i + 1024))
            pos = torch.arange(length - n + i, length - n + min(n, i + 1024), device="cuda")[:, None]
            see = j <= pos
            if window:
                see &= (pos - j < window) | (j < sinks)
            for h in range(kv_heads):
                kk, vv = kx[where, j % page, h], vx[where, j % page, h]
                for a in range(h * group, (h + 1) * group):
                    x = q[rows, a].double()
                    score[rows, a] = ((x.abs() @ kk.abs().t()) * scale).masked_fill_(~see, 0.0).amax(-1)
                    x = (x @ kk.t() * scale).masked_fill_(~see, -math.inf)
                    lse[rows, a] = x.logsumexp(-1)
                    x = (x - lse[rows, a][:, None].nan_to_num(neginf=0.0)).exp()
                    out[rows, a], size[rows, a] = x @ vv, x @ vv.abs()
    return out, lse, size, score


def check_large(seed, news, lengths, *, heads, kv_heads, dim, dtype, held8, page=64, block=16, window=0, sinks=0, by_head=False, width=None):
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(seed)
    starts, lengths, table, pages = kv_cases.batch(g, news, lengths, page, width=width)
    k, ks, v, vs = kv_cases.pools(g, pages, page, kv_heads, dim, dtype, held8, block, by_head)
    for x in (k, v):
        kv_cases.poison(x, table, lengths, page)
    q = torch.randn((starts[-1], heads, dim), generator=g).mul_(2).to(dtype).cuda()
    gpu = [on_gpu(k), on_gpu(v), dev(ks), dev(vs)]
    got, lse = torch.full(q.shape, 7.0, dtype=dtype, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    kv.attend(q, kv.PagedCache(*gpu), dev(table), dev(starts), dev(lengths), scale=dim ** -0.5, window=window, sinks=sinks, out=got, lse=lse)
    want = attend64(q, *gpu, table, starts, lengths, dim ** -0.5, window, sinks)
    compare_attend(got.cpu(), lse.cpu(), *(x.cpu() for x in want), v, vs, dtype, held8, dim, max(lengths))


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("heads,kv_heads,dim,new,length", [(64, 16, 64, 2100, 2100), (48, 16, 96, 2800, 2900), (32, 32, 128, 4200, 4500)])
def test_row_tiles_of_256(heads, kv_heads, dim, new, length, dtype, held8):
    """Prompts long enough for them: over 2 workgroups of 256 rows for each of 256 compute units."""
    check_large(58, [new], [length], heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, held8=held8)


def test_row_tiles_of_256_of_several_prompts():
    check_large(59, [1500, 1, 900, 0, 1300], [1500, 777, 1000, 0, 1333], heads=64, kv_heads=16, dim=64, dtype=torch.bfloat16, held8=True)


@pytest.mark.parametrize("dtype,held8,dim", [(torch.bfloat16, True, 128), (torch.float16, True, 64), (torch.bfloat16, False, 64),
                                             (torch.float16, False, 64), (torch.bfloat16, True, 112)])
@pytest.mark.parametrize("new", [1, 3, 8])
def test_two_heads_of_the_cache_a_workgroup(dtype, held8, dim, new):
    """Many sequences and a wide table, as the host's choice goes by; lengths that leave tiles of one step and of many shares."""
    lengths = [max(new, x) for x in ([4096, 1, 33, 4000, 700, 64, 129, 2500] + [3 + 61 * i % 900 for i in range(40)])]
    check_large(60, [new] * 48, lengths, heads=32, kv_heads=8, dim=dim, dtype=dtype, held8=held8, page=32, width=128)


@pytest.mark.parametrize("batch", [65, 257, 300, 600])
@pytest.mark.parametrize("news", [(1,), (1, 3, 0, 2)])
def test_many_sequences(batch, news):
    """More than a workgroup's threads: each then counts several."""
    n = [news[i % len(news)] for i in range(batch)]
    lengths = [x + 41 * i % 230 for i, x in enumerate(n)]
    check_large(61, n, lengths, heads=4, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True, page=16)


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 192])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1900, 100)])
def test_prompts_split_over_their_tokens(dtype, held8, dim, window, sinks):
    """A few rows on many tokens: five and more parts a row tile, and none for a part that a row sees nothing of."""
    check_large(62, [70], [2900], heads=4, kv_heads=2, dim=dim, dtype=dtype, held8=held8, page=32, window=window, sinks=sinks)
    check_large(63, [33, 1, 90], [2600, 500, 2700], heads=8, kv_heads=2, dim=dim, dtype=dtype, held8=held8, page=32, window=window,
                sinks=sinks)


@pytest.mark.parametrize("kv_heads", [5, 7, 13, 600])
@pytest.mark.parametrize("news,lengths", [([1, 2], [900, 40]), ([60, 1], [300, 600])])
def test_odd_and_many_heads_of_the_cache(kv_heads, news, lengths):
    """Shares that do not divide by the heads, and more heads than a workgroup each can have at once."""
    check_large(69, news, lengths, heads=2 * kv_heads, kv_heads=kv_heads, dim=16, dtype=torch.bfloat16, held8=True, page=32)
