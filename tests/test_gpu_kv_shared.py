"""Attention to a cache for sequences that share their first tokens, and the reading of a cache, on the GPU against
their statements in 64 bits.

Tolerances are those of attention by itself (tests/test_gpu_kv.py): what a row found among the shared tokens is kept in
32 bits and joined under the larger of two references, a few roundings of 2^-24 and two exponentials of 2^-22 each,
within the 2^-19 that stands there for sums and exponentials.  A value that is read is a product in 32 bits (2^-24)
rounded once: 2^-24 + u of it, and nothing where the scale is a power of two and the product a normal number of the type.
"""

from __future__ import annotations

import pytest
import torch

from oracle import kv_oracle
from tests import kv_cases
from tests.kv_cases import E4M3, half_step
from tests.test_gpu_kv import compare_attend, dev, on_gpu

pytestmark = pytest.mark.gpu


def shared_batch(g, news, lengths, groups, shared, page, spare=3):
    """starts and a table in which a group's whole shared pages stand in its first sequence's row alone."""
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    width = max(-(-n // page) for n in lengths + [1])
    pages = sum(-(-n // page) for n in lengths) + spare
    order = torch.randperm(pages, generator=g).tolist()
    table = []
    for b, n in enumerate(lengths):
        leader, common = kv_oracle.sharing(groups, shared, starts, lengths, starts[-1], width * page, b)
        from_ = common // page if leader != b else 0
        row = [-1] * from_ + [order.pop() for _ in range(from_, -(-n // page))]
        table.append(row + [-1] * (width - len(row)))
    return starts, table, pages


def poison(x, table, starts, lengths, groups, shared, page):
    """NaN wherever no row has to look: unused pages, ends of last ones, and a sequence's own copies of shared tokens."""
    keep = torch.zeros(x.shape[:2], dtype=torch.bool)
    cap = len(table[0]) * page
    for b, n in enumerate(lengths):
        leader, common = kv_oracle.sharing(groups, shared, starts, lengths, starts[-1], cap, b)
        for j in range(min(n, cap)):
            pg = table[leader if j < common else b][j // page]
            if 0 <= pg < x.shape[0]:
                keep[pg, j % page] = True
    if x.dtype == E4M3:
        x.view(torch.uint8)[~keep] = 0x7F
    else:
        x[~keep] = float("nan")


def widened(table, page, kv_heads, dim, held8):
    """The table with rows so wide (nothing is there) that reading all of them would be 256 MiB at least."""
    width = 2 ** 28 // (len(table) * kv_heads * dim * 2 * (1 if held8 else 2) * page) + 1
    return [row + [-1] * (width - len(row)) for row in table]


def check(seed, news, lengths, groups, shared, *, heads=8, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True, page=32, block=16,
          by_head=False, lse=True, tweak=None, given=None, spread=2.0, scale=None):
    """`given`: (starts, groups, shared) as the call gets them, where those are out of order."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(seed)
    starts, table, pages = shared_batch(g, news, lengths, groups, shared, page)
    k, ks, v, vs = kv_cases.pools(g, pages, page, kv_heads, dim, dtype, held8, block, by_head)
    q = (torch.randn((starts[-1], heads, dim), generator=g) * spread).to(dtype)
    if tweak:
        tweak(q=q, k=k, v=v, table=table, starts=starts, lengths=lengths, groups=groups, shared=shared)
    for x in (k, v):
        if tweak is None:
            poison(x, table, starts, lengths, groups, shared, page)
    scale = dim ** -0.5 if scale is None else scale
    want = kv_oracle.attend(q, k, v, ks, vs, table, starts, lengths, scale, fill=7.0, groups=groups, shared=shared)
    cache = kv.PagedCache(on_gpu(k), on_gpu(v), dev(ks), dev(vs))
    got = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    got_lse = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    # A call chooses its kernels by what rows of the table could hold: with wide ones groups' shared tokens go through a
    # launch of their own.  The last call finds what the others have left of the workspace.
    for t in (table, widened(table, page, kv_heads, dim, held8), table):
        got.fill_(7.0)
        r = kv.attend_shared(dev(q), cache, dev(t), dev(starts), dev(lengths), dev(groups), dev(shared), scale=scale, out=got, lse=got_lse)
        assert r is got
        compare_attend(got.cpu(), None if got_lse is None else got_lse.cpu(), *want, v, vs, dtype, held8, dim, max(lengths + [1]))
    return cache, q, table, starts, want


TYPES = [(torch.bfloat16, True), (torch.float16, True), (torch.bfloat16, False), (torch.float16, False)]


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 112, 128, 144, 192, 240, 256])
def test_single_tokens(dtype, held8, dim):
    check(1, [1] * 5, [150, 131, 133, 300, 171], [0, 5], [130], dim=dim, dtype=dtype, held8=held8)


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 192, 256])
def test_many_rows(dtype, held8, dim):
    """Over 64 rows a group and a sequence: the row tiles."""
    check(2, [75, 40, 30], [275, 250, 310], [0, 3], [195], heads=6, kv_heads=3, dim=dim, dtype=dtype, held8=held8)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (16, 1), (5, 1), (14, 2), (48, 16), (130, 1)])
@pytest.mark.parametrize("n", [1, 3, 30])
def test_shared_heads(heads, kv_heads, n):
    check(3, [n, 1, n], [n + 70, 80, 200], [0, 3], [67], heads=heads, kv_heads=kv_heads)


@pytest.mark.parametrize("shared", [1, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 127, 128, 129, 1000])
@pytest.mark.parametrize("n", [1, 20])
def test_where_the_shared_tokens_end(shared, n):
    """Anywhere in a page, a block or a step; own tokens from the new ones alone on."""
    check(4, [n, n, n, n], [shared + n, shared + n + 1, shared + n + 40, shared + n + 200], [0, 4], [shared], heads=4, kv_heads=1,
          dtype=torch.float16, held8=False)


@pytest.mark.parametrize("groups,shared", [([0, 1, 2, 3, 4, 5, 6], [30, 100, 64, 1, 99, 16]), ([0, 2, 6], [100, 40]), ([1, 5], [90]), ([2, 3, 6], [70, 60]),
                                           ([0, 6], [90]), ([0], []), ([0, 3, 3, 6], [50, 40, 60])])
@pytest.mark.parametrize("news", [[1] * 6, [3, 1, 20, 1, 1, 7]])
def test_groups(groups, shared, news):
    """Groups of one, several, none; sequences in none; a group of no sequences."""
    check(5, news, [110, 120, 130, 125, 140, 133], groups, shared, held8=True, page=16)


def test_many_groups():
    n = 150
    groups = sorted({0, n, *range(0, n, 2), *range(0, n, 7)})
    check(6, [1 + b % 3 for b in range(n)], [60 + 13 * b % 90 for b in range(n)], groups, [5 + 17 * i % 50 for i in range(len(groups) - 1)], kv_heads=1,
          heads=2, page=16)


@pytest.mark.parametrize("held8", [True, False])
def test_new_tokens_among_the_shared_ones(held8):
    """A sequence whose new tokens begin before the shared ones end looks for itself; the others do not notice."""
    check(7, [1, 50, 1, 30], [200, 140, 150, 121], [0, 4], [100], held8=held8)


def test_one_sequence_alone_and_long():
    check(8, [1], [5003], [0, 1], [4990])
    check(9, [1, 1, 2], [5003, 9000, 5010], [0, 3], [5000], heads=16, kv_heads=4, dim=128, by_head=True)


@pytest.mark.parametrize("held8", [True, False])
def test_prefix_split_over_row_tiles(held8):
    """Some hundred rows of a group and a long prefix: parts of the row tiles' tokens, joined by the sequences."""
    check(10, [1] * 70, [2100 + 3 * b for b in range(70)], [0, 70], [2077], heads=8, kv_heads=2, dim=64, held8=held8, page=64, block=32)
    check(11, [90, 1, 100], [2200, 2101, 2300], [0, 3], [2077], heads=8, kv_heads=2, dim=96, held8=held8, page=64, block=32)


@pytest.mark.parametrize("page,block", [(16, 16), (48, 16), (64, 64), (128, 32)])
@pytest.mark.parametrize("by_head", [False, True])
def test_pages(page, block, by_head):
    check(12, [2, 1, 30], [391, 290, 350], [0, 3], [260], heads=4, dim=96, dtype=torch.float16, page=page, block=block, by_head=by_head)


def test_pages_that_are_not_there():
    def drop(table, **_):
        for b, p in ((0, 1), (0, 3), (1, 8), (2, 9)):
            table[b][p] = -1
        table[0][5] = 10_000
        table[1][7] = -5
    for news in ([1, 1, 1], [40, 35, 30]):
        check(13, news, [400, 380, 395], [0, 3], [200], tweak=drop, held8=False)
        check(13, news, [400, 380, 395], [0, 3], [200], tweak=drop)


def test_no_shared_page_is_there():
    """Rows that find nothing among the shared tokens, and rows that find nothing at all."""
    def drop(table, **_):
        table[0][:6] = [-1] * 6
        table[2] = [-1] * len(table[2])
    for news in ([1, 1, 1], [40, 35, 30]):
        check(14, news, [250, 240, 244], [0, 3], [192], tweak=drop)


def test_numbers_that_are_none():
    """NaN and infinities among shared and own keys and values reach the rows that see them and no others."""
    inf = float("inf")

    def plant(k, v, table, **_):
        v[table[0][0], 3, 0, 5] = inf        # shared: all rows of the group
        v[table[1][3], 10, 1, 7] = float("nan")   # sequence 1's own
        k[table[2][3], 20, 0, 1] = float("nan")
    for news in ([1, 1, 1, 1], [40, 35, 30, 38]):
        check(15, news, [140, 138, 139, 150], [0, 3, 4], [96, 80], tweak=plant, held8=False)


def test_sequences_and_groups_out_of_order():
    from tensor_layout_amd import kv
    cache, q, table, starts, want = check(16, [1, 2, 1, 1, 2, 1], [150, 120, 130, 125, 140, 133], [0, 3, 6], [64, 96], page=32,
                                          tweak=lambda table, groups, **_: [table[b].__setitem__(i, table[a][i]) for a, e, n in ((0, 3, 2), (3, 6, 3))
                                                                            for b in range(a, e) for i in range(n)])
    lengths = [150, 120, 130, 125, 140, 133]

    wide = widened(table, 32, 2, 64, True)

    def call(groups, shared, starts=starts, lengths=lengths, table=table):
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        out = kv.attend_shared(dev(q), cache, dev(table), dev(starts), dev(lengths), dev(groups), dev(shared), out=torch.full_like(q, 7.0, device="cuda"),
                               lse=lse)
        return out.cpu(), lse.cpu()
    # Groups that are none: their sequences look for themselves, in tables that name the shared pages too.
    for groups, shared in (([0, 3, 6], [64, 0]), ([0, 3, 6], [-1, 96]), ([0, 3, 6], [1 << 30, 96]), ([-5, 3, 6], [64, 96]), ([0, 3, 100], [64, 96]),
                           ([0, 100, 6], [64, 96]), ([3, 0], [64]), ([6, 6], [64]), ([-3, -1], [64])):
        for t in (table, wide):
            got, lse = call(groups, shared, table=t)
            compare_attend(got, lse, *want, cache.v.cpu(), cache.v_scale.cpu(), torch.bfloat16, True, 64, 150)
    # Skipped sequences: rows stay as they were, the others are served.
    for bad_starts, bad_lengths, skipped in ((starts, [150, 1, 130, 125, 140, 133], [1]), (starts, [0, 120, 130, 125, 140, 133], [0]),
                                             (starts, [150, 120, 130, 125, 140, -7], [5]), ([0, 1, -9, 4, 5, 7, 8], lengths, [1, 2]),
                                             ([0, 1, 3, 99, 5, 7, 8], lengths, [2, 3]), ([-1, 1, 3, 4, 5, 7, 8], lengths, [0])):
        for t in (table, wide):
            got, lse = call([0, 3, 6], [64, 96], bad_starts, bad_lengths, t)
            for b in range(6):
                rows = slice(starts[b], starts[b + 1])
                if b in skipped:
                    assert bool((got[rows] == 7).all()) and bool((lse[rows] == 7).all())
                else:
                    compare_attend(got[rows], lse[rows], *(x[rows] for x in want), cache.v.cpu(), cache.v_scale.cpu(), torch.bfloat16, True, 64, 150)


def test_rows_of_no_sequence():
    from tensor_layout_amd import kv
    cache, q, table, starts, want = check(17, [1, 1, 1], [100, 90, 95], [0, 3], [64])
    wide = torch.cat([q, q, q])
    for tokens, t in ((4, table), (9, table), (4, widened(table, 32, 2, 64, True))):
        out = torch.full((tokens, *q.shape[1:]), 7.0, dtype=q.dtype, device="cuda")
        kv.attend_shared(dev(wide[:tokens]), cache, dev(t), dev(starts), dev([100, 90, 95]), dev([0, 3]), dev([64]), out=out)
        assert bool((out[3:] == 7).all())
        compare_attend(out[:3].cpu(), None, *want, cache.v.cpu(), cache.v_scale.cpu(), torch.bfloat16, True, 64, 100)


@pytest.mark.parametrize("wide", [False, True])
def test_strides_streams_and_a_graph(wide):
    """Heads and rows apart, a named stream beside another's calls, and a captured call replayed on new numbers."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(18)
    page, dim = 32, 64
    groups, cases = [0, 4, 6], []
    for news, lengths, shared in (([1] * 6, [150, 140, 145, 139, 133, 170], [130, 100]), ([1] * 6, [170, 141, 160, 139, 133, 120], [96, 107]),
                                  ([1] * 6, [150, 140, 99, 139, 133, 170], [100, 133])):
        starts, table, pages = shared_batch(g, news, [170] * 6, groups, [0, 0], page)
        cases.append((starts, widened(table, page, 2, dim, True) if wide else table, lengths, shared))
    pages = 6 * 6 + 3
    k, ks, v, vs = kv_cases.pools(g, pages, page, 2, dim, torch.bfloat16, True, 16, False)
    cache = kv.PagedCache(dev(k), dev(v), dev(ks), dev(vs))
    q = torch.randn((6, 8, dim), generator=g).to(torch.bfloat16)
    big = torch.zeros((6, 16, 2 * dim), dtype=q.dtype, device="cuda")
    big[:, ::2, :dim] = q.cuda()
    qs = big[:, ::2, :dim]
    out = torch.empty((8, 6, dim), dtype=q.dtype, device="cuda").transpose(0, 1)
    ints = [dev(x) for x in (cases[0][1], cases[0][0], cases[0][2], groups, cases[0][3])]

    def want(i):
        starts, table, lengths, shared = cases[i]
        return kv_oracle.attend(q, k, v, ks, vs, table, starts, lengths, dim ** -0.5, groups=groups, shared=shared)
    kv.attend_shared(qs, cache, *ints, out=out)
    compare_attend(out.cpu(), None, *want(0), v, vs, torch.bfloat16, True, dim, 170)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = kv.attend_shared(qs, cache, *ints, stream=side.cuda_stream)
    kv.attend_shared(qs, cache, *ints, out=out)
    torch.cuda.synchronize()
    assert torch.equal(other, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.attend_shared(qs, cache, *ints, out=out)
    for i in (1, 2, 0, 1):
        for t, x in zip(ints, (cases[i][1], cases[i][0], cases[i][2], groups, cases[i][3])):
            t.copy_(dev(x))
        out.zero_()
        graph.replay()
        eager = kv.attend_shared(qs, cache, *ints)
        torch.cuda.synchronize()
        compare_attend(out.cpu(), None, *want(i), v, vs, torch.bfloat16, True, dim, 170)
        assert torch.equal(eager, out)


def test_it_gives_what_attend_gives_in_turn_with_it():
    """One workspace for both, and a table that names the shared pages in every row."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(19)
    starts, lengths, table, pages = kv_cases.batch(g, [1] * 12, [1000 + 9 * b for b in range(12)], 32)
    for b in range(12):
        table[b][:31] = table[0][:31]
    k, ks, v, vs = kv_cases.pools(g, pages, 32, 4, 128, torch.float16, True, 16, False)
    cache = kv.PagedCache(dev(k), dev(v), dev(ks), dev(vs))
    q = dev((torch.randn((12, 16, 128), generator=g) * 2).half())
    args = (q, cache, dev(table), dev(starts), dev(lengths))
    want = kv_oracle.attend(q.cpu(), k, v, ks, vs, table, starts, lengths, 128 ** -0.5)
    wide = (*args[:2], dev(widened(table, 32, 4, 128, True)), *args[3:])
    for _ in range(3):
        for got in (kv.attend(*args), kv.attend_shared(*args, dev([0, 12]), dev([992])), kv.attend_shared(*wide, dev([0, 12]), dev([992]))):
            compare_attend(got.cpu(), None, *want, v, vs, torch.float16, True, 128, 1100)


def far_pool(pages, page, heads, dim):
    """Storage whose last pages lie beyond 2^32 bytes and 2^31 elements, of which only what is used is written."""
    return torch.empty((pages, page, heads, dim), dtype=torch.bfloat16, device="cuda")


def test_pages_far_apart():
    """Offsets past 32 bits: attention in both ways, reading."""
    from tensor_layout_amd import kv
    pages, page, heads, dim = 600_000, 16, 1, 256   # 2.5 * 10^9 elements
    g = torch.Generator().manual_seed(29)
    used = [599_999, 3, 599_000, 300_001, 1, 598_765, 400_000, 2, 599_998]
    near = [torch.randn((len(used), page, heads, dim), generator=g).to(torch.bfloat16) for _ in range(2)]
    pools = [far_pool(pages, page, heads, dim) for _ in range(2)]
    where = torch.tensor(used, device="cuda")
    for pool, x in zip(pools, near):
        pool[where] = x.cuda()
    cache = kv.PagedCache(*pools)
    lengths, starts = [70, 75, 100], [0, 1, 2, 42]
    table = [[0, 1, 2, 3, 4, -1, -1], [-1, -1, -1, 5, 6, -1, -1], [-1, -1, -1, 7, 8, 6, 5]]
    there = [[used[x] if x >= 0 else -1 for x in row] for row in table]
    q = torch.randn((42, 4, dim), generator=g).to(torch.bfloat16)
    want = kv_oracle.attend(q, near[0], near[1], None, None, table, starts, lengths, dim ** -0.5, groups=[0, 3], shared=[48])
    for t in (there, widened(there, page, heads, dim, False)):
        lse = torch.empty((42, 4), device="cuda")
        got = kv.attend_shared(dev(q), cache, dev(t), dev(starts), dev(lengths), dev([0, 3]), dev([48]), lse=lse)
        compare_attend(got.cpu(), lse.cpu(), *want, near[1], None, torch.bfloat16, False, dim, 100)
    rows = [torch.empty((42, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kv.read(cache, dev(there), dev(starts), dev(lengths), *rows)
    for x, pool in zip(rows, near):
        assert torch.equal(x.cpu().double(), kv_oracle.read(pool, None, table, starts, lengths, 42, 0.0))


def test_many_sequences_of_one_group():
    """More than the 256 that a workgroup counts a thread each."""
    n = 300
    check(30, [1] * n, [70 + 7 * b % 60 for b in range(n)], [0, n], [64], heads=4, kv_heads=1, page=16)
    check(31, [1 + b % 2 for b in range(n)], [70 + 7 * b % 60 for b in range(n)], [0, 100, 101, 290], [64, 30, 50], heads=2, kv_heads=2, page=16, held8=False)


@pytest.mark.parametrize("n", [40, 100, 300])
def test_own_tokens_of_several_tiles_a_workgroup(n):
    """16 heads leave fewer workgroups a head than there are sequences: each takes several whole tiles, of unequal lengths,
    some of no rows; then with one long sequence among them equal parts of all steps."""
    news = [0 if b % 11 == 5 else 1 + (b % 7 == 3) * 20 for b in range(n)]
    own = [1 + 23 * b % 200 for b in range(n)]
    check(32, news, [64 + a + b for a, b in zip(own, news)], [0, n], [64], heads=16, kv_heads=16, dim=16, page=16)
    own[n // 2] = 2500
    check(33, news, [64 + a + b for a, b in zip(own, news)], [0, n // 3, n], [64, 50], heads=16, kv_heads=16, dim=16, page=16, held8=False)


# ---------------------------------------------------------------- reading


def check_read(seed, news, lengths, *, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True, page=32, block=16, by_head=False, drop=(),
               width=None, odd_scales=False, strided=False, which="kv", starts_=None):
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(seed)
    starts, lengths, table, pages = kv_cases.batch(g, news, lengths, page, drop=drop, width=width)
    tokens = starts[-1]
    starts = starts if starts_ is None else starts_
    k, ks, v, vs = kv_cases.pools(g, pages, page, kv_heads, dim, dtype, held8, block, by_head)
    if odd_scales:
        ks, vs = ks * (1 + torch.rand(ks.shape, generator=g)), vs * (1 + torch.rand(vs.shape, generator=g))
    cache = kv.PagedCache(on_gpu(k), on_gpu(v), dev(ks), dev(vs))
    if strided:
        big = torch.full((kv_heads, 2, tokens, dim + 16), 7.0, dtype=dtype, device="cuda")
        outs = [big[:, i, :, 8:8 + dim].transpose(0, 1) for i in range(2)]
    else:
        outs = [torch.full((tokens, kv_heads, dim), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    kv.read(cache, dev(table), dev(starts), dev(lengths), outs[0] if "k" in which else None, outs[1] if "v" in which else None)
    for name, pool, scale, got in (("k", k, ks, outs[0]), ("v", v, vs, outs[1])):
        want = kv_oracle.read(pool, scale, table, starts, lengths, tokens, 7.0) if name in which else torch.full(got.shape, 7.0).double()
        got = got.cpu().double()
        if odd_scales:
            assert bool(((got - want).abs() <= (2.0 ** -24 + half_step(dtype) * (1 + 2.0 ** -23)) * want.abs() + 2.0 ** -25 * (dtype == torch.float16)).all())
        else:
            assert torch.equal(got, want.to(dtype).double())
    if strided:
        assert bool((big[..., :8] == 7).all()) and bool((big[..., 8 + dim:] == 7).all())


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 112, 128, 192, 256])
def test_read(dtype, held8, dim):
    check_read(20, [1, 40, 33, 90], [1, 77, 33, 500], dim=dim, dtype=dtype, held8=held8)


@pytest.mark.parametrize("news,lengths", [([1], [1]), ([1], [2049]), ([0, 1, 0], [5, 6, 0]), ([700, 1, 300], [700, 5, 444]),
                                          ([1] * 300, [1 + 13 * b % 190 for b in range(300)]), ([3, 0, 0, 5], [9, 0, 3, 5])])
def test_read_batches(news, lengths):
    check_read(21, news, lengths, kv_heads=3)


@pytest.mark.parametrize("page,block", [(16, 16), (48, 16), (64, 64), (96, 48)])
@pytest.mark.parametrize("by_head", [False, True])
@pytest.mark.parametrize("kv_heads", [1, 5, 16])
def test_read_pages(page, block, by_head, kv_heads):
    check_read(22, [100, 7], [391, 190], page=page, block=block, by_head=by_head, kv_heads=kv_heads, dtype=torch.float16, strided=True)


def test_read_rounds_once_under_any_scale():
    for dtype in (torch.bfloat16, torch.float16):
        check_read(23, [60, 20], [200, 100], odd_scales=True, dtype=dtype)


@pytest.mark.parametrize("which", ["k", "v"])
def test_read_one_of_both(which):
    check_read(24, [60, 20], [200, 100], which=which)


def test_read_pages_that_are_not_there_and_sequences_out_of_order():
    check_read(25, [120, 200], [150, 300], drop=[(0, 2), (1, 5), (1, 9)])
    check_read(26, [120, 200], [150, 300], width=6)
    check_read(27, [4, 5, 6], [50, 60, 70], starts_=[0, 4, -3, 15])
    check_read(27, [4, 5, 6], [50, 60, 70], starts_=[0, 4, 99, 15])
    check_read(27, [4, 5, 6], [50, 3, 70])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_what_append_wrote_comes_back_and_can_be_written_again(dtype):
    """read gives append's rows back, rounded to e4m3 under their block's scale; written into another sequence they are
    the same (a power of two divides them without rounding), also from the middle of a page on."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(28)
    pages, page, heads, dim = 12, 32, 3, 96
    pools = [torch.zeros((pages, page, heads, dim), device="cuda").to(E4M3) for _ in range(2)]
    scales = [torch.ones((pages, heads, 2), device="cuda") for _ in range(2)]
    cache = kv.PagedCache(*pools, *scales)
    k, v = (dev(torch.randn((100, heads, dim), generator=g).to(dtype)) for _ in range(2))
    table = dev([[3, 7, 1, 9], [3, 7, 1, 5]])
    kv.append(cache, k, v, table[:1], dev([0, 100]), dev([100]))
    got = [torch.zeros_like(k), torch.zeros_like(v)]
    kv.read(cache, table[:1], dev([0, 100]), dev([100]), *got)
    for x, y in zip(got, (k, v)):   # e4m3: half a step of the value, or of its smallest normal's step under the block's scale
        amax = y.float().abs().amax().item()
        assert bool(((x.float() - y.float()).abs() <= y.float().abs() * half_step(E4M3) + amax / 224 * 2.0 ** -10).all())
    # The second sequence takes the first's last four tokens into a page of its own.
    part = [torch.zeros_like(k[:4]), torch.zeros_like(v[:4])]
    kv.read(cache, table[:1], dev([0, 4]), dev([100]), *part)
    kv.append(cache, *part, table[1:], dev([0, 4]), dev([100]))
    again = [torch.zeros_like(k), torch.zeros_like(v)]
    kv.read(cache, table[1:], dev([0, 100]), dev([100]), *again)
    for x, y in zip(got, again):
        assert torch.equal(x, y)
