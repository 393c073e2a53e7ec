"""The paged key/value cache operators on the GPU against their statement in 64 bits.

Tolerances.  A rounding to a type errs by at most half a step u of the value.

* A score in 32 bits: dim products summed, each addition rounding by 2^-24 of
  at most S = sum |scale q k|, then two more roundings (the factor and the
  reference): E = (dim + 8) 2^-24 S.  A weight is off by a factor e^E twice
  (itself and in the sum), and by 2^-20 for the exponential and the sum.
* A weight is rounded once for the product with the values (u of the product's
  type; two bf16 numbers together keep 16 bits), in fp16 by 2^-25 at least of
  the largest weight.  So an output is off by at most
  (2 (e^E - 1) + u_w + 2^-19) A + n 2^-25 max|v| + u |out| with A = sum |weight * value|.
* lse: E + 2^-20 + 2^-22 |lse|.
* A rotated channel: two products and their sum, cosine and sine rounded:
  4 * 2^-24 (|a| + |b|), then u.
"""

from __future__ import annotations

import math

import pytest
import torch

from oracle import kv_oracle
from tests import kv_cases
from tests.kv_cases import E4M3, half_step

pytestmark = pytest.mark.gpu


def dev(x):
    return None if x is None else x.cuda() if isinstance(x, torch.Tensor) else torch.tensor(x, dtype=torch.int32).cuda()


def on_gpu(pool):
    """The pool on the GPU with its order in memory."""
    if pool.stride(2) > pool.stride(1):
        return pool.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    return pool.contiguous().cuda()


def check_attend(seed, news, lengths, *, heads, kv_heads, dim, dtype, held8, page=32, block=16, window=0, sinks=0,
                 by_head=False, drop=(), scale=None, width=None, spread=2.0, tweak=None, lse=True):
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(seed)
    starts, lengths, table, pages = kv_cases.batch(g, news, lengths, page, drop=drop, width=width)
    k, ks, v, vs = kv_cases.pools(g, pages, page, kv_heads, dim, dtype, held8, block, by_head)
    for x in (k, v):
        kv_cases.poison(x, table, lengths, page)
    q = (torch.randn((starts[-1], heads, dim), generator=g) * spread).to(dtype)
    if tweak:
        tweak(q=q, k=k, v=v, table=table, starts=starts, lengths=lengths)
    scale = dim ** -0.5 if scale is None else scale
    out, want_lse, size, score = kv_oracle.attend(q, k, v, ks, vs, table, starts, lengths, scale, window, sinks, fill=7.0)
    cache = kv.PagedCache(on_gpu(k), on_gpu(v), dev(ks), dev(vs))
    got = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    got_lse = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    r = kv.attend(dev(q), cache, dev(table), dev(starts), dev(lengths), scale=scale, window=window, sinks=sinks, out=got,
                  lse=got_lse)
    assert r is got
    compare_attend(got.cpu(), None if got_lse is None else got_lse.cpu(), out, want_lse, size, score, v, vs, dtype, held8, dim,
                   max(lengths + [1]))


def compare_attend(got, got_lse, out, want_lse, size, score, v, vs, dtype, held8, dim, n):
    err = (dim + 8) * 2.0 ** -24 * score
    u_w = half_step(torch.bfloat16) if held8 and dtype == torch.bfloat16 else 2.0 ** -16 if held8 else half_step(dtype)
    vmax = kv_oracle.values(v, vs)
    vmax = float(vmax[vmax.isfinite()].abs().max())
    small = 0.0 if held8 or dtype == torch.bfloat16 else n * 2.0 ** -25 * vmax
    tol = (2 * torch.expm1(err)[..., None] + u_w + 2.0 ** -19) * size + small + half_step(dtype) * out.abs() + 1e-30
    bad = ~((got.double() - out).abs() <= tol) & ~(got.isnan() & out.isnan()) & (got.double() != out)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got.double() - out).abs() - tol).nan_to_num().max()))
    if got_lse is not None:
        same = got_lse.double() == want_lse
        off = (got_lse.double() - want_lse).abs() <= err + 2.0 ** -20 + 2.0 ** -22 * want_lse.abs()
        assert bool((same | off | (got_lse.isnan() & want_lse.isnan())).all())


TYPES = [(torch.bfloat16, True), (torch.float16, True), (torch.bfloat16, False), (torch.float16, False)]


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 112, 128, 192, 256])
def test_decode(dtype, held8, dim):
    check_attend(1, [1] * 5, [1, 17, 33, 150, 700], heads=8, kv_heads=2, dim=dim, dtype=dtype, held8=held8)


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 192, 256])
def test_prompt(dtype, held8, dim):
    check_attend(2, [75], [203], heads=6, kv_heads=3, dim=dim, dtype=dtype, held8=held8)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (16, 1), (5, 1), (14, 2), (48, 16), (130, 1)])
@pytest.mark.parametrize("n", [1, 3, 30, 130])
def test_shared_heads(heads, kv_heads, n):
    check_attend(3, [n, 1], [n + 70, 40], heads=heads, kv_heads=kv_heads, dim=64, dtype=torch.bfloat16, held8=True)


@pytest.mark.parametrize("news,lengths", [
    ([1], [1]), ([1], [2049]), ([2, 3, 1, 4], [2, 77, 500, 4]), ([0, 1, 0], [5, 6, 0]), ([17, 33], [17, 1000]),
    ([200, 1, 1, 90], [300, 40, 511, 90]), ([1] * 70, [1 + 13 * i % 190 for i in range(70)])])
@pytest.mark.parametrize("held8", [True, False])
def test_batches(news, lengths, held8):
    check_attend(4, news, lengths, heads=8, kv_heads=2, dim=128, dtype=torch.bfloat16, held8=held8, page=16)


@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (48, 16), (64, 64), (128, 32), (96, 48)])
@pytest.mark.parametrize("by_head", [False, True])
@pytest.mark.parametrize("n", [1, 90])
def test_pages(page, block, by_head, n):
    check_attend(5, [n, 1], [391, 190], heads=4, kv_heads=2, dim=96, dtype=torch.float16, held8=True, page=page, block=block,
                 by_head=by_head)


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (33, 4), (100, 65), (1000, 4), (64, 1000), (5, 16)])
@pytest.mark.parametrize("news", [[1, 1, 1], [5, 2, 7], [90, 70, 1]])
def test_window(window, sinks, news):
    check_attend(6, news, [400, 75, 210], heads=8, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True, window=window,
                 sinks=sinks)


@pytest.mark.parametrize("news", [[1, 1, 3], [80, 70, 70]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_pages_that_are_not_there(news, window, sinks):
    """Missing pages anywhere, among them all that a row sees; entries over the pool; a table that is too narrow."""
    def over(table, **_):
        table[0][5] = 10_000
        table[2] = [-1] * len(table[2])
    check_attend(7, news, [400, 500, 100], heads=4, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=False,
                 drop=[(0, 0), (0, 3), (1, 1), (1, 11)], window=window, sinks=sinks, tweak=over)
    check_attend(8, news, [400, 500, 100], heads=4, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True, width=7,
                 window=window, sinks=sinks)


def test_sequences_out_of_order_are_skipped():
    def shuffle(starts, lengths, **_):
        starts[1], lengths[3] = 100, 1   # rows past the end; more new tokens than tokens
    check_attend(9, [2, 2, 2, 2, 2], [50, 60, 70, 80, 90], heads=4, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True,
                 tweak=shuffle)


@pytest.mark.parametrize("news", [[1, 1], [3, 70]])
@pytest.mark.parametrize("held8", [True, False])
def test_large_scores(news, held8):
    """Scores far apart and far from zero: references that move, weights that vanish."""
    check_attend(10, news, [300, 200], heads=4, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=held8, spread=60.0)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("n", [1, 4, 90])
def test_values_that_are_no_numbers(value, n):
    """In a row's own sight they show, in a head's other channels and in other sequences they do not."""
    def put(k, v, table, **_):
        v[table[0][0], 3, 0, 5] = value
        k[table[1][0], 2, 1, 0] = math.nan
    check_attend(11, [n, n], [120, 150], heads=4, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=False, tweak=put)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("n", [5, 30, 90])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 2)])
@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 80), (torch.float16, 128)])
def test_values_that_are_no_numbers_beside_rows_that_do_not_see_them(value, n, window, sinks, dtype, dim):
    """Tokens among the new ones: the rows before them, and those whose window has left them, stay as they are."""
    def put(k, v, table, lengths, **_):
        for b, back, h, c in ((0, 2, 0, 5), (0, n - 1, 1, dim - 1), (1, n // 2, 1, 0), (1, n // 2, 1, 17)):
            j = lengths[b] - back
            v[table[b][j // 32], j % 32, h, c] = value
    check_attend(33, [n, n], [120, 150], heads=4, kv_heads=2, dim=dim, dtype=dtype, held8=False, tweak=put, window=window,
                 sinks=sinks)
    if math.isnan(value):
        check_attend(34, [n, n], [120, 150], heads=4, kv_heads=2, dim=dim, dtype=dtype, held8=True, tweak=put, window=window,
                     sinks=sinks)


def test_scales_that_are_no_powers_of_two():
    """Another writer's scales, among them one under the smallest normal number."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(35)
    for n in (1, 6, 90):
        starts, lengths, table, pages = kv_cases.batch(g, [n, 1], [300, 75], 32)
        k, ks, v, vs = kv_cases.pools(g, pages, 32, 2, 64, torch.float16, True, 16, False)
        ks, vs = ks * (1 + torch.rand(ks.shape, generator=g)), vs * (1 + torch.rand(vs.shape, generator=g))
        vs[table[0][1], 0, 0] = 2.0 ** -126
        q = torch.randn((n + 1, 4, 64), generator=g).half()
        want = kv_oracle.attend(q, k, v, ks, vs, table, starts, lengths, 0.125)
        got, lse = torch.empty_like(q, device="cuda"), torch.empty((n + 1, 4), device="cuda")
        kv.attend(dev(q), kv.PagedCache(on_gpu(k), on_gpu(v), dev(ks), dev(vs)), dev(table), dev(starts), dev(lengths),
                  scale=0.125, out=got, lse=lse)
        compare_attend(got.cpu(), lse.cpu(), *want, v, vs, torch.float16, True, 64, 300)


def test_strides():
    """q and out as parts of wider tensors, lse by heads, a table row inside a wider table."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(12)
    starts, lengths, table, pages = kv_cases.batch(g, [1, 70], [90, 130], 16)
    k, ks, v, vs = kv_cases.pools(g, pages, 16, 2, 64, torch.bfloat16, True, 16, False)
    wide = torch.randn((71, 8 + 4, 64), generator=g).to(torch.bfloat16)
    out, lse, size, score = kv_oracle.attend(wide[:, :8], k, v, ks, vs, table, starts, lengths, 0.125)
    cache = kv.PagedCache(on_gpu(k), on_gpu(v), dev(ks), dev(vs))
    big = torch.full((71, 10, 80), 3.0, dtype=torch.bfloat16, device="cuda")
    glse = torch.empty((8, 71), device="cuda").t()
    gt = torch.full((2, 40), 5, dtype=torch.int32, device="cuda")
    gt[:, :len(table[0])] = dev(table)
    kv.attend(dev(wide)[:, :8], cache, gt[:, :len(table[0])], dev(starts), dev(lengths), scale=0.125, out=big[:, 1:9, :64],
              lse=glse)
    compare_attend(big[:, 1:9, :64].cpu(), glse.cpu(), out, lse, size, score, v, vs, torch.bfloat16, True, 64, 130)
    assert bool((big[:, 0] == 3).all() and (big[:, 9] == 3).all() and (big[:, :, 64:] == 3).all())


def test_far_pages():
    """Page offsets past 2^31 elements."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(13)
    page, kv_heads, dim = 64, 4, 128
    pages = (1 << 31) // (page * kv_heads * dim) + 40
    k, ks, v, vs = kv_cases.pools(g, 16, page, kv_heads, dim, torch.bfloat16, True, 64, False)
    big = []
    at = [pages - 1 - 3 * i for i in range(16)]
    for x in (k, v):
        y = torch.zeros((pages, page, kv_heads, dim), dtype=torch.uint8, device="cuda")
        y[at] = x.view(torch.uint8).cuda()
        big.append(y.view(E4M3))
    sc = []
    for x in (ks, vs):
        y = torch.zeros((pages, kv_heads, 1), device="cuda")
        y[at] = x.cuda()
        sc.append(y)
    for n in (1, 70):
        starts, lengths, table = [0, n], [1000], [list(range(16))]
        q = torch.randn((n, 8, dim), generator=g).to(torch.bfloat16)
        out, lse, size, score = kv_oracle.attend(q, k, v, ks, vs, table, starts, lengths, 0.1)
        got, glse = torch.empty_like(q, device="cuda"), torch.empty((n, 8), device="cuda")
        kv.attend(dev(q), kv.PagedCache(*big, *sc), dev([[at[i] for i in range(16)]]), dev(starts), dev(lengths), scale=0.1,
                  out=got, lse=glse)
        compare_attend(got.cpu(), glse.cpu(), out, lse, size, score, v, vs, torch.bfloat16, True, dim, 1000)


# ---------------------------------------------------------------- append


def check_append(seed, news, lengths, *, heads, kv_heads, dim, dtype, held8, rot=None, interleaved=False, sections=None,
                 far=None, page=32, block=16, by_head=False, drop=(), width=None, tweak=None, in_place=False, old=None):
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(seed)
    starts, lengths, table, pages = kv_cases.batch(g, news, lengths, page, drop=drop, width=width)
    k_pool, ks, v_pool, vs = kv_cases.pools(g, pages, page, kv_heads, dim, dtype, held8, block, by_head)
    if old is not None:
        ks, vs = torch.full_like(ks, old), torch.full_like(vs, old)
    tokens = starts[-1]
    k = (torch.randn((tokens, kv_heads, dim), generator=g) * torch.exp(torch.randn((1, kv_heads, dim), generator=g))).to(dtype)
    v = torch.randn((tokens, kv_heads, dim), generator=g).to(dtype)
    q = torch.randn((tokens, heads, dim), generator=g).to(dtype)
    if tweak:
        tweak(k=k, v=v, q=q, table=table, starts=starts, lengths=lengths)
    rot = dim if rot is None else rot
    inv_freq = (10_000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None
    positions = None
    if far is not None:
        axes = len(sections) if sections else 1
        positions = torch.randint(0, far + 1, (axes, tokens), generator=g).to(torch.int32)
    want = kv_oracle.append(q, k, v, k_pool, v_pool, ks, vs, table, starts, lengths, inv_freq,
                            None if positions is None else positions.tolist(), sections, interleaved)
    gk, gv, gks, gvs = on_gpu(k_pool), on_gpu(v_pool), dev(ks), dev(vs)
    cache = kv.PagedCache(gk, gv, gks, gvs)
    gq = dev(q)
    q_out = kv.append(cache, dev(k), dev(v), dev(table), dev(starts), dev(lengths), q=gq, q_out=gq if in_place else None,
                      inv_freq=dev(inv_freq), positions=dev(positions), sections=sections, interleaved=interleaved)
    rows = torch.zeros(tokens, dtype=torch.bool)
    for b in range(len(lengths)):
        r0, n, _ = kv_oracle.ordered(starts, lengths, tokens, b)
        rows[r0:r0 + n] = True
    u = half_step(dtype)

    def near(x, y, amount, small=0.0):
        ok = ((x.double() - y).abs() <= amount + small) | (~y.isfinite() & x.isnan()) | (x.double() == y)
        assert bool(ok.all()), (int((~ok).sum()), (~ok).nonzero()[:4].tolist(), x[~ok][:4].tolist(), y[~ok][:4].tolist())

    tiny = torch.finfo(dtype).smallest_normal * half_step(dtype) * 2
    slack = 2.0 ** -22
    near(q_out.cpu()[rows], want[0][rows], u * want[0][rows].abs() + slack * q.double().abs().amax() , tiny)
    for i, (x, pool, scale, gx, gs) in enumerate(((k, k_pool, ks, gk, gks), (v, v_pool, vs, gv, gvs))):
        y, sc = want[1 + 2 * i], want[2 + 2 * i]
        touched = want[5][:, :, None, None].expand_as(y)
        if not held8:
            near(gx.cpu()[touched], y[touched], u * y[touched].abs() + slack * x[x.isfinite()].double().abs().amax(), tiny)
            assert torch.equal(gx.cpu()[~touched].view(torch.int16), pool[~touched].view(torch.int16))
            continue
        assert torch.equal(gs.cpu().double(), sc)
        h = gx.cpu().float()
        near(h[touched], y[touched], (2.0 ** -4 + slack) * y[touched].abs(), 2.0 ** -10 + slack * 448)
        assert torch.equal(gx.cpu().view(torch.uint8)[~touched], pool.view(torch.uint8)[~touched])
    return q_out, gk, gv, gks, gvs


@pytest.mark.parametrize("dtype,held8", TYPES)
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (64, 32, True), (80, 40, False), (96, 96, True), (112, 56, False),
                                                 (128, 128, False), (192, 64, False), (256, 256, False), (16, 2, False),
                                                 (128, 36, False), (128, 6, True), (128, 0, False)])
def test_append(dtype, held8, dim, rot, interleaved):
    check_append(21, [1, 20, 37, 1], [1, 45, 37, 64], heads=6, kv_heads=2, dim=dim, dtype=dtype, held8=held8, rot=rot,
                 interleaved=interleaved)


@pytest.mark.parametrize("news,lengths", [([1], [1]), ([1], [16]), ([1], [17]), ([0, 3, 0, 1], [4, 3, 0, 9]), ([300], [317]),
                                          ([1] * 90, [1 + 7 * i % 50 for i in range(90)]), ([40, 1, 200], [40, 33, 333])])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 64), (96, 48)])
def test_append_batches(news, lengths, page, block):
    for held8 in (True, False):
        check_append(22, news, lengths, heads=3, kv_heads=3, dim=64, dtype=torch.bfloat16, held8=held8, page=page, block=block,
                     by_head=held8, in_place=True)


@pytest.mark.parametrize("sections", [None, (8, 12, 12), (0, 32), (32, 0), (1, 2, 3, 26)])
@pytest.mark.parametrize("far", [100, 30_000, 2_000_000_000])
def test_far_positions(sections, far):
    """The angle in 64 bits: at two thousand million the phase is still right."""
    check_append(23, [3, 20], [40, 25], heads=4, kv_heads=2, dim=64, dtype=torch.float16, held8=False, sections=sections, far=far)
    check_append(23, [3, 20], [40, 25], heads=4, kv_heads=2, dim=64, dtype=torch.float16, held8=True, sections=sections, far=far)


@pytest.mark.parametrize("old", [2.0 ** -30, 2.0 ** 20, 0.0123, 2.0 ** -7])
def test_scale_of_a_block_that_holds_tokens(old):
    """It grows or stays; a scale that is no power of two stays as another writer set it."""
    check_append(24, [1, 3, 9], [6, 20, 16], heads=2, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True, old=old)


def test_append_values_at_the_borders():
    """Zeros, a block's largest at 448 times a power of two exactly and one step over, infinities and NaN."""
    def put(v, **_):
        v[0] = 0.0
        v[1] = 0.0
        v[1, 0, 3] = 448.0
        v[17, 0, 3] = 450.0
        v[40, 0, 1] = math.inf
        v[41, 0, 2] = math.nan
        v[42, 1] = -math.inf
        v[60] = 1e-38
        v[70, :, 0] = 3e38
    check_append(25, [1] + [16] * 5, [16] + [16] * 5, heads=2, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True, tweak=put,
                 rot=0)


def test_append_to_pages_that_are_not_there():
    def over(table, **_):
        table[1][1] = 4000
    for held8 in (True, False):
        check_append(26, [70, 80], [80, 90], heads=2, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=held8, drop=[(0, 1)],
                     tweak=over)
        check_append(27, [70, 80], [80, 90], heads=2, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=held8, width=2)


def test_append_out_of_order():
    def shuffle(starts, lengths, **_):
        starts[1], lengths[3] = 100, 1
    check_append(28, [2] * 5, [50, 60, 70, 80, 90], heads=2, kv_heads=2, dim=64, dtype=torch.bfloat16, held8=True, tweak=shuffle)


def test_append_strides():
    """k, v and q as views of one fused projection."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(29)
    starts, lengths, table, pages = kv_cases.batch(g, [5, 30], [9, 30], 16)
    pool, _, vpool, _ = kv_cases.pools(g, pages, 16, 2, 64, torch.bfloat16, False, 16, False)
    fused = torch.randn((35, 4 + 2 + 2, 64), generator=g).to(torch.bfloat16)
    inv = torch.rand((32,), generator=g)
    want = kv_oracle.append(fused[:, :4], fused[:, 4:6], fused[:, 6:], pool, vpool, None, None, table, starts, lengths, inv)
    gk, gv, f = dev(pool), dev(vpool), dev(fused)
    q = kv.append(kv.PagedCache(gk, gv), f[:, 4:6], f[:, 6:], dev(table), dev(starts), dev(lengths), q=f[:, :4], inv_freq=dev(inv))
    u = half_step(torch.bfloat16)
    for x, y in ((q, want[0]), (gk, want[1]), (gv, want[3])):
        assert bool(((x.cpu().double() - y).abs() <= u * y.abs() + 2.0 ** -20).all())


# ---------------------------------------------------------------- streams and graphs


def test_two_streams_and_a_graph():
    """One captured step (append, then attend) replayed on new lengths, and eager calls on two streams between."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(31)
    page, kv_heads, heads, dim, batch = 16, 2, 8, 64, 3
    starts, lengths, table, pages = kv_cases.batch(g, [1] * batch, [600, 90, 300], page)
    k, ks, v, vs = kv_cases.pools(g, pages, page, kv_heads, dim, torch.bfloat16, True, 16, False)
    inv = dev((10_000.0 ** (-torch.arange(0, dim, 2) / dim)).float())
    gt, gs, gl = dev(table), dev(starts), dev([500, 60, 200])
    new = [torch.randn((batch, n, dim), generator=g).to(torch.bfloat16).cuda() for n in (kv_heads, kv_heads, heads)]

    def caches():
        return kv.PagedCache(on_gpu(k), on_gpu(v), dev(ks), dev(vs))

    def step(c, q_out, out):
        kv.append(c, new[0], new[1], gt, gs, gl, q=new[2], q_out=q_out, inv_freq=inv)
        kv.attend(q_out, c, gt, gs, gl, out=out)

    a, b = caches(), caches()
    bufs = [torch.empty_like(new[2]) for _ in range(4)]
    step(caches(), bufs[0], bufs[1])   # loads what there is to load
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, bufs[0], bufs[1])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        gl += 1
        for x in new:
            x.copy_(torch.randn(x.shape, generator=g))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            step(b, bufs[2], bufs[3])
        torch.cuda.synchronize()
        for x, y in ((a.k, b.k), (a.v, b.v)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert torch.equal(a.k_scale, b.k_scale) and torch.equal(bufs[0], bufs[2]) and torch.equal(bufs[1], bufs[3])
        want = kv_oracle.attend(bufs[2].cpu(), b.k.cpu(), b.v.cpu(), b.k_scale.cpu(), b.v_scale.cpu(), table, starts,
                                gl.tolist(), dim ** -0.5)
        compare_attend(bufs[1].cpu(), None, *want, b.v.cpu(), b.v_scale.cpu(), torch.bfloat16, True, dim, 700)


def test_same_inputs_same_bits():
    """The join takes parts in their order: no result depends on which workgroup ended first."""
    from tensor_layout_amd import kv
    g = torch.Generator().manual_seed(32)
    starts, lengths, table, pages = kv_cases.batch(g, [1, 1, 120], [3000, 70, 500], 32)
    k, ks, v, vs = kv_cases.pools(g, pages, 32, 2, 64, torch.float16, True, 16, False)
    q = torch.randn((122, 4, 64), generator=g).half().cuda()
    c = kv.PagedCache(on_gpu(k), on_gpu(v), dev(ks), dev(vs))
    t = [dev(x) for x in (table, starts, lengths)]
    first = kv.attend(q, c, *t).clone()
    for _ in range(5):
        assert torch.equal(kv.attend(q, c, *t), first)
