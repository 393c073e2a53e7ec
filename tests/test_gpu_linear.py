"""Linear attention over a pool of states on the GPU against the recurrence in 64 bits.

Tolerances.  A is the sum of magnitudes behind a number (the oracle's `size` and `states`).

* A state: each k v product is exact in 32 bits up to 2^-24 of it; its weight l^d = 2^(g d) is off by
  2^-23 (1 + |g d|) (the logarithm's product rounded once more than the exponential), and counts at most
  2^-23 (1 + 30) as far as it counts at all (2^-30 of the sum is below the other terms); in chunks the weighted
  value is the sum of two 16-bit numbers, off by 2^-17 (bf16: two numbers of 8 bits) or 2^-22 (fp16, of the largest one of its
  channel and chunk); sums of n tokens in fp32 round by 2^-24 of A each, some n of them at most.  So
  (2^-17 + 31 2^-23 + (n + 8) 2^-24) A, and for fp16 2^-38 of the largest in a chunk beside it, counted in its 2^-22.
  Token by token the decay multiplies the state: each step rounds by 2^-24 and carries l's own error of 2^-22:
  n 2^-22 at most, within (n + 8) 2^-22.
* An output: the same for what it sums, a product of dim terms more (dim 2^-24), state and scores as two 16-bit
  numbers (2^-17 each), its own rounding of half a step, or in fp16 of half of 2^-24, the step of its smallest
  numbers: 2^-25.  In fp16 the state's parts are brought to a power of two
  under the largest number of 32 channels: numbers 2^-22 of that largest, q's sum beside them.
"""

from __future__ import annotations

import pytest
import torch

from oracle import linear_oracle
from tests.kv_cases import half_step

pytestmark = pytest.mark.gpu


def dev(x):
    return None if x is None else x.cuda() if isinstance(x, torch.Tensor) else torch.tensor(x, dtype=torch.int32).cuda()


def tolerances(want, news, dk, dtype):
    out, state, size, states = want
    n = max(news + [1])
    e = 2.0 ** -17 + 31 * 2.0 ** -23 + (n + 8) * 2.0 ** -22
    rest = 2.0 ** -22 if dtype == torch.float16 else 0.0
    lim = lambda x: x.nan_to_num(0.0, 0.0, 0.0)   # noqa: E731
    by_state = rest * lim(states).amax((1, 2, 3)).amax() if states.numel() else 0.0
    return ((2 * e + dk * 2.0 ** -24 + 2.0 ** -17) * size + half_step(dtype) * out.abs() + rest * lim(size).amax() + 2.0 ** -25 * (dtype == torch.float16)
            + 1e-30, e * states + by_state + 1e-30)


def near(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol) & (got.double() != want) & ~(~got.isfinite() & ~want.isfinite())
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((((got.double() - want).abs() - tol)).nan_to_num().max()))


def inputs(g, tokens, heads, key_heads, dk, dv, slots, dtype):
    q, k = (torch.randn((tokens, key_heads, dk), generator=g).to(dtype) for _ in range(2))
    v = torch.randn((tokens, heads, dv), generator=g).to(dtype)
    state = torch.randn((slots, heads, dk, dv), generator=g)
    decay = -torch.exp2(-8.0 * torch.arange(1, heads + 1) / heads)
    return q, k, v, state, decay


def check(seed, news, *, heads=3, key_heads=None, dk=64, dv=64, dtype=torch.bfloat16, sources="others", starts=None, tweak=None, scale=None,
          strided=False, slots=None):
    from tensor_layout_amd import linear
    g = torch.Generator().manual_seed(seed)
    key_heads = heads if key_heads is None else key_heads
    n = len(news)
    good = [sum(news[:b]) for b in range(n + 1)]
    tokens = good[-1]
    q, k, v, state, decay = inputs(g, tokens, heads, key_heads, dk, dv, 2 * n + 1, dtype)
    order = torch.randperm(2 * n, generator=g).tolist()
    slots = order[:n] if slots is None else slots
    sources = {"others": order[n:], "same": None, "none": [-1] * n}[sources] if isinstance(sources, str) else sources
    starts = good if starts is None else starts
    if tweak:
        tweak(q=q, k=k, v=v, state=state, decay=decay, slots=slots, sources=sources)
    s = dk ** -0.5 if scale is None else scale
    want = linear_oracle.attend(q, k, v, state, decay, slots, starts, sources, s, fill=7.0)
    tol_out, tol_state = tolerances(want, news, dk, dtype)
    if strided:
        big = torch.full((heads, tokens, dv + 8), 7.0, dtype=dtype, device="cuda")
        out = big[:, :, :dv].transpose(0, 1)
        wide = torch.zeros((tokens, 2, key_heads, dk + 8), dtype=dtype, device="cuda")
        wide[:, 0, :, :dk], wide[:, 1, :, :dk] = dev(q), dev(k)
        qd, kd, vd = wide[:, 0, :, :dk], wide[:, 1, :, :dk], dev(v.transpose(0, 1).contiguous()).transpose(0, 1)
        store = torch.full((heads, 2 * n + 1, dk + 1, dv + 4), 5.0, device="cuda")
        pooled = store[:, :, :dk, :dv].transpose(0, 1)
        pooled.copy_(state)
    else:
        out = torch.full(v.shape, 7.0, dtype=dtype, device="cuda")
        qd, kd, vd, pooled = dev(q), dev(k), dev(v), dev(state)
    pool = linear.StatePool(pooled, dev(decay))
    r = linear.attend(qd, kd, vd, pool, dev(slots), dev(starts), sources=dev(sources), scale=scale, out=out)
    assert r is out
    near(out.cpu(), want[0], tol_out)
    near(pooled.cpu(), want[1], tol_state)
    if strided:
        assert bool((big[:, :, dv:] == 7).all()) and bool((store[:, :, dk:] == 5).all()) and bool((store[..., dv:] == 5).all())
    return out, pooled, want


DTYPES = [torch.bfloat16, torch.float16]
DIMS = [(16, 16), (32, 48), (64, 64), (80, 96), (96, 80), (112, 32), (128, 128), (144, 160), (192, 256), (256, 192), (256, 256), (208, 16)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", DIMS)
def test_single_tokens(dtype, dk, dv):
    check(1, [1] * 5, dk=dk, dv=dv, dtype=dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", DIMS)
def test_prompt(dtype, dk, dv):
    """One sequence: whole chunks and a part of one, in one segment."""
    check(2, [150], dk=dk, dv=dv, dtype=dtype, heads=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 96), (128, 128), (192, 64), (256, 256)])
def test_long_prompt(dtype, dk, dv):
    """Segments of one sequence, the last one short."""
    check(3, [1003], dk=dk, dv=dv, dtype=dtype, heads=2)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513])
@pytest.mark.parametrize("sources", ["others", "same", "none"])
def test_lengths(n, sources):
    check(4, [n], heads=2, sources=sources)


@pytest.mark.parametrize("news", [[1, 40, 3, 0, 100, 16, 17], [0, 1, 0], [70, 70], [5] * 40, [300, 1, 1, 700], [1] * 70, [16, 17] * 3, [0, 0, 90]])
@pytest.mark.parametrize("dtype", DTYPES)
def test_batches(news, dtype):
    check(5, news, dtype=dtype, heads=4, key_heads=2, dv=96)


@pytest.mark.parametrize("heads,key_heads", [(1, 1), (8, 1), (6, 3), (5, 5)])
@pytest.mark.parametrize("news", [[1, 1], [100, 3]])
def test_key_heads(heads, key_heads, news):
    check(6, news, heads=heads, key_heads=key_heads)


@pytest.mark.parametrize("news", [[1, 1, 4], [90, 20, 5], [700]])
def test_strides(news):
    check(7, news, strided=True)
    check(7, news, strided=True, dtype=torch.float16, dk=128, dv=32)


@pytest.mark.parametrize("news", [[1, 2], [200, 70], [900]])
@pytest.mark.parametrize("values", [[0.0, -1e-7, -1e-3], [-5.0, -80.0, -1000.0], [float("-inf"), 0.5, -1e30], [-3e38, float("nan"), -0.1]])
def test_decays(news, values):
    """None at all, to nothing at once, over zero (which counts as zero), and no number: that head's rows and states are none."""
    def put(decay, **_):
        decay.copy_(torch.tensor(values))
    check(8, news, tweak=put)
    check(8, news, tweak=put, dtype=torch.float16, dk=96, dv=32)


@pytest.mark.parametrize("news", [[1, 1, 1], [100, 90, 20]])
def test_slots_that_are_not_there(news):
    """A state of zeros to begin with, none kept; the pool's other slots stay as they are."""
    check(9, news, slots=[2, -1, 100], sources=[100, 0, -7])
    check(9, news, slots=[2, -1, 4], sources=None)


def test_forks_of_one_state():
    """Several sequences read one slot and write their own."""
    check(10, [1, 1, 1], slots=[1, 2, 3], sources=[0, 0, 0])
    check(10, [30, 70, 1], slots=[1, 2, 3], sources=[0, 0, 0])
    check(10, [500, 700], slots=[1, 2], sources=[0, 0], heads=1)


@pytest.mark.parametrize("news", [[2, 1, 3], [90, 20, 70], [300, 300, 1]])
def test_sequences_out_of_order_are_skipped(news):
    good = [sum(news[:b]) for b in range(4)]
    for bad in ([0, -4, good[2], good[3]], [0, good[1], 10_000, good[3]], [0, good[1], good[1], good[3]], [-1, good[1], good[2], good[3]],
                [0, good[1], good[2], 10_000], [5, 4, 3, 2]):
        check(11, news, starts=bad)
        check(11, news, starts=bad, sources="same", dtype=torch.float16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("at", [0, 3, 40, 63, 64, 100, 149])
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_numbers_that_are_none(dtype, at, which):
    """They show from their token on (a query's in its own row), and in no row before it."""
    from tensor_layout_amd import linear
    for bad in (float("inf"), float("nan")):
        def plant(**kw):
            kw[which][at, 0, 5] = bad
        for news in ([150], [150, 30]):
            out, pooled, want = check(12, news, heads=2, dk=32, dv=64, dtype=dtype, tweak=plant)
            assert bool(out[:at].isfinite().all())
            assert bool(out[at + 1:150, 1].isfinite().all())
            if which == "q":
                assert bool(pooled.isfinite().all()) and not bool(out[at, 0].isfinite().any())
            else:
                assert not bool(out[at, 0].isfinite().all())


def test_states_that_are_no_numbers():
    """Of one sequence alone, and only of its head."""
    def plant(state, slots, sources, **_):
        state[sources[1], 0, 3, 7] = float("nan")
    for news in ([1, 1, 1], [90, 40, 33]):
        out, pooled, want = check(13, news, tweak=plant)
        assert not bool(out[news[0]:news[0] + news[1], 0, 7].isfinite().any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [2.0 ** -12, 2.0 ** 7])
@pytest.mark.parametrize("news", [[1, 3], [140], [800]])
def test_small_and_large_numbers(dtype, scale, news):
    """Magnitudes far from one, states further yet."""
    def grow(k, v, state, **_):
        k.mul_(scale)
        v.mul_(scale)
        state.mul_(scale * scale)
    check(14, news, tweak=grow, dtype=dtype, scale=1.0 if scale < 1 else 2.0 ** -14, heads=2)


def test_streams_and_a_graph():
    """A named stream beside another's calls, and a captured call replayed on new numbers."""
    from tensor_layout_amd import linear
    g = torch.Generator().manual_seed(15)
    for news in ([1, 1, 1, 1], [30, 1, 90, 7], [400, 380, 1, 33]):
        tokens = sum(news)
        q, k, v, state, decay = inputs(g, tokens, 2, 2, 64, 64, 8, torch.bfloat16)
        cases = [(list(range(4)), news, [4, 5, 6, 7]), ([1, 0, 3, 2], news[::-1], [7, -1, 5, 4])]

        def of(case):
            slots, counts, sources = case
            starts = [sum(counts[:b]) for b in range(5)]
            return [dev(slots), dev(starts), dev(sources)], linear_oracle.attend(q, k, v, state, decay, slots, starts, sources, 0.125)
        ints, want = of(cases[0])
        args = [dev(x) for x in (q, k, v)]
        pooled = dev(state)
        pool = linear.StatePool(pooled, dev(decay))

        def compare(out, w):
            tol = tolerances(w, news, 64, torch.bfloat16)
            near(out.cpu(), w[0], tol[0])
            near(pooled.cpu(), w[1], tol[1])
        first = linear.attend(*args, pool, ints[0], ints[1], sources=ints[2])
        compare(first, want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = torch.empty_like(args[2])
        twin = linear.StatePool(dev(state), dev(decay))
        torch.cuda.synchronize()
        linear.attend(*args, twin, ints[0], ints[1], sources=ints[2], out=other, stream=side.cuda_stream)
        again = linear.attend(*args, pool, ints[0], ints[1], sources=ints[2])
        torch.cuda.synchronize()
        assert torch.equal(other, again) and torch.equal(first, again) and torch.equal(twin.state, pooled)
        out = torch.empty_like(args[2])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            linear.attend(*args, pool, ints[0], ints[1], sources=ints[2], out=out)
        for i in (1, 0, 1):
            now, want = of(cases[i])
            for a, x in zip(ints, now):
                a.copy_(x)
            pooled.copy_(dev(state))
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            compare(out, want)
            torch.randn(1000, device="cuda").sum().item()


def test_prompt_drafts_and_tokens_in_turn():
    """A prompt in pieces of any size, in place, is the prompt at once."""
    from tensor_layout_amd import linear
    g = torch.Generator().manual_seed(16)
    q, k, v, state, decay = inputs(g, 700, 2, 1, 64, 64, 1, torch.bfloat16)
    state.zero_()
    want = linear_oracle.attend(q, k, v, state, decay, [0], [0, 700], [-1], 0.125)
    tol = tolerances(want, [700], 64, torch.bfloat16)
    pool = linear.StatePool(dev(state), dev(decay))
    args = [dev(x) for x in (q, k, v)]
    at, outs = 0, []
    for n in (300, 1, 1, 7, 64, 16, 17, 1, 293):
        outs.append(linear.attend(*(x[at:at + n] for x in args), pool, dev([0]), dev([0, n]), sources=dev([0 if at else -1])))
        at += n
    near(torch.cat(outs).cpu(), want[0], tol[0])
    near(pool.state.cpu(), want[1], tol[1])


def test_a_call_gives_the_same_again():
    """Bit for bit, whatever runs first."""
    from tensor_layout_amd import linear
    g = torch.Generator().manual_seed(17)
    q, k, v, state, decay = inputs(g, 1300, 4, 4, 128, 128, 4, torch.float16)
    outs = []
    for _ in range(3):
        pool = linear.StatePool(dev(state), dev(decay))
        outs.append((linear.attend(dev(q), dev(k), dev(v), pool, dev([0, 1]), dev([0, 1200, 1300])), pool.state))
    for o, s in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(s, outs[0][1])


def test_slots_far_apart():
    """States beyond 2^31 elements."""
    from tensor_layout_amd import linear
    g = torch.Generator().manual_seed(18)
    slots, dk, dv = 40_000, 256, 256   # 2.6 * 10^9 numbers
    far = torch.empty((slots, 1, dk, dv), device="cuda")
    used = [39_999, 7, 39_000, 20_001]
    q, k, v, some, decay = inputs(g, 91, 1, 1, dk, dv, 4, torch.bfloat16)
    far[torch.tensor(used, device="cuda")] = some.cuda()
    starts = [0, 1, 91]
    want = linear_oracle.attend(q, k, v, some, decay, [0, 1], starts, [2, 3], dk ** -0.5)
    out = linear.attend(dev(q), dev(k), dev(v), linear.StatePool(far, dev(decay)), dev(used[:2]), dev(starts), sources=dev(used[2:]))
    tol = tolerances(want, [1, 90], dk, torch.bfloat16)
    near(out.cpu(), want[0], tol[0])
    near(far[torch.tensor(used, device="cuda")].cpu(), want[1], tol[1])


@pytest.mark.parametrize("news", [[1], [7], [60], [600]])
def test_values_in_place(news):
    """The result over the values: each is read before its own row is written."""
    from tensor_layout_amd import linear
    g = torch.Generator().manual_seed(19)
    q, k, v, state, decay = inputs(g, news[0], 2, 2, 64, 160, 1, torch.bfloat16)
    want = linear_oracle.attend(q, k, v, state, decay, [0], [0, news[0]], None, 0.125)
    x = dev(v)
    linear.attend(dev(q), dev(k), x, linear.StatePool(dev(state), dev(decay)), dev([0]), dev([0, news[0]]), out=x)
    near(x.cpu(), want[0], tolerances(want, news, 64, torch.bfloat16)[0])


def test_many_sequences():
    """More than the 64 that a wave looks through at a time, of all lengths; segments of some."""
    check(20, [b % 23 for b in range(150)], heads=2, dk=32, dv=32)
    check(21, [300 if b % 9 == 0 else 1 + b % 11 for b in range(100)], heads=1, dk=32, dv=32)
    check(22, [1200, 900, 3, 1100], heads=1, dk=32, dv=64, dtype=torch.float16)
