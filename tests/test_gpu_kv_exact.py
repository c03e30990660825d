"""Attention over the 4-bit cache where the scores are known exactly, so that the bounds are sharp.

Queries are whole numbers of at most 11 bits, keys whole numbers of -7..7 times a power of two: every
product of a query and a key and every partial sum of them fits fp32's 24 bits, in whichever order
they are added.  What is left of a call's documented roundings is
  * a few steps of fp32 in the score's factor, the cap and the exponent: e = 8 * 2^-24 (|score| + 1),
  * the weights' (with the value's scale in the kernel of few rows) rounding to fp16, 2^-11, or
    2^-25 under a row whose largest weight is at least 2^6, which with codes up to 8 under scales up to
    2^vlog, at most twice the largest, is 2^-29 of the largest value a key;
  * the values' rounding to fp16 in bf16 calls of many rows, 2^-11;
  * sums in fp32, 2^-23 a key, and the output's rounding to its type.
An rms limit adds up the same roundings as independent ones: (2^-11 twice + output) / sqrt(3).
"""
import math

import pytest
import torch

from tests.gpu_helpers import lib
from tests.serving_model import U, kv_values
from tests.test_gpu_kv_attention import BF16, F16, F32, offsets
from tests.test_gpu_kv_cache import build

pytestmark = pytest.mark.gpu
STEP = 0.125                # scale of every run of the keys
KERNELS = ["few_rows", "many_rows"]


def whole_keys(n, heads, dim, gen):
    """Whole numbers [n, heads, dim], 7 the largest magnitude of every run of 32, whose sum is 0: what
    the queries have in common cancels."""
    half = torch.randint(1, 8, (n, heads, dim // 32, 16), generator=gen)
    half[..., 0] = 7
    run = torch.cat([half, -half], -1)
    order = torch.rand(run.shape, generator=gen).argsort(-1)
    return run.gather(-1, order).flatten(-2).double()


def expected(q, keys, values, lens, news, window=0, cap=0.0, hidden=None):
    """(out, bound) for q [tokens, hq, d] on stored keys and values (64 bits) of the sequences; hidden: of
    each sequence the places [first, last) that have no page."""
    dt, q = q.dtype, q.double()
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    hq, d = q.shape[1:]
    at = 0
    for b, (k, v, n, m) in enumerate(zip(keys, values, lens, news)):
        group = hq // k.shape[1]
        place, t = torch.arange(n - m, n)[:, None], torch.arange(n)[None]
        gone = (t > place) | (t <= place - window) if window else t > place
        if hidden:
            gone = gone | (t >= hidden[b][0]) & (t < hidden[b][1])
        for h in range(hq):
            kk, vv = k[:, h // group], v[:, h // group]
            x = q[at:at + m, h] @ kk.T / math.sqrt(d)
            if cap:
                x = cap * torch.tanh(x / cap)
            e = 8 * 2.0 ** -24 * (x.abs().masked_fill(gone, 0).amax(1, keepdim=True) + 1)
            p = torch.softmax(x.masked_fill(gone, float("-inf")), 1)
            o = p @ vv
            rel = torch.expm1(2 * e) + 2 * 2.0 ** -11 + n * 2.0 ** -23
            out[at:at + m, h] = o
            bound[at:at + m, h] = rel * (p @ vv.abs()) + U[dt] * o.abs() + n * 2.0 ** -29 * vv.abs().amax()
        at += m
    return out, bound


def rms(err, want):
    return float(err.square().mean().sqrt() / want.square().mean().sqrt())


def rms_limit(dt):
    return math.sqrt((2 * 2.0 ** -22 + U[dt] ** 2) / 3)


def stored(q, lens, hkv, dim, page, dtype, seed, dirty=True, order=None):
    """A cache of whole keys times STEP and random values, its table and what it stores per sequence.  order:
    of a sequence's whole keys [n, heads, dim], its places in the order they are to be stored."""
    cache, table, cu, ln, _, v = build(q, lens, lens, hkv, dim, page, dtype, seed, dirty)
    whole = whole_keys(sum(lens), hkv, dim, torch.Generator().manual_seed(seed + 100))
    if order:
        whole = torch.cat([x.gather(0, order(x).unsqueeze(-1).expand(x.shape)) for x in whole.split(lens)])
    k = (STEP * whole).to(dtype)
    assert torch.equal(kv_values(k), STEP * whole)
    q.kv_append(cache, k.cuda(), v.cuda(), table, cu, ln)
    cut = lambda x: list(kv_values(x).split(lens))
    return cache, table, ln, cut(k), cut(v)


def check(got, want, bound, label, limit=None):
    g = got.cpu().double()
    assert torch.isfinite(g).all(), f"{label}: not finite"
    err = (g - want).abs()
    off = rms(err, want)
    print(f"{label}: rms {off:.2e}, worst {float((err / bound).max()):.3f} of the bound", flush=True)
    assert bool((err <= bound).all()), f"{label}: {int((err > bound).sum())} elements past the bound, rms {off:.2e}"
    assert off <= (limit or rms_limit(got.dtype)), f"{label}: rms error {off:.2e}"


def sharp(want, bound, *others, part=0.9):
    """The bound tells the result from zeros and from other results in nearly every element (in `part`)."""
    for other in (torch.zeros_like(want), *others):
        assert ((want - other).abs() > bound).double().mean() > part


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("common", [0, 1500])
def test_queries_with_a_common_offset(kernel, dtype, dim, common):
    """An offset that all channels of the queries share, as biased projections give, costs no bits."""
    q = lib()
    print(f"offset queries {kernel} {dtype} dim={dim} offset={common}", flush=True)
    lens, news, hq, hkv = [300, 77], [40, 20], 4, 2
    cache, table, ln, keys, values = stored(q, lens, hkv, dim, 64, dtype, dim)
    x = common + torch.randint(-4, 5, (sum(news), hq, dim), generator=torch.Generator().manual_seed(dim))
    want, bound = expected(x.to(dtype), keys, values, lens, news)
    sharp(want, bound, expected(x.to(dtype), [k.roll(1, 0) for k in keys], values, lens, news)[0])
    with q.forced_kv_kernel(kernel):
        got = q.kv_attention(cache, x.to(dtype).cuda(), table, offsets(news), ln, max(news), max(lens))
    check(got, want, bound, f"offset {common}")


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_window_of_any_size_with_rows_before_place_0(kernel, dtype):
    """The largest window an int32 holds is no window at all, also for a wave whose first rows are at
    places before 0."""
    q = lib()
    news, length, before, hq, hkv, dim = [80], 70, 10, 4, 1, 64
    cache, table, _, keys, values = stored(q, [length], hkv, dim, 32, dtype, 3)
    x = torch.randint(-4, 5, (80, hq, dim), generator=torch.Generator().manual_seed(1)).to(dtype)
    ln = torch.tensor([length], dtype=torch.int32, device="cuda")
    for window in (2 ** 31 - 1, 2 ** 31 - 5, 2 ** 31 - 80, 71, 33):
        print(f"window {window} {kernel} {dtype}", flush=True)
        want, bound = expected(x[before:], keys, values, [length], [length], window)
        sharp(want[8:], bound[8:])
        with q.forced_kv_kernel(kernel):
            got = q.kv_attention(cache, x.cuda(), table, offsets(news), ln, 80, length, window=window)
        assert not got[:before].any()
        check(got[before:], want, bound, f"window {window}")


def along(x, shape):
    """The order of whole keys [n, heads, dim] in which their products with `direction` rise, fall or do
    one after the other."""
    n = x.shape[0]
    rising = (x * direction(x.shape[2])).sum(-1).argsort(0)
    if shape == "rising":
        return rising
    if shape == "falling":
        return rising.flip(0)
    return torch.cat([rising[0:n:2], rising[1:n:2].flip(0)])


def direction(dim):
    return torch.randint(-4, 5, (dim,), generator=torch.Generator().manual_seed(dim)).double()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("shape", ["rising", "falling", "peak"])
def test_scores_along_the_cache(kernel, dtype, shape):
    """Scores that rise, fall or do both along the cache, from all alike to one that takes everything: the
    softmax's reference moves with nearly every block, or never."""
    q = lib()
    dim, lens, news, hq, hkv = 64, [2000, 500], [20, 33], 4, 2
    cache, table, ln, keys, values = stored(q, lens, hkv, dim, 64, dtype, 11, order=lambda x: along(x, shape))
    row = torch.tensor([1.0, 2.0, -1.0, 1.0, -2.0])[torch.arange(sum(news) * hq) % 5].view(sum(news), hq, 1)
    for power in (-14, 0, 3, 6, 10):
        print(f"scores {shape} 2^{power} {kernel} {dtype}", flush=True)
        x = (2.0 ** power * row * direction(dim)).to(dtype)
        want, bound = expected(x, keys, values, lens, news)
        sharp(want, bound, *([expected(x, [k.roll(1, 0) for k in keys], values, lens, news)[0]] if power >= 0 else []), part=0.8)
        with q.forced_kv_kernel(kernel):
            got = q.kv_attention(cache, x.cuda(), table, offsets(news), ln, max(news), max(lens))
        torch.cuda.synchronize()
        g = got.cpu().double()
        off = rms(g - want, want)
        print(f"  rms {off:.2e}, worst {float(((g - want).abs() / bound).max()):.3f} of the bound", flush=True)
        assert bool(((g - want).abs() <= bound).all())
        # scores are off by e, whose effect the bound holds; an output is an average of `n` values at least
        assert off <= rms_limit(dtype) * 2 ** 0.5 + 16 * 2.0 ** -24 * 2.0 ** max(power, 0) * 40


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_queries(kernel, cap, sign):
    """An infinite query's row is NaN where it sees a key (its scores are infinite or NaN, of which a
    softmax makes NaN, also where all are -inf), under a cap too.  Rows that see no key stay zeros, other
    rows what they are."""
    q = lib()
    print(f"infinite queries {kernel} cap={cap} {sign}", flush=True)
    dim, length, before, hq = 64, 40, 2, 2
    cache, table, _, keys, values = stored(q, [length], 1, dim, 64, F16, 5)
    ln = torch.tensor([length], dtype=torch.int32, device="cuda")
    m = length + before
    x = torch.randint(-4, 5, (m, hq, dim), generator=torch.Generator().manual_seed(1)).to(F16)
    fine, bound = expected(x[before:], keys, values, [length], [length], 0, cap)
    bad = x.clone()
    bad[::2, 0, 7] = sign * float("inf")         # of places -2, 0, 2, ...
    with q.forced_kv_kernel(kernel):
        got = q.kv_attention(cache, bad.cuda(), table, offsets([m]), ln, m, length, softcap=cap).cpu().double()
    assert not got[:before].any()
    got = got[before:]
    assert got[::2, 0].isnan().all()
    err = (got - fine).abs()
    assert bool((err <= bound)[1::2].all()) and bool((err <= bound)[:, 1].all())


# The rms limit is doubled below where few values of unlike sizes make up an output: their roundings
# average less.
def reloads(q, kernel, lens, news, hq, hkv, dim, dtype, waves, hole, window=0):
    """A call whose plan gives every sequence one split, past 64 blocks a wave (few rows) or a workgroup
    (many); page `hole` of the first sequence is missing.  The keys' scores rise towards the page's end from both
    sides, so the pages around it decide the result."""
    page = 64

    def order(x):
        near = (torch.arange(len(x)) - (hole * page + page)).abs().argsort(stable=True)
        rank = torch.empty_like(near)
        rank[near] = torch.arange(len(x))
        return along(x, "falling")[rank]

    cache, table, ln, keys, values = stored(q, lens, hkv, dim, page, dtype, dim + 1, order=order)
    print(f"reload {kernel} {lens[:3]} new={news[:3]} dim={dim} {dtype} window={window}", flush=True)
    x = (1.5 * (1 + torch.arange(sum(news) * hq) % 2).view(sum(news), hq, 1) * direction(dim)).to(dtype)
    table = table.cpu()
    table[0, hole] = cache.pages + 5
    hidden = [(hole * page, hole * page + page)] + [(0, 0)] * (len(lens) - 1)
    want, bound = expected(x, keys, values, lens, news, window, hidden=hidden)
    # a page's keys taken for the next one's from the reload on
    wrong = [torch.cat([k[:hole * page], k[hole * page:].roll(page, 0)]) for k in keys]
    first = slice(0, news[0])
    sharp(want[first], bound[first], expected(x[first], wrong[:1], values[:1], lens[:1], news[:1], window, hidden=hidden[:1])[0],
          expected(x[first], keys[:1], values[:1], lens[:1], news[:1], window)[0])
    with q.forced_kv_kernel(kernel):
        plan = q.kv_attention_plan(cache, len(lens), sum(news), hq, max(news), 64, dtype, window)
        assert plan == {"kernel": kernel, "waves": waves, "splits": 1}
        got = q.kv_attention(cache, x.cuda(), table.cuda(), offsets(news), ln, max(news), 64, window=window)
    check(got, want, bound, "reload", 2 * rms_limit(dtype))


@pytest.mark.parametrize("window", [0, 18100])
@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, F32)])
def test_few_rows_past_64_blocks_a_wave(dim, dtype, window):
    """Eight waves of 79 blocks each (71 with the window, which begins inside a page)."""
    hole = (20011 - 18100 if window else 0) // 64 + 16384 // 64 + 1
    reloads(lib(), "few_rows", [20011], [2], 4, 1, dim, dtype, 8, hole, window)


def test_few_rows_past_64_blocks_a_wave_of_four():
    reloads(lib(), "few_rows", [9001] + [40 + b for b in range(32)], [1] * 33, 16, 8, 64, F16, 4, 8192 // 64 + 1)


@pytest.mark.parametrize("window", [0, 4300])
@pytest.mark.parametrize("dim,dtype", [(64, F16), (96, BF16), (128, F16), (192, F32), (256, F16), (256, BF16)])
def test_many_rows_past_64_blocks(dim, dtype, window):
    """142 blocks in a split, 136 or 137 with the window."""
    hole = (4531 - 40 - 4300 if window else 0) // 64 + 2048 // 64 + 1
    reloads(lib(), "many_rows", [4531], [40], 1, 1, dim, dtype, 4, hole, window)


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("length", [700, 9000])
def test_joins_of_few_and_many_splits(dim, dtype, length):
    """Two splits, which one wave a row joins, and more than it takes in one round; a short sequence whose
    later splits are empty beside it."""
    q = lib()
    print(f"joins dim={dim} {dtype} {length}", flush=True)
    lens, news, hq, hkv = [length, 45], [1, 2], 3, 1
    cache, table, ln, keys, values = stored(q, lens, hkv, dim, 64, dtype, dim + 7)
    splits = q.kv_attention_plan(cache, 2, 3, hq, 2, length, dtype)["splits"]
    assert splits > 16 if length == 9000 else splits == 2
    x = 2 * torch.randint(-4, 5, (3, hq, dim), generator=torch.Generator().manual_seed(3)).to(dtype)
    want, bound = expected(x, keys, values, lens, news)
    sharp(want, bound, expected(x, [k.roll(1, 0) for k in keys], values, lens, news)[0], part=0.8)
    got = q.kv_attention(cache, x.cuda(), table, offsets(news), ln, 2, length)
    check(got, want, bound, f"{splits} splits", 2 * rms_limit(dtype))


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (256, F16)])
def test_pages_past_4_gib(dim, dtype):
    """Pages whose bytes lie past 2^32 from the cache's start: append, read-out and both kernels."""
    q = lib()
    page, heads, length, new, hq = 64, 8, 500, 40, 8
    pages = (5 << 30) // (36 * dim * heads * (page // 32))
    print(f"far pages dim={dim} {dtype} {pages} pages", flush=True)
    cache = q.kv_cache(pages, page, heads, dim)
    need = -(-length // page)
    first = pages - need
    assert cache.buffer.numel() * first // pages > 1 << 32
    table = (first + torch.randperm(need, generator=torch.Generator().manual_seed(2))).int().view(1, need).cuda()
    gen = torch.Generator().manual_seed(dim)
    k = (STEP * whole_keys(length, heads, dim, gen)).to(dtype)
    v = torch.randn(length, heads, dim, generator=gen).to(dtype)
    ln = torch.tensor([length], dtype=torch.int32, device="cuda")
    q.kv_append(cache, k.cuda(), v.cuda(), table, offsets([length]), ln)
    rk, rv = q.kv_read(cache, table, offsets([length]), ln, length)
    assert torch.equal(rk.cpu().double(), kv_values(k)) and torch.equal(rv.cpu().double(), kv_values(v))
    assert not cache.buffer[:cache.buffer.numel() // pages * first].any()
    x = torch.randint(-4, 5, (new, hq, dim), generator=gen).to(dtype)
    want, bound = expected(x, [kv_values(k)], [kv_values(v)], [length], [new])
    sharp(want, bound)
    for kernel in KERNELS:
        with q.forced_kv_kernel(kernel):
            got = q.kv_attention(cache, x.cuda(), table, offsets([new]), ln, new, length)
        check(got, want, bound, kernel)
