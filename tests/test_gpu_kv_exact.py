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


def expected(q, keys, values, lens, news, window=0, cap=0.0):
    """(out, bound) for q [tokens, hq, d] on stored keys and values (64 bits) of the sequences."""
    dt, q = q.dtype, q.double()
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    hq, d = q.shape[1:]
    at = 0
    for k, v, n, m in zip(keys, values, lens, news):
        group = hq // k.shape[1]
        place, t = torch.arange(n - m, n)[:, None], torch.arange(n)[None]
        gone = (t > place) | (t <= place - window) if window else t > place
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


def stored(q, lens, hkv, dim, page, dtype, seed, dirty=True):
    """A cache of whole keys times STEP and random values, its table and what it stores per sequence."""
    cache, table, cu, ln, _, v = build(q, lens, lens, hkv, dim, page, dtype, seed, dirty)
    whole = whole_keys(sum(lens), hkv, dim, torch.Generator().manual_seed(seed + 100))
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


def sharp(want, bound, *others):
    """The bound tells the result from zeros and from other results in nearly every element."""
    for other in (torch.zeros_like(want), *others):
        assert ((want - other).abs() > bound).double().mean() > 0.9


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
