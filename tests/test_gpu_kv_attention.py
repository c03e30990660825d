"""Attention over the 4-bit cache on the GPU against its formula in 64 bits.

Two bounds, both set by the roundings the call documents.  Element by element the worst case of
serving_model.attention; over a call the rms error relative to the rms output, where independent
roundings of 2^-11 (keys, weights, values; scores of a spread of a few) and the output's type add
up to well under 2^-9 for 16-bit and fp32 outputs and, for bf16 (2^-8 / sqrt(3) alone), 2^-8.
"""
import pytest
import torch

from tests.gpu_helpers import lib
from tests.serving_model import attention, kv_values
from tests.test_gpu_kv_cache import build

pytestmark = pytest.mark.gpu
RMS = {torch.float16: 2.0 ** -9, torch.float32: 2.0 ** -9, torch.bfloat16: 2.0 ** -8}
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def fill(q, lens, heads, dim, page, dtype, seed):
    """A cache holding whole sequences, its table, and the stored keys and values per sequence."""
    cache, table, cu, ln, k, v = build(q, lens, lens, heads, dim, page, dtype, seed)
    q.kv_append(cache, k.cuda(), v.cuda(), table, cu, ln)
    at = [sum(lens[:b]) for b in range(len(lens) + 1)]
    keys = [kv_values(k[at[b]:at[b + 1]]) for b in range(len(lens))]
    values = [kv_values(v[at[b]:at[b + 1]]) for b in range(len(lens))]
    return cache, table, ln, keys, values


def offsets(news):
    return torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], dtype=torch.int32, device="cuda")


def check(got, want, bound, label):
    g = got.cpu().double()
    assert torch.isfinite(g).all(), f"{label}: not finite"
    err = (g - want).abs()
    rms = float(err.square().mean().sqrt() / want.square().mean().sqrt().clamp(min=1e-30))
    worst = float((err / bound).max())
    print(f"{label}: rms {rms:.2e}, worst {worst:.3f} of the bound", flush=True)
    assert worst <= 1, f"{label}: {int((err > bound).sum())} elements past the bound"
    assert rms <= RMS[got.dtype], f"{label}: rms error {rms:.3e}"


def run(q, news, lens, hq, hkv, dim, page, dtype, window=0, cap=0.0, seed=0, spread=1.5):
    cache, table, ln, keys, values = fill(q, lens, hkv, dim, page, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    x = (spread * torch.randn(sum(news), hq, dim, generator=g)).to(dtype)
    got = q.kv_attention(cache, x.cuda(), table, offsets(news), ln, max(max(news), 1), max(lens), window=window,
                         softcap=cap)
    torch.cuda.synchronize()
    want, bound = attention(x, keys, values, lens, news, window, cap)
    check(got, want, bound, f"news={news[:4]} lens={lens[:4]} hq={hq} hkv={hkv} dim={dim} page={page} {dtype} w={window} c={cap}")


CASES = [
    # new tokens, lengths, hq, hkv, dim, page, dtype, window, cap
    ([1], [1], 1, 1, 64, 32, F16, 0, 0.0),
    ([1], [509], 32, 8, 64, 64, BF16, 0, 0.0),
    ([1, 1, 1], [1, 32, 33], 4, 4, 96, 32, F16, 0, 0.0),
    ([1, 1], [700, 31], 8, 1, 128, 64, F32, 0, 0.0),
    ([1, 1], [1500, 64], 8, 2, 128, 64, BF16, 0, 30.0),
    ([1, 1], [2100, 999], 6, 1, 192, 128, F16, 0, 0.0),
    ([1], [3001], 12, 2, 256, 64, F16, 1024, 50.0),
    ([1, 1, 1], [200, 64, 65], 16, 16, 128, 32, F16, 1, 0.0),
    ([1, 1], [200, 97], 20, 1, 64, 32, BF16, 33, 0.0),          # more than 16 heads a cache head
    ([5, 5], [300, 5], 64, 8, 128, 64, BF16, 0, 0.0),
    ([9, 2, 1], [1000, 40, 1], 8, 1, 256, 256, F16, 0, 20.0),
    ([7, 3], [900, 901], 12, 4, 96, 64, F32, 50, 0.0),
    ([4], [2500], 24, 3, 64, 64, F16, 31, 0.0),
    # prompts
    ([65], [65], 1, 1, 64, 64, F16, 0, 0.0),
    ([130, 77], [130, 300], 8, 2, 128, 64, BF16, 0, 0.0),
    ([200], [1111], 4, 4, 96, 32, F16, 0, 50.0),
    ([300, 1, 150], [300, 40, 700], 4, 1, 256, 128, BF16, 100, 0.0),
    ([129], [640], 6, 2, 192, 64, F32, 0, 0.0),
    ([511], [512], 8, 2, 64, 64, F16, 64, 0.0),
    ([70], [2300], 2, 1, 128, 64, BF16, 0, 0.0),
]


@pytest.mark.parametrize("news,lens,hq,hkv,dim,page,dtype,window,cap", CASES)
def test_attention(news, lens, hq, hkv, dim, page, dtype, window, cap):
    run(lib(), news, lens, hq, hkv, dim, page, dtype, window, cap, seed=dim + hq)


@pytest.mark.parametrize("news", [[1, 1, 1], [90, 80, 1]])
def test_rows_that_see_nothing(news):
    """Tokens before place 0 and tokens whose every visible place has no page give zeros; a bad page
    in the middle hides its tokens only."""
    q = lib()
    lens, hq, hkv, dim, page = [100, 100, 100], 4, 2, 64, 32
    print(f"attention rows that see nothing {news}", flush=True)
    cache, table, ln, keys, values = fill(q, lens, hkv, dim, page, F16, 2)
    table = table.cpu()
    table[1, :] = cache.pages + 7               # nothing of the second sequence is anywhere
    table[2, 1] = -1
    g = torch.Generator().manual_seed(7)
    x = torch.randn(sum(news), hq, dim, generator=g).to(F16)
    short = torch.tensor([news[0] - 1, 100, 100], dtype=torch.int32, device="cuda")     # the first row is at place -1
    got = q.kv_attention(cache, x.cuda(), table.cuda(), offsets(news), short, max(news), 100).cpu()
    torch.cuda.synchronize()
    assert not got[0].any()
    assert not got[news[0]:news[0] + news[1]].any()
    seen = [torch.ones(100, dtype=torch.bool) for _ in lens]
    seen[2][32:64] = False
    want, bound = attention(x[-news[2]:], keys[2:], values[2:], [100], news[2:], seen=seen[2:])
    check(got[-news[2]:], want, bound, "bad page in the middle")
    if news[0] > 1:
        want, bound = attention(x[1:news[0]], [keys[0][:news[0] - 1]], [values[0][:news[0] - 1]], [news[0] - 1],
                                [news[0] - 1])
        check(got[1:news[0]], want, bound, "rows after place 0")


def test_empty_sequences():
    """A sequence without new tokens, and one of length 0 with a new token."""
    q = lib()
    print("attention empty sequences", flush=True)
    cache, table, ln, keys, values = fill(q, [40, 70, 33], 2, 64, 32, F16, 4)
    x = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).to(F16)
    cu = torch.tensor([0, 1, 1, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 70, 33], dtype=torch.int32, device="cuda")
    got = q.kv_attention(cache, x.cuda(), table, cu, lens, 1, 70).cpu()
    assert not got[0].any()
    want, bound = attention(x[1:], keys[2:], values[2:], [33], [1])
    check(got[1:], want, bound, "after an empty one")
    none = q.kv_attention(cache, x[:0].cuda(), table, torch.zeros(4, dtype=torch.int32, device="cuda"), lens, 1, 70)
    assert tuple(none.shape) == (0, 4, 64)


@pytest.mark.parametrize("new", [1, 80])
def test_lengths_above_the_bound_are_served(new):
    """max_ctx only shapes the launch."""
    q = lib()
    print(f"attention past max_ctx new={new}", flush=True)
    cache, table, ln, keys, values = fill(q, [1700], 2, 64, 64, F16, 4)
    x = torch.randn(new, 4, 64, generator=torch.Generator().manual_seed(1)).to(F16)
    for bound_ctx in (new, 600, 5000):
        got = q.kv_attention(cache, x.cuda(), table, offsets([new]), ln, new, bound_ctx)
        want, bound = attention(x, keys, values, [1700], [new])
        check(got, want, bound, f"max_ctx {bound_ctx}")


@pytest.mark.parametrize("news", [[1, 1], [70, 100]])
def test_score_ranges(news):
    """Huge and tiny queries: one key takes everything, or all count alike; scores falling and rising
    along the cache move the softmax's reference many times."""
    q = lib()
    lens, hq, hkv, dim = [600, 333], 4, 2, 64
    for spread in (1e-6, 60.0, 2000.0):
        print(f"attention spread {spread} {news}", flush=True)
        cache, table, ln, keys, values = fill(q, lens, hkv, dim, 64, F16, 3)
        x = (spread * torch.randn(sum(news), hq, dim, generator=torch.Generator().manual_seed(5))).to(F16)
        got = q.kv_attention(cache, x.cuda(), table, offsets(news), ln, max(news), 600)
        torch.cuda.synchronize()
        want, bound = attention(x, keys, values, lens, news)
        err = (got.cpu().double() - want).abs()
        assert (err <= bound).all(), f"spread {spread}"


def test_infinite_and_nan_queries_stay_in_their_row():
    q = lib()
    print("attention nan queries", flush=True)
    for news in ([2], [100]):
        cache, table, ln, keys, values = fill(q, [300], 1, 64, 64, F16, 3)
        x = torch.randn(news[0], 4, 64, generator=torch.Generator().manual_seed(5)).to(F16)
        bad = x.clone()
        bad[1, 2, 5] = float("nan")
        got = q.kv_attention(cache, bad.cuda(), table, offsets(news), ln, news[0], 300).cpu()
        assert got[1, 2].isnan().all()
        x[1, 2] = 0
        got[1, 2] = 0
        want, bound = attention(x, keys, values, [300], news)
        want[1, 2] = 0
        check(got, want, bound, "other rows")


@pytest.mark.parametrize("news,lens", [([1, 1], [3000, 1234]), ([120, 64], [900, 64])])
def test_results_repeat_and_replay(news, lens):
    """Two calls agree bit for bit; a captured call replays to the eager result, with eager work in
    between; a call on another stream, with its own output and workspace, gives the same."""
    q = lib()
    hq, hkv, dim = 8, 2, 128
    print(f"attention graph {news}", flush=True)
    cache, table, ln, _, _ = fill(q, lens, hkv, dim, 64, BF16, 6)
    cu = offsets(news)
    x = torch.randn(sum(news), hq, dim, generator=torch.Generator().manual_seed(5)).to(BF16).cuda()
    need = q.kv_attention_workspace_bytes(cache, 2, sum(news), hq, max(news), max(lens))
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    call = lambda: q.kv_attention(cache, x, table, cu, ln, max(news), max(lens), out=out, workspace=ws)
    want = call().clone()
    assert torch.equal(call(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = q.kv_attention(cache, x, table, cu, ln, max(news), max(lens))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(other, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
        call()
        torch.cuda.synchronize()


def test_strided_queries():
    q = lib()
    print("attention strided queries", flush=True)
    cache, table, ln, keys, values = fill(q, [100, 200], 2, 64, 64, BF16, 6)
    g = torch.Generator().manual_seed(5)
    fused = torch.randn(3, 8, 64, generator=g).to(BF16)
    want, bound = attention(fused[:, 1:5], keys, values, [100, 200], [1, 2])
    got = q.kv_attention(cache, fused.cuda()[:, 1:5], table, offsets([1, 2]), ln, 2, 200)
    check(got, want, bound, "slice of a fused projection")
    odd = torch.empty(3 * 4 * 64 + 1, dtype=BF16, device="cuda")[1:].view(3, 4, 64)
    odd.copy_(fused[:, 1:5])
    assert torch.equal(q.kv_attention(cache, odd, table, offsets([1, 2]), ln, 2, 200), got)


def test_scales_out_of_the_middle_range():
    """Values near fp16's end and subnormal scales go through the products without overflow."""
    q = lib()
    print("attention extreme values", flush=True)
    for factor in (9000.0, 3e-7):
        cache, table, cu, ln, k, v = build(q, [200], [200], 1, 64, 64, F32, 8)
        v = v * factor
        q.kv_append(cache, k.cuda(), v.cuda(), table, cu, ln)
        for new in (1, 100):
            x = torch.randn(new, 4, 64, generator=torch.Generator().manual_seed(5))
            got = q.kv_attention(cache, x.cuda(), table, offsets([new]), ln, new, 200)
            want, bound = attention(x, [kv_values(k)], [kv_values(v)], [200], [new])
            # a value below 2^-14 rounds to a multiple of 2^-24 on its way into the product
            err = (got.cpu().double() - want).abs()
            assert (err <= bound + 2.0 ** -25).all(), (factor, new)
