"""The paged 4-bit cache on the GPU against its definition: kv_append and kv_read.

What the cache stands for (value * scale, 4 + 11 bits) is exact in fp32 and every step that
decides a code is taken as defined, so the comparison is for equality.
"""
import pytest
import torch

from tests.gpu_helpers import lib
from tests.serving_model import kv_values

pytestmark = pytest.mark.gpu


def build(q, news, lens, heads, dim, page, dtype, seed, dirty=True):
    """A cache whose pages hold leftovers (every byte 0xFF unless dirty is False), a shuffled page
    table, and the new tokens' keys and values."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
        order = order[n:]
    cache = q.kv_cache(pages, page, heads, dim, "cuda")
    if dirty:
        cache.buffer.fill_(0xFF)
    cu = torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], dtype=torch.int32)
    k, v = (torch.randn(sum(news), heads, dim, generator=g).to(dtype) for _ in range(2))
    return cache, table.cuda(), cu.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), k, v


CASES = [
    # new tokens, lengths, heads, dim, page, dtype
    ([1], [1], 1, 64, 32, torch.float16),
    ([1, 1, 1], [1, 33, 70], 8, 128, 64, torch.bfloat16),
    ([5, 0, 3], [37, 12, 3], 2, 96, 32, torch.float32),
    ([100, 31, 64, 1], [163, 31, 128, 65], 3, 256, 128, torch.float16),
    ([300, 7], [301, 500], 2, 192, 256, torch.bfloat16),
    ([33] * 70, list(range(33, 103)), 1, 64, 64, torch.float16),      # more sequences than a wave has lanes
]


@pytest.mark.parametrize("news,lens,heads,dim,page,dtype", CASES)
def test_append_and_read(news, lens, heads, dim, page, dtype):
    q = lib()
    print(f"kv append news={news[:4]} lens={lens[:4]} heads={heads} dim={dim} page={page} {dtype}", flush=True)
    cache, table, cu, ln, k, v = build(q, news, lens, heads, dim, page, dtype, seed=dim + page)
    q.kv_append(cache, k.cuda(), v.cuda(), table, cu, ln)
    gk, gv = q.kv_read(cache, table, cu, ln, sum(news))
    torch.cuda.synchronize()
    assert torch.equal(gk.cpu().double(), kv_values(k))
    assert torch.equal(gv.cpu().double(), kv_values(v))


def test_tokens_one_by_one_equal_a_prompt():
    """65 single-token calls leave what one call of 65 tokens leaves, older tokens untouched."""
    q = lib()
    n, heads, dim = 65, 2, 128
    print("kv append one by one", flush=True)
    cache, table, _, _, k, v = build(q, [n], [n], heads, dim, 64, torch.float16, seed=3)
    k, v = k.cuda(), v.cuda()
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for t in range(n):
        q.kv_append(cache, k[t:t + 1], v[t:t + 1], table, one, torch.tensor([t + 1], dtype=torch.int32, device="cuda"))
    every = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    gk, gv = q.kv_read(cache, table, every, every[1:], n)
    torch.cuda.synchronize()
    assert torch.equal(gk.cpu().double(), kv_values(k.cpu()))
    assert torch.equal(gv.cpu().double(), kv_values(v.cpu()))


def test_special_values():
    """Zeros, infinities, NaN, a range past fp16's and ties, each in a run of 32 channels."""
    q = lib()
    nan, inf = float("nan"), float("inf")
    x = torch.zeros(40, 1, 64)
    x[1, 0, :32] = nan
    x[2, 0, :3] = torch.tensor([inf, -inf, 1.0])
    x[3, 0, :3] = torch.tensor([1e30, -1e30, 5e29])
    x[4, 0, :4] = torch.tensor([7.0, 0.5, 1.5, -2.5])       # scale 1: ties to even
    x[5, 0, :2] = torch.tensor([-7.0, nan])
    x[6, 0, :2] = torch.tensor([1e-9, -1e-9])               # scale rounds to 0
    x[7, 0, :2] = torch.tensor([3e-7, 1e-7])                # a subnormal scale
    x[8] = 1e-30
    print("kv append special values", flush=True)
    cache, table, cu, ln, _, _ = build(q, [40], [40], 1, 64, 32, torch.float32, seed=1)
    q.kv_append(cache, x.cuda(), x.flip(2).cuda(), table, cu, ln)
    gk, gv = q.kv_read(cache, table, cu, ln, 40)
    torch.cuda.synchronize()
    assert torch.isfinite(gk).all() and torch.isfinite(gv).all()
    assert torch.equal(gk.cpu().double(), kv_values(x))
    assert torch.equal(gv.cpu().double(), kv_values(x.flip(2)))


def test_places_without_a_page():
    """Tokens before place 0, past the table and on bad page numbers are stored nowhere and read as
    zeros; the other tokens, and pages of no sequence, are as they should be."""
    q = lib()
    news, lens, heads, dim, page = [70, 40, 100], [60, 40, 100], 2, 64, 32
    print("kv append places without a page", flush=True)
    cache, table, cu, ln, k, v = build(q, news, lens, heads, dim, page, torch.float16, seed=5, dirty=False)
    table = table.cpu()
    table[1, 0] = cache.pages                   # just past the cache
    table[2, 1] = -1
    table = table[:, :3].contiguous().cuda()    # the last sequence's fourth page is past the table
    q.kv_append(cache, k.cuda(), v.cuda(), table, cu, ln)
    gk, gv = q.kv_read(cache, table, cu, ln, sum(news))
    torch.cuda.synchronize()
    held = torch.ones(sum(news), dtype=torch.bool)
    held[:10] = False                           # places -10 .. -1
    held[70:102] = False                        # the second sequence's first page
    held[110 + 32:110 + 64] = False
    held[110 + 96:] = False
    for got, x in ((gk, k), (gv, v)):
        want = kv_values(x)
        want[~held] = 0
        assert torch.equal(got.cpu().double(), want)
    used = {int(p) for p in table.flatten().tolist() if 0 <= p < cache.pages}
    rest = cache.buffer.view(cache.pages, -1)[[p for p in range(cache.pages) if p not in used]]
    assert not rest.any()


def test_strided_and_misaligned_rows():
    """Slices of a fused projection are read in place; rows off 16 bytes are copied first."""
    q = lib()
    n, heads, dim = 50, 2, 64
    print("kv append strided", flush=True)
    cache, table, cu, ln, _, _ = build(q, [n], [n], heads, dim, 64, torch.bfloat16, seed=9)
    g = torch.Generator().manual_seed(4)
    both = torch.randn(n, 6, dim, generator=g).to(torch.bfloat16).cuda()
    odd = torch.randn(n * heads * dim + 1, generator=g).to(torch.bfloat16).cuda()[1:].view(n, heads, dim)
    k = both[:, 2:4]
    q.kv_append(cache, k, odd, table, cu, ln)
    gk, gv = q.kv_read(cache, table, cu, ln, n)
    torch.cuda.synchronize()
    assert torch.equal(gk.cpu().double(), kv_values(k.cpu()))
    assert torch.equal(gv.cpu().double(), kv_values(odd.cpu()))
