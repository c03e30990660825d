"""Both attention kernels over the 4-bit cache at small sizes, each chosen by the call's option: the plan
alone takes the kernel of many rows for large work only.  Bounds and models as in
test_gpu_kv_attention."""
import pytest
import torch

from tests.gpu_helpers import lib
from tests.serving_model import attention
from tests.test_gpu_kv_attention import BF16, F16, F32, check, fill, offsets, run

pytestmark = pytest.mark.gpu

CASES = [
    # new tokens, lengths, hq, hkv, dim, page, dtype, window, cap
    ([33], [33], 1, 1, 64, 32, F16, 0, 0.0),
    ([65], [97], 1, 1, 64, 64, BF16, 0, 0.0),
    ([130, 77], [130, 300], 8, 2, 128, 64, BF16, 0, 0.0),
    ([130, 77], [130, 300], 8, 2, 128, 64, F16, 0, 0.0),
    ([200], [1111], 4, 4, 96, 32, F16, 0, 50.0),
    ([300, 1, 150], [300, 40, 700], 4, 1, 256, 128, BF16, 100, 0.0),
    ([300, 1, 150], [300, 40, 700], 4, 1, 256, 128, F16, 100, 0.0),
    ([129], [640], 6, 2, 192, 64, F32, 0, 0.0),
    ([129], [641], 6, 2, 192, 64, BF16, 0, 0.0),
    ([511], [512], 8, 2, 64, 64, F16, 64, 0.0),
    ([70], [2300], 2, 1, 128, 64, BF16, 0, 0.0),               # splits
    ([70], [2300], 2, 1, 128, 64, F32, 900, 30.0),
    ([40], [1500], 3, 1, 96, 64, BF16, 1, 0.0),
    # eight waves a workgroup: as many sequences and heads as CUs, unlike lengths
    ([33 + b % 7 for b in range(64)], [50 + 3 * b for b in range(64)], 4, 4, 64, 32, F16, 0, 0.0),
    ([33 + b % 5 for b in range(65)], [40 + 2 * b for b in range(65)], 4, 4, 96, 32, BF16, 0, 0.0),
    ([40] * 32, [300 - 5 * b for b in range(32)], 16, 8, 128, 64, F16, 0, 0.0),
    ([40] * 32, [300 - 5 * b for b in range(32)], 16, 8, 128, 64, BF16, 70, 0.0),
]


@pytest.mark.parametrize("kernel", ["many_rows", "few_rows"])
@pytest.mark.parametrize("news,lens,hq,hkv,dim,page,dtype,window,cap", CASES)
def test_attention(kernel, news, lens, hq, hkv, dim, page, dtype, window, cap):
    q = lib()
    print(f"kernel {kernel} news={news[:3]} lens={lens[:3]} dim={dim} {dtype}", flush=True)
    with q.forced_kv_kernel(kernel):
        cache = q.kv_cache(1, page, hkv, dim)
        plan = q.kv_attention_plan(cache, len(news), sum(news), hq, max(news), max(lens), dtype, window)
        assert plan["kernel"] == kernel
        run(q, news, lens, hq, hkv, dim, page, dtype, window, cap, seed=dim + hq)


@pytest.mark.parametrize("kernel", ["many_rows", "few_rows"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_bad_pages_and_rows_before_place_0(kernel, dtype):
    """Rows that see nothing give zeros and a page outside the cache hides its tokens only."""
    q = lib()
    print(f"kernel {kernel} rows that see nothing {dtype}", flush=True)
    news, lens, hq, hkv, dim, page = [90, 80, 50], [100, 100, 100], 4, 2, 64, 32
    cache, table, ln, keys, values = fill(q, lens, hkv, dim, page, dtype, 2)
    table = table.cpu()
    table[1, :] = cache.pages + 7
    table[2, 1] = -1
    x = torch.randn(sum(news), hq, dim, generator=torch.Generator().manual_seed(7)).to(dtype)
    short = torch.tensor([news[0] - 1, 100, 100], dtype=torch.int32, device="cuda")
    with q.forced_kv_kernel(kernel):
        got = q.kv_attention(cache, x.cuda(), table.cuda(), offsets(news), short, max(news), 100).cpu()
    assert not got[0].any()
    assert not got[news[0]:news[0] + news[1]].any()
    seen = [torch.ones(100, dtype=torch.bool)]
    seen[0][32:64] = False
    want, bound = attention(x[-news[2]:], keys[2:], values[2:], [100], news[2:], seen=seen)
    check(got[-news[2]:], want, bound, "bad page in the middle")
    want, bound = attention(x[1:news[0]], [keys[0][:news[0] - 1]], [values[0][:news[0] - 1]], [news[0] - 1], [news[0] - 1])
    check(got[1:news[0]], want, bound, "rows after place 0")


@pytest.mark.parametrize("kernel", ["many_rows", "few_rows"])
def test_nan_queries_and_score_ranges(kernel):
    q = lib()
    print(f"kernel {kernel} nan and ranges", flush=True)
    for spread in (1e-6, 1.0, 60.0, 2000.0):
        cache, table, ln, keys, values = fill(q, [600], 2, 64, 64, F16, 3)
        x = (spread * torch.randn(100, 4, 64, generator=torch.Generator().manual_seed(5))).to(F16)
        bad = x.clone()
        bad[7, 2, 5] = float("nan")
        with q.forced_kv_kernel(kernel):
            got = q.kv_attention(cache, bad.cuda(), table, offsets([100]), ln, 100, 600).cpu()
        assert got[7, 2].isnan().all()
        x[7, 2] = 0
        want, bound = attention(x, keys, values, [600], [100])
        err = (got.double() - want).abs()
        err[7, 2] = 0
        assert (err <= bound).all(), f"spread {spread}"


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_rows_repeat_and_replay(dtype):
    """Two calls and three replays with eager work between them agree bit for bit, splits among them."""
    q = lib()
    print(f"many rows graph {dtype}", flush=True)
    news, lens, hq, hkv, dim = [120, 64], [900, 64], 8, 2, 128
    cache, table, ln, _, _ = fill(q, lens, hkv, dim, 64, dtype, 6)
    cu = offsets(news)
    x = torch.randn(sum(news), hq, dim, generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
    ws = torch.empty(max(q.kv_attention_workspace_bytes(cache, 2, sum(news), hq, 120, 900), 256), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    with q.forced_kv_kernel("many_rows"):
        assert q.kv_attention_plan(cache, 2, sum(news), hq, 120, 900, dtype)["splits"] > 1
        call = lambda: q.kv_attention(cache, x, table, cu, ln, 120, 900, out=out, workspace=ws)
        want = call().clone()
        assert torch.equal(call(), want)
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


def test_the_plan_takes_both_kernels():
    """The plain call's kernel by its sizes, and both agree within their bounds where they meet."""
    q = lib()
    print("plan", flush=True)
    small, large = q.kv_cache(1, 64, 8, 64), q.kv_cache(1, 64, 8, 128)
    assert q.kv_attention_plan(small, 1, 512, 32, 512, 512, F16)["kernel"] == "few_rows"
    assert q.kv_attention_plan(large, 64, 64, 32, 1, 16384, BF16)["kernel"] == "few_rows"
    assert q.kv_attention_plan(large, 3, 6144, 32, 2048, 8192, BF16) == {"kernel": "many_rows", "waves": 8, "splits": 1}
    run(q, [40] * 32, [300 - 5 * b for b in range(32)], 64, 8, 64, 64, BF16, seed=9)
