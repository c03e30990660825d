"""Attention of trees of drafted tokens over the 4-bit cache on the GPU against its formula in 64 bits.

Bounds as in test_gpu_kv_attention.py: element by element the roundings that the call documents, over a
call rms errors of 2^-9 (16-bit and fp32 outputs) and 2^-8 (bf16).  What a row sees or does not see moves
whole weights: outputs are averages over dozens of values of size one, and a key too many or too few
moves a row of a short sequence by far more than its bound.
"""
import pytest
import torch

from tests.gpu_helpers import lib
from tests.serving_model import kv_values
from tests.test_gpu_kv_attention import BF16, F16, F32, check, fill, offsets
from tests.test_gpu_kv_cache import build
from tests.tree_model import forest, tree_attention

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(q, trees, lens, hq, hkv, dim, page, dtype, window=0, cap=0.0, seed=0, kernel=None, spread=1.5):
    cache, table, ln, keys, values = fill(q, lens, hkv, dim, page, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    news = [len(t) for t in trees]
    x = (spread * torch.randn(sum(news), hq, dim, generator=g)).to(dtype)
    args = (cache, x.cuda(), ints([p for t in trees for p in t]), table, offsets(news), ln, max(max(news), 1), max(lens))
    if kernel:
        with q.forced_kv_kernel(kernel):
            got = q.kv_tree_attention(*args, window=window, softcap=cap)
    else:
        got = q.kv_tree_attention(*args, window=window, softcap=cap)
    torch.cuda.synchronize()
    want, bound = tree_attention(x, keys, values, trees, lens, window, cap)
    check(got, want, bound, f"news={news[:4]} lens={lens[:4]} hq={hq} hkv={hkv} dim={dim} page={page} {dtype} w={window} "
                            f"c={cap} {kernel}")
    return got


CASES = [
    # nodes, lengths, kind of tree, hq, hkv, dim, page, dtype, window, cap
    ([1], [1], "roots", 1, 1, 64, 32, F16, 0, 0.0),
    ([13], [521], "near", 32, 8, 64, 64, BF16, 0, 0.0),
    ([16, 9, 1, 5], [700, 9, 31, 64], "far", 8, 2, 128, 64, F16, 0, 0.0),
    ([32], [32], "far", 2, 1, 64, 32, F32, 0, 0.0),              # nothing before the tree
    ([33], [40], "star", 4, 4, 96, 32, BF16, 0, 0.0),
    ([31, 64], [95, 64], "roots", 3, 1, 128, 64, F16, 0, 30.0),
    ([26, 14], [1500, 700], "near", 16, 4, 256, 64, BF16, 100, 50.0),
    ([20, 20], [60, 21], "chain", 6, 1, 192, 128, F16, 7, 0.0),
    ([40, 40], [60, 41], "far", 6, 3, 64, 32, F16, 3, 0.0),      # windows that end inside the tree
    ([7], [3000], "wild", 20, 1, 128, 64, F32, 0, 0.0),
    ([50, 3], [2100, 100], "wild", 5, 5, 64, 64, BF16, 1, 0.0),  # every node sees itself alone
    ([200], [333], "near", 4, 1, 64, 64, F16, 0, 0.0),
    ([130, 64], [130, 900], "far", 8, 2, 128, 64, BF16, 0, 0.0),
    ([512], [600], "far", 1, 1, 64, 64, F16, 0, 0.0),            # the most nodes, one row a node
    ([512, 500], [512, 1333], "near", 2, 2, 128, 64, F32, 20, 0.0),
    ([300], [301], "chain", 4, 2, 256, 32, F16, 0, 0.0),
    ([3] * 70, list(range(3, 73)), "near", 4, 2, 64, 32, BF16, 0, 0.0),
]


@pytest.mark.parametrize("nodes,lens,kind,hq,hkv,dim,page,dtype,window,cap", CASES)
def test_against_the_formula(nodes, lens, kind, hq, hkv, dim, page, dtype, window, cap):
    q = lib()
    trees = [forest(n, kind, b) for b, n in enumerate(nodes)]
    run(q, trees, lens, hq, hkv, dim, page, dtype, window, cap, seed=dim + nodes[0])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kernel", ["few_rows", "tree", "many_rows"])
def test_every_kernel(kernel, dim, dtype):
    """Every instance, at places where a tree begins and ends inside a block, with and without a window."""
    q = lib()
    for lens, window in (([70, 97, 33], 0), ([66, 95, 40], 9)):
        run(q, [forest(n, "far", n) for n in (37, 21, 33)], lens, 4, 2, dim, 32, dtype, window, seed=dim, kernel=kernel)


@pytest.mark.parametrize("kernel", ["few_rows", "tree", "many_rows"])
@pytest.mark.parametrize("group", [1, 3, 8, 40])
@pytest.mark.parametrize("start", [0, 1, 31, 32, 63])
def test_places_of_the_tree(start, group, kernel):
    """Trees that begin at every kind of place in a block, rows of one node in unlike tiles."""
    q = lib()
    run(q, [forest(66, "near", start), forest(35, "far", start)], [66 + start, 35 + 64 + start], group, 1, 64, 64, F16, seed=start,
        kernel=kernel)


@pytest.mark.parametrize("kernel,news,lens,hq,hkv,dim,same", [
    ("few_rows", [4, 2], [700, 64], 8, 2, 128, False), ("few_rows", [16, 9], [90, 333], 3, 3, 64, True),
    ("few_rows", [4, 2], [500, 64], 8, 2, 128, True),
    ("many_rows", [9, 4], [700, 64], 8, 2, 128, True), ("many_rows", [70, 33], [200, 400], 4, 1, 64, True)])
def test_a_chain_is_causal_attention(kernel, news, lens, hq, hkv, dim, same):
    """Parents i - 1 give kv_attention's output: bit for bit where one kernel with one plan serves both (the same
    products in the same order), else within the bound of either (trees split long caches less)."""
    q = lib()
    cache, table, ln, keys, values = fill(q, lens, hkv, dim, 64, F16, 3)
    x = torch.randn(sum(news), hq, dim, generator=torch.Generator().manual_seed(1)).half().cuda()
    where = (table, offsets(news), ln, max(news), max(lens))
    with q.forced_kv_kernel(kernel):
        want = q.kv_attention(cache, x, *where)
        got = q.kv_tree_attention(cache, x, ints([i - 1 for n in news for i in range(n)]), *where)
    if same:
        assert torch.equal(got, want)
    bound = tree_attention(x.cpu(), keys, values, [forest(n, "chain") for n in news], lens)[1]
    assert float(((got.double() - want.double()).abs().cpu() / bound).max()) <= 2


def test_rows_without_keys_and_hidden_pages():
    """Nodes whose places are before 0 or on no page, and a prefix without pages: what is left counts, rows
    that see nothing give zeros."""
    q = lib()
    lens, trees = [70, 20], [forest(20, "near", 1), forest(30, "far", 2)]           # more nodes than tokens
    cache, table, ln, keys, values = fill(q, lens, 2, 64, 32, F16, 5)
    table = table.clone()
    table[0, 0] = -1                                                              # the first page of sequence 0
    table[0, 2] = 10 ** 6                                                         # its last one: places 64 .. 69
    x = torch.randn(50, 8, 64, generator=torch.Generator().manual_seed(2)).half()
    where = (table, offsets([20, 30]), ln, 30, 70)
    paged = [torch.tensor([32 <= t < 64 for t in range(70)]), torch.ones(20, dtype=torch.bool)]
    want, bound = tree_attention(x, keys, values, trees, lens, paged=paged)
    for kernel in ("few_rows", "tree", "many_rows"):
        with q.forced_kv_kernel(kernel):
            got = q.kv_tree_attention(cache, x.cuda(), ints(trees[0] + trees[1]), *where)
        check(got, want, bound, f"hidden {kernel}")
        assert (got[20:30] == 0).all()                                            # places -10 .. -1


@pytest.mark.parametrize("kernel", ["few_rows", "tree", "many_rows"])
@pytest.mark.parametrize("dim,dtype,window", [(128, F16, 0), (64, BF16, 0), (256, F32, 0), (96, BF16, 7000)])
def test_a_split_cache(kernel, dim, dtype, window):
    """Long caches of few rows split the keys; the join and a poisoned workspace."""
    q = lib()
    trees, lens = [forest(9, "near", 1), forest(5, "far", 2)], [9000, 300]
    cache, table, ln, keys, values = fill(q, lens, 1, dim, 64, dtype, 5)
    x = torch.randn(14, 8, dim, generator=torch.Generator().manual_seed(2)).to(dtype)
    need = q.kv_tree_attention_workspace_bytes(cache, 2, 14, 8, 9, 9000)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    with q.forced_kv_kernel(kernel):
        got = q.kv_tree_attention(cache, x.cuda(), ints(trees[0] + trees[1]), table, offsets([9, 5]), ln, 9, 9000, window=window,
                                  workspace=ws)
    want, bound = tree_attention(x, keys, values, trees, lens, window)
    check(got, want, bound, f"split {kernel} {dim}")


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scales_that_rise_and_fall(dim, dtype):
    """Values whose scales differ by 2^30 along the cache, in either order, and scores that climb far: the running
    references move, and what was summed before stays in range."""
    q = lib()
    n, m = 200, 24
    cache, table, cu, ln, k, v = build(q, [n], [n], 1, dim, 64, torch.float32, 3)
    for order in (1, -1):
        size = torch.logspace(-6, 3, n)[:, None, None]
        size = size if order == 1 else size.flip(0)
        kk, vv = k * (0.2 + 0.02 * torch.arange(n))[:, None, None], v * size
        q.kv_append(cache, kk.cuda(), vv.cuda(), table, cu, ln)
        x = torch.randn(m, 4, dim, generator=torch.Generator().manual_seed(2)).to(dtype)
        tree = forest(m, "near", 3)
        want, bound = tree_attention(x, [kv_values(kk)], [kv_values(vv)], [tree], [n])
        for kernel in ("few_rows", "tree", "many_rows"):
            with q.forced_kv_kernel(kernel):
                got = q.kv_tree_attention(cache, x.cuda(), ints(tree), table, offsets([m]), ln, m, n).cpu().double()
            # the roundings of weights are relative to their products with scales: of the largest in the row's sum
            assert torch.isfinite(got).all()
            assert float(((got - want).abs() / bound).max()) <= 1, (kernel, order)


def test_queries_that_are_not_finite():
    q = lib()
    trees, lens = [forest(12, "near", 1)], [80]
    cache, table, ln, keys, values = fill(q, lens, 1, 64, 32, F16, 5)
    x = torch.randn(12, 4, 64, generator=torch.Generator().manual_seed(2)).half()
    x[3, 1, 7], x[5, 0, 0] = float("nan"), float("inf")
    got = q.kv_tree_attention(cache, x.cuda(), ints(trees[0]), table, offsets([12]), ln, 12, 80).cpu()
    bad = torch.zeros(12, 4, dtype=torch.bool)
    bad[3, 1] = bad[5, 0] = True
    assert got[bad].isnan().all() and not got[~bad].isnan().any()


def test_strides_and_rows_behind_the_last_sequence():
    q = lib()
    trees, lens = [forest(12, "near", 1), forest(6, "far", 1)], [80, 50]
    cache, table, ln, keys, values = fill(q, lens, 2, 64, 32, BF16, 5)
    wide = torch.randn(25, 3, 4, 64, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    x = wide[:, 1]                                                                # a slice of a fused projection
    up = torch.full((25, 2), 99, dtype=torch.int32, device="cuda")
    up[:18, 0] = ints(trees[0] + trees[1])
    out = torch.full((25, 4, 64), 7.0, dtype=BF16, device="cuda")
    q.kv_tree_attention(cache, x, up[:, 0], table, offsets([12, 6]), ln, 12, 80, out=out)
    want, bound = tree_attention(x[:18].cpu(), keys, values, trees, lens)
    check(out[:18], want, bound, "strides")
    assert (out[18:] == 7.0).all()


def test_captured_and_replayed():
    """A graph's replays follow the tree, the lengths and the table that its tensors hold then."""
    q = lib()
    lens = [300, 90]
    cache, table, ln, keys, values = fill(q, lens, 2, 64, 32, F16, 5)
    x = torch.randn(20, 4, 64, generator=torch.Generator().manual_seed(2)).half().cuda()
    up, cu = ints([-1] * 20), offsets([12, 8])
    out = torch.empty_like(x)
    ws = torch.empty(q.kv_tree_attention_workspace_bytes(cache, 2, 20, 4, 12, 300), dtype=torch.uint8, device="cuda")
    call = lambda: q.kv_tree_attention(cache, x, up, table, cu, ln, 12, 300, out=out, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):
        trees = [forest(12, "near", step), forest(8, "far", step)]
        now = [lens[0] - 7 * step, lens[1] - 30 * step]
        up.copy_(ints(trees[0] + trees[1]))
        ln.copy_(ints(now))
        graph.replay()
        torch.cuda.synchronize()
        want, bound = tree_attention(x.cpu(), [k[:n] for k, n in zip(keys, now)], [v[:n] for v, n in zip(values, now)], trees, now)
        check(out, want, bound, f"replay {step}")
