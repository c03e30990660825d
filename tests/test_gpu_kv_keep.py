"""Accepted paths moved together in the paged 4-bit cache, against their definition: whole codes and scales
move, so the comparison is for equality, of every byte that is not moved too."""
import pytest
import torch

from tests.gpu_helpers import lib
from tests.serving_model import kv_values
from tests.test_gpu_kv_cache import build
from tests.tree_model import ancestors, forest

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def model(values, trees, lens, leaves, most):
    """(kept, path, values [per sequence]) after the move; values: [n, heads, dim] of every sequence."""
    kept, paths, out = [], [], []
    for x, tree, n, leaf in zip(values, trees, lens, leaves):
        p0 = n - len(tree)
        path = ancestors(tree)[leaf] if 0 <= leaf < min(len(tree), most) else []
        y = x.clone()
        for k, j in enumerate(path):
            if p0 + k >= 0:
                y[p0 + k] = x[p0 + j]
        kept.append(max(p0 + len(path), 0))
        paths.append(path + [-1] * (most - len(path)))
        out.append(y)
    return kept, paths, out


def filled(q, lens, heads, dim, page, seed):
    """A cache of whole sequences, and what it stands for: (keys, values) per sequence in fp32."""
    cache, table, cu, ln, k, v = build(q, lens, lens, heads, dim, page, torch.float16, seed)
    q.kv_append(cache, k.cuda(), v.cuda(), table, cu, ln)
    at = [sum(lens[:b]) for b in range(len(lens) + 1)]
    cut = lambda x: [kv_values(x[a:b]).float() for a, b in zip(at, at[1:])]
    return cache, table, cu, ln, cut(k), cut(v)


def check(q, caches, table, cu, ln, want):
    for cache, (k, v) in zip(caches, want):
        gk, gv = q.kv_read(cache, table, cu, ln, sum(len(x) for x in k))
        assert torch.equal(gk.cpu(), torch.cat(k)) and torch.equal(gv.cpu(), torch.cat(v))


CASES = [
    # nodes, lengths, kind, leaf (-1: none, "last", "mid", "root"), heads, dim, page, caches
    ([1], [1], "roots", "last", 1, 64, 32, 1),
    ([13, 7], [70, 40], "near", "last", 8, 128, 64, 2),
    ([40, 33, 5], [163, 33, 64], "far", "last", 2, 96, 32, 1),
    ([64, 64], [95, 300], "near", "mid", 3, 256, 128, 3),
    ([20, 20, 20], [52, 20, 100], "chain", "last", 2, 192, 64, 1),       # all in place: nothing moves
    ([30, 30], [60, 61], "star", "last", 1, 64, 32, 2),
    ([25, 9], [60, 61], "wild", "mid", 2, 64, 32, 1),
    ([512, 130], [700, 131], "near", "last", 2, 64, 64, 1),
    ([512], [512], "chain", "mid", 1, 128, 32, 1),
    ([6] * 70, list(range(6, 76)), "near", "last", 2, 64, 32, 2),
]


@pytest.mark.parametrize("nodes,lens,kind,which,heads,dim,page,count", CASES)
def test_against_the_definition(nodes, lens, kind, which, heads, dim, page, count):
    q = lib()
    print(f"kv keep nodes={nodes[:4]} lens={lens[:4]} {kind} {which} heads={heads} dim={dim} page={page} {count} caches", flush=True)
    trees = [forest(n, kind, b) for b, n in enumerate(nodes)]
    leaves = [{"last": n - 1, "mid": n // 2, "root": 0}[which] for n in nodes]
    sets = [filled(q, lens, heads, dim, page, seed=dim + i) for i in range(count)]
    table, whole, ln = sets[0][1:4]
    # one table for all caches
    caches = []
    for cache, tb, _, _, k, v in sets:
        q.kv_append(cache, torch.cat(k).cuda(), torch.cat(v).cuda(), table, whole, ln)
        caches.append(cache)
    stored = [tuple([kv_values(x).float() for x in y] for y in (k, v)) for *_, k, v in sets]
    cu = ints([sum(nodes[:b]) for b in range(len(nodes) + 1)])
    most = max(nodes)
    kept, path = q.kv_keep(caches if count > 1 else caches[0], ints([p for t in trees for p in t]), ints(leaves), table, cu, ln, most)
    torch.cuda.synchronize()
    want = []
    for k, v in stored:
        wk, wp, mk = model(k, trees, lens, leaves, most)
        want.append((mk, model(v, trees, lens, leaves, most)[2]))
    assert kept.tolist() == wk and path.tolist() == wp
    check(q, caches, table, whole, ln, want)


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_every_other_byte_stays(dim):
    """Only the destinations' codes and scales change: the buffer is compared with one in which the moved
    rows were stored by kv_append at their new places (stored values are their own codes)."""
    q = lib()
    lens, nodes = [75, 41], [30, 41]
    trees = [forest(30, "near", 1), forest(41, "far", 2)]
    cache, table, whole, ln, k, v = filled(q, lens, 2, dim, 32, 9)
    before = cache.buffer.clone()
    leaves = [29, 40]
    cu = ints([0, 30, 71])
    kept, _ = q.kv_keep(cache, ints(trees[0] + trees[1]), ints(leaves), table, cu, ln, 64)
    changed = cache.buffer != before
    _, _, mk = model(k, trees, lens, leaves, 64)
    _, _, mv = model(v, trees, lens, leaves, 64)
    check(q, [cache], table, whole, ln, [(mk, mv)])
    paths = [ancestors(t)[leaf] for t, leaf in zip(trees, leaves)]
    moved = sum(sum(j != i for i, j in enumerate(p)) for p in paths)
    assert moved > 0
    # at most: a token's keys' words and scales whole, and the bytes that hold its values' nibbles
    assert int(changed.sum()) <= moved * 2 * (dim // 2 + dim + 4 * (dim // 32))
    assert kept.tolist() == [45 + len(paths[0]), len(paths[1])]


def test_leaves_outside_the_tree():
    q = lib()
    lens, nodes = [50, 40, 30, 20], [10, 10, 10, 0]
    trees = [forest(10, "near", b) for b in range(3)] + [[]]
    cache, table, whole, ln, k, v = filled(q, lens, 1, 64, 32, 3)
    before = cache.buffer.clone()
    cu = ints([0, 10, 20, 30, 30])
    up = ints([p for t in trees for p in t])
    kept, path = q.kv_keep(cache, up, ints([-1, 10, 2 ** 31 - 1, 0]), table, cu, ln, 16)
    assert kept.tolist() == [40, 30, 20, 20] and (path == -1).all()
    kept, path = q.kv_keep(cache, up, ints([9, 4, 3, 0]), table, cu, ln, 3)      # nodes past max_new
    assert kept.tolist() == [40, 30, 20, 20] and (path == -1).all() and path.shape == (4, 3)
    assert torch.equal(cache.buffer, before)


def test_no_tokens_at_all():
    q = lib()
    cache, table, whole, ln, k, v = filled(q, [50, 40], 1, 64, 32, 3)
    kept, path = q.kv_keep(cache, ints([]), ints([0, 5]), table, ints([0, 0, 0]), ln, 4)
    assert kept.tolist() == [50, 40] and (path == -1).all()


def test_places_without_pages():
    """Nodes on no page come as zeros, destinations on none are not stored, places before 0 are none."""
    q = lib()
    lens = [70, 20]
    trees = [[-1] + [0] * 29 + [5] * 10, [-1] + list(range(29))]                 # 40 and 30 nodes
    cache, table, whole, ln, k, v = filled(q, lens, 2, 64, 32, 7)
    k, v = [x.clone() for x in k], [x.clone() for x in v]
    holes = table.clone()
    holes[0, 2] = -1                                                             # places 64 .. 69 of sequence 0
    leaves = [39, 25]                                                            # place 69; a chain: in place
    kept, path = q.kv_keep(cache, ints(trees[0] + trees[1]), ints(leaves), holes, ints([0, 40, 70]), ln, 40)
    assert kept.tolist() == [33, 16]
    assert path[0, :4].tolist() == [0, 5, 39, -1]
    for x in (k, v):
        x[0][31], x[0][32] = x[0][35].clone(), 0.0
    check(q, [cache], table, whole, ln, [(k, v)])


def test_captured_and_replayed():
    """Append, attention-free step and move in a graph: replays give what eager calls give."""
    q = lib()
    lens, nodes = [75, 41], [12, 9]
    caches = [filled(q, lens, 2, 64, 32, 9)]
    cache, table, whole, ln, _, _ = caches[0]
    other = q.kv_cache(cache.pages, 32, 2, 64)
    other.buffer.copy_(cache.buffer)
    cu = ints([0, 12, 21])
    k, v = (torch.randn(21, 2, 64, generator=torch.Generator().manual_seed(i)).half().cuda() for i in (1, 2))
    up, leaf = ints([-1] * 21), ints([0, 0])
    kept, path = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, 12, dtype=torch.int32, device="cuda")

    def step(c, kept, path):
        q.kv_append(c, k, v, table, cu, ln)
        q.kv_keep(c, up, leaf, table, cu, ln, 12, kept=kept, path=path)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, kept, path)
    torch.cuda.current_stream().wait_stream(side)
    other.buffer.copy_(cache.buffer)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, kept, path)
    for i in range(4):
        up.copy_(ints(forest(12, "near", i) + forest(9, "far", i)))
        leaf.copy_(ints([11 - i, 8 - i]))
        k.mul_(-1.25)
        graph.replay()
        torch.cuda.synchronize()
        k2, p2 = torch.empty_like(kept), torch.empty_like(path)
        step(other, k2, p2)
        torch.cuda.synchronize()
        assert torch.equal(cache.buffer, other.buffer) and torch.equal(kept, k2) and torch.equal(path, p2), i
