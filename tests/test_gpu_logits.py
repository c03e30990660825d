"""Rules on logits on the GPU against their definition, every step in fp32 as written: for equality."""
import pytest
import torch

from tests.gpu_helpers import lib
from tests.tree_model import ancestors, forest

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def model(logits, c):
    """The definition in torch's fp32 on the CPU; c: the call's arguments."""
    rows, v = logits.shape
    out = logits.float().clone()
    touched = torch.zeros(rows, dtype=torch.bool)
    cu = c["cu"].tolist() if c.get("cu") is not None else list(range(rows + 1))
    most = c.get("max_new", 1) if c.get("cu") is not None else 1
    value = lambda name, b, none: c[name][b] if c.get(name) is not None else torch.tensor(none)  # noqa: E731
    inside = lambda ids: [t for t in ids if 0 <= t < v]  # noqa: E731
    for b in range(len(cu) - 1):
        old, prompt = [], 0
        if c.get("history") is not None:
            n = min(max(int(c["history_lens"][b]), 0), c["history"].shape[1])
            old = c["history"][b, :n].tolist()
            prompt = int(value("prompt_lens", b, 0))
        m = min(cu[b + 1] - cu[b], most)
        ids = c["ids"][cu[b]:cu[b] + m].tolist() if c.get("ids") is not None else None
        paths = [list(range(i + 1)) for i in range(m)]
        if c.get("parents") is not None:
            paths = ancestors(c["parents"][cu[b]:cu[b] + m].tolist())
        for i in range(m):
            row = cu[b] + i
            touched[row] = True
            own = [ids[j] for j in paths[i]] if ids is not None else []
            seen, made = torch.zeros(v, dtype=torch.bool), torch.zeros(v)
            for t in inside(old + own):
                seen[t] = True
            for t in inside([t for j, t in enumerate(old) if j >= prompt] + own):
                made[t] += 1
            x = out[row]
            rep = value("repetition", b, 1.0)
            x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
            x = torch.where(made > 0, (x - value("frequency", b, 0.0) * made) - value("presence", b, 0.0), x)
            if c.get("bias") is not None:
                last = {t: w for t, w in zip(c["bias_ids"][b].tolist(), c["bias"][b]) if 0 <= t < v}
                for t, w in last.items():
                    x[t] = x[t] + w
            if c.get("mask") is not None:
                word = c["mask"][row].long()
                bits = (word[:, None] >> torch.arange(32)) & 1
                x = torch.where(bits.flatten()[:v] == 1, x, torch.tensor(float("-inf")))
            out[row] = x
    return out.to(logits.dtype), touched


def same(got, want):
    got, want = got.cpu(), want
    assert got.dtype == want.dtype and torch.equal(got.isnan(), want.isnan())
    off = (got != want) & ~want.isnan()
    assert not off.any(), [(i.tolist(), float(got[tuple(i)]), float(want[tuple(i)])) for i in off.nonzero()[:4]]


def case(batch, news, v, dtype, hist, seed, tree="near", **on):
    """Logits and arguments; `on` switches parts off by False."""
    g = torch.Generator().manual_seed(seed)
    rows = sum(news)
    ids = lambda *s: torch.randint(-2, v + 2, s, generator=g, dtype=torch.int32)  # noqa: E731
    some = lambda *s: torch.where(torch.rand(*s, generator=g) < 0.6, ids(*s) % min(v, 40), ids(*s))  # noqa: E731
    c = dict(cu=ints([sum(news[:b]) for b in range(batch + 1)]), max_new=max(news + [1]), ids=some(rows),
             parents=ints([p for b, m in enumerate(news) for p in forest(m, tree, b)]), history=some(batch, hist),
             history_lens=torch.randint(-1, hist + 3, (batch,), generator=g, dtype=torch.int32),
             prompt_lens=torch.randint(0, hist + 2, (batch,), generator=g, dtype=torch.int32),
             repetition=0.7 + torch.rand(batch, generator=g), presence=torch.randn(batch, generator=g),
             frequency=torch.randn(batch, generator=g), bias_ids=some(batch, 30), bias=torch.randn(batch, 30, generator=g),
             mask=torch.randint(-2 ** 31, 2 ** 31, (rows, (v + 31) // 32 + 1), generator=g).to(torch.int32))
    for name, keep in on.items():
        if not keep:
            c[name] = None
    return (4 * torch.randn(rows, v, generator=g)).to(dtype), c


def run(q, logits, c, **more):
    on = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in c.items()}
    return q.logits_adjust(logits.cuda(), **on, **more)


CASES = [
    # nodes of each sequence, vocabulary, type, history
    ([1], 1, F32, 1),
    ([1, 1, 1], 37, F16, 5),
    ([1] * 8, 32000, F32, 600),
    ([5, 1, 9], 4100, BF16, 100),
    ([16] * 4, 5000, F32, 300),
    ([33, 0, 20], 1023, F16, 1000),
    ([64, 40], 9999, F32, 64),
    ([3] * 70, 260, BF16, 20),
    ([16] * 8, 32000, F32, 2000),                # rows of a sequence share a count
    ([512], 1200, F32, 10),
]


@pytest.mark.parametrize("news,v,dtype,hist", CASES)
def test_everything_at_once(news, v, dtype, hist):
    q = lib()
    print(f"logits news={news[:4]} v={v} {dtype} history={hist}", flush=True)
    for tree in ("near", "wild"):
        logits, c = case(len(news), news, v, dtype, hist, seed=v, tree=tree)
        want, touched = model(logits, c)
        same(run(q, logits, c)[touched.cuda()], want[touched])


PARTS = ["ids", "history", "prompt_lens", "repetition", "presence", "frequency", "bias", "mask"]


@pytest.mark.parametrize("part", PARTS)
def test_each_part(part):
    """Each part alone, and all but it."""
    q = lib()
    for alone in (True, False):
        off = {p: (p == part) == alone for p in PARTS}
        if part in ("prompt_lens", "repetition", "presence", "frequency") and alone:
            off["history"] = True
        off["parents"] = off["ids"]
        off["bias_ids"] = off["bias"]
        logits, c = case(3, [6, 2, 3], 700, F32, 50, seed=3, **off)
        want, touched = model(logits, c)
        assert touched.all()
        same(run(q, logits, c), want)


def test_single_tokens_and_chains():
    """Rows of a sequence each (no cu), with and without their own tokens; drafts in a row (no parents)."""
    q = lib()
    for own in (False, True):
        logits, c = case(5, [1] * 5, 3000, F32, 40, seed=1, ids=own, parents=False, cu=False)
        same(run(q, logits, c), model(logits, c)[0])
    logits, c = case(3, [4, 1, 300], 3000, F16, 40, seed=1, parents=False)
    same(run(q, logits, c), model(logits, c)[0])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_pitches_and_in_place(dtype):
    """Rows off their alignment and apart, adjusted in place and into rows of another pitch; what stands
    between rows, behind the last sequence and past max_new stays."""
    q = lib()
    for v, pad in ((1001, 7), (1000, 1), (1000, 8)):
        logits, c = case(2, [5, 3], v, dtype, 20, seed=v)
        want, _ = model(logits, c)
        wide = torch.full((10, v + pad), 5.0, dtype=dtype, device="cuda")
        view = wide[:8, :v]
        view.copy_(logits)
        other = torch.full((10, v + 2 * pad), 7.0, dtype=dtype, device="cuda")
        on = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in c.items()}
        q.logits_adjust(view, **on, out=other[:8, :v])
        same(other[:8, :v], want)
        assert (other[:, v:] == 7).all() and (other[8:] == 7).all()
        q.logits_adjust(view, **on, out=view)
        same(view, want)
        assert (wide[:, v:] == 5).all() and (wide[8:] == 5).all()


def test_untouched_rows():
    q = lib()
    logits, c = case(3, [6, 4, 2], 500, F32, 20, seed=5)
    c["max_new"] = 3
    more = torch.cat([logits, torch.randn(4, 500)])
    for name in ("ids", "parents", "mask"):
        c[name] = torch.cat([c[name], torch.zeros(4, *c[name].shape[1:], dtype=torch.int32)])
    want, touched = model(more, c)
    assert touched.sum() == 8
    out = torch.full_like(more, 9.0).cuda()
    run(q, more, c, out=out)
    same(out[touched.cuda()], want[touched])
    assert (out[~touched.cuda()] == 9).all()


def test_values_that_are_not_finite():
    q = lib()
    logits, c = case(2, [3, 2], 400, F32, 60, seed=5, mask=False)
    logits[:, ::7], logits[:, 1::7], logits[:, 2::7] = float("nan"), float("inf"), float("-inf")
    same(run(q, logits, c), model(logits, c)[0])
    mask = torch.zeros(5, 13, dtype=torch.int32)                 # nothing is allowed, in NaN's places either
    got = run(q, logits, dict(c, mask=mask))
    assert (got == float("-inf")).all()


def test_no_rows():
    q = lib()
    got = q.logits_adjust(torch.empty(0, 50, device="cuda"))
    assert got.shape == (0, 50)


def test_captured_and_replayed():
    """Replays follow the history, its length and the mask that the tensors hold then."""
    q = lib()
    logits, c = case(4, [7, 3, 1, 9], 5000, F32, 80, seed=5)
    on = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in c.items()}
    x, out = logits.cuda(), torch.empty(20, 5000, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.logits_adjust(x, **on, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.logits_adjust(x, **on, out=out)
    for step in range(3):
        new, d = case(4, [7, 3, 1, 9], 5000, F32, 80, seed=50 + step)
        x.copy_(new)
        for k, t in d.items():
            if isinstance(t, torch.Tensor):
                on[k].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        same(out, model(new, d)[0])


def test_offsets_that_do_not_rise():
    """An offset above the next one's: the rows before it are its sequence's no more, and no other's."""
    q = lib()
    logits, c = case(4, [5, 4, 0, 0], 700, F32, 30, seed=11)
    c["cu"] = ints([0, 5, 9, 1, 9])
    out = torch.full((9, 700), 7.0, device="cuda")
    on = {k: (x.cuda() if isinstance(x, torch.Tensor) else x) for k, x in c.items()}
    q.logits_adjust(logits.cuda(), **on, out=out)
    one = {k: (x[:1] if k in ("repetition", "presence", "frequency", "history", "history_lens", "prompt_lens", "bias", "bias_ids",
                              "ids", "parents", "mask") else x) for k, x in c.items()}
    want, _ = model(logits[:1], dict(one, cu=ints([0, 1])))
    same(out[:1], want)                                           # the first row is the first sequence's still
    assert (out[1:] == 7.0).all()
