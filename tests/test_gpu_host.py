"""Serving calls marshalled in C++ against the same calls marshalled in Python: one result, one set of errors."""
import pytest
import torch

from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu
I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Python:
    """Leaves every call to Python."""

    def __getattr__(self, name):
        return lambda *a: None


def state(q, dtype=torch.bfloat16, caches=2):
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    s = dict(caches=[q.kv_cache(12, 64, 2, 64) for _ in range(caches)], table=ints([[3, 1, 7, 5], [2, 0, 4, 6]]),
             cu=ints([0, 5, 12]), lens=ints([130, 77]), parents=ints([-1, 0, 0, 1, 3, -1, 0, 1, 1, 2, 4, 4]), leaf=ints([4, 5]),
             q=rand(12, 6, 64), k=rand(12, 2, 64), v=rand(12, 2, 64))
    old = [ints([0, 130, 207]), ints([130, 77])]
    for c in s["caches"]:
        q.kv_append(c, rand(207, 2, 64), rand(207, 2, 64), s["table"], *old)
    return s


def rules(rows=12, v=333):
    g = torch.Generator().manual_seed(5)
    pick = lambda *n: torch.randint(0, v, n, generator=g, dtype=I32).cuda()  # noqa: E731
    return dict(cu=ints([0, 5, 12]), max_new=7, history=pick(2, 40), history_lens=ints([40, 13]), prompt_lens=ints([10, 13]),
                ids=pick(rows), parents=ints([-1, 0, 0, 1, 3, -1, 0, 1, 1, 2, 4, 4]), repetition=torch.tensor([1.5, 0.7]).cuda(),
                presence=torch.tensor([0.2, 0.3]).cuda(), frequency=torch.tensor([0.1, 0.0]).cuda(), bias_ids=pick(2, 9),
                bias=torch.randn(2, 9, generator=g).cuda(),
                mask=torch.randint(-2**31, 2**31 - 1, (rows, (v + 31) // 32), generator=g, dtype=I32).cuda())


def calls(q, where):
    """name -> a call of a fresh state; `where`: what else to pass (outputs, workspaces)."""
    def attend(parents, given):
        s = state(q)
        more = {}
        if given:
            more = dict(out=torch.empty_like(s["q"]), workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
        got = q.kv_attention(s["caches"][0], s["q"], s["table"], s["cu"], s["lens"], 7, 130, parents=s["parents"] if parents else None, **more)
        assert not given or got is more["out"]
        return got

    def moved(given):
        s = state(q)
        for c in s["caches"]:
            q.kv_append(c, s["k"], s["v"], s["table"], s["cu"], s["lens"])
        more = dict(kept=torch.empty(2, dtype=I32, device="cuda"), path=torch.empty(2, 7, dtype=I32, device="cuda")) if given else {}
        kept, path = q.kv_keep(s["caches"], s["parents"], s["leaf"], s["table"], s["cu"], s["lens"], 7, **more)
        return [kept, path, *[x for c in s["caches"] for x in q.kv_read(c, s["table"], s["cu"], s["lens"], 12)]]

    def adapted(fwd, given):
        g = torch.Generator().manual_seed(9)
        n, k, m = 96, 256, 20
        s = q.adapters(3, 8, n, k)
        for i in range(3):
            q.adapters_load(s, i, torch.randn(8, k, generator=g).cuda(), torch.randn(n, 8, generator=g).cuda(), 0.5)
        x, y, at = torch.randn(m, k, generator=g).cuda(), torch.randn(m, n, generator=g).cuda(), ints([0, 2, 1, -1] * 5)
        more = dict(out=torch.empty(m, n, device="cuda")) if given else {}
        if not fwd:
            return q.adapters_add(y, x, s, at, **more)
        w = q.pack(torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8).cuda(),
                   (0.01 + 0.01 * torch.rand(k // 32, n, generator=g)).half().cuda(), 32)
        return q.adapters_fwd(w, x, s, at, **more)

    def adjusted(given):
        x = torch.randn(12, 333, generator=torch.Generator().manual_seed(2)).cuda()
        return q.logits_adjust(x, **rules(), **(dict(out=x) if given else {}))

    return dict(causal=lambda: attend(False, False), causal_given=lambda: attend(False, True), tree=lambda: attend(True, False),
                tree_given=lambda: attend(True, True), moved=lambda: moved(False), moved_given=lambda: moved(True),
                add=lambda: adapted(False, False), add_given=lambda: adapted(False, True), fwd=lambda: adapted(True, False),
                fwd_given=lambda: adapted(True, True), logits=lambda: adjusted(False), logits_given=lambda: adjusted(True))[where]


NAMES = ["causal", "causal_given", "tree", "tree_given", "moved", "moved_given", "add", "add_given", "fwd", "fwd_given", "logits",
         "logits_given"]


@pytest.mark.parametrize("name", NAMES)
def test_the_same_as_from_python(name, monkeypatch):
    q = lib()
    native = calls(q, name)()
    monkeypatch.setattr(q.binding, "_host", Python())
    plain = calls(q, name)()
    if not isinstance(native, list):
        native, plain = [native], [plain]
    for a, b in zip(native, plain):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)


def test_regular_calls_do_not_come_back_to_python(monkeypatch):
    q = lib()
    s = state(q)

    def never(*a, **k):
        raise AssertionError("marshalled in Python")
    for name in ("_kv_seqs", "_token_rows", "_table", "_adapter_rows"):
        monkeypatch.setattr(q.binding, name, never)
    where = (s["table"], s["cu"], s["lens"])
    q.kv_append(s["caches"][0], s["k"], s["v"], *where)
    q.kv_tree_attention(s["caches"][0], s["q"], s["parents"], *where, 7, 130)
    q.kv_attention(s["caches"][0], s["q"], *where, 7, 130)
    q.kv_keep(s["caches"], s["parents"], s["leaf"], *where, 7)
    q.kv_read(s["caches"][0], *where, 12)
    q.logits_adjust(torch.randn(12, 333, device="cuda"), **rules())


def test_tensors_that_have_to_be_copied():
    """Strided arguments take the way through Python and give the same."""
    q = lib()
    s = state(q)
    where = (s["table"], s["cu"], s["lens"])
    want = q.kv_tree_attention(s["caches"][0], s["q"], s["parents"], *where, 7, 130)
    apart = torch.empty(12, 64, 6, dtype=s["q"].dtype, device="cuda").transpose(1, 2)
    apart.copy_(s["q"])
    up = torch.stack([s["parents"], s["parents"]], 1)[:, 0]
    assert torch.equal(q.kv_tree_attention(s["caches"][0], apart, up, *where, 7, 130), want)
    fused = torch.empty(12, 10, 64, dtype=s["q"].dtype, device="cuda")                 # a slice of a fused projection
    fused[:, :6] = s["q"]
    assert torch.equal(q.kv_tree_attention(s["caches"][0], fused[:, :6], s["parents"], *where, 7, 130), want)


def test_refusals_are_the_librarys_and_pythons():
    q = lib()
    s = state(q)
    where = (s["table"], s["cu"], s["lens"])
    for kw in (dict(max_new=513, max_ctx=600), dict(max_new=7, max_ctx=130, softcap=float("nan")), dict(max_new=7, max_ctx=130, softcap=-1.0)):
        with pytest.raises(q.Q4gswError):
            q.kv_tree_attention(s["caches"][0], s["q"], s["parents"], *where, **kw)
    with pytest.raises((q.Q4gswError, ValueError)):
        q.kv_tree_attention(s["caches"][0], s["q"], s["parents"], *where, 7, 130, window=-1)
    with pytest.raises(ValueError):
        q.kv_tree_attention(s["caches"][0], s["q"], s["parents"], *where, 1 << 31, 130)
    with pytest.raises(ValueError):
        q.kv_tree_attention(s["caches"][0], s["q"], s["parents"].long(), *where, 7, 130)
    with pytest.raises(q.Q4gswError):
        q.kv_tree_attention(s["caches"][0], s["q"], s["parents"], *where, 7, 130, out=s["q"])          # out over q
    with pytest.raises(q.Q4gswError):
        q.kv_tree_attention(s["caches"][0], s["q"], s["parents"], *where, 7, 1 << 20, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(q.Q4gswError):
        q.kv_keep([s["caches"][0]] * 2, s["parents"], s["leaf"], *where, 7)                            # one cache twice
    with pytest.raises(q.Q4gswError):
        q.kv_keep(s["caches"], s["parents"], s["leaf"], *where, 7, kept=s["lens"])                     # an output over an input
    x = torch.randn(12, 333, device="cuda")
    with pytest.raises(ValueError):
        q.logits_adjust(x, ids=torch.zeros(11, dtype=I32, device="cuda"))
    with pytest.raises(ValueError):
        q.logits_adjust(x, parents=torch.zeros(12, dtype=I32, device="cuda"))
    with pytest.raises(q.Q4gswError):
        q.logits_adjust(x[:, :300], out=x[:, 20:320])                                                  # out over the logits, shifted


def step(q, s, a, x, y, at, logits, more):
    """One step's calls on the current stream; nothing is written that another step reads."""
    where = (s["table"], s["cu"], s["lens"])
    return [q.kv_tree_attention(s["caches"][0], s["q"], s["parents"], *where, 7, 130), q.adapters_add(y, x, a, at),
            q.logits_adjust(logits, **more)]


def steps(q, seed):
    g = torch.Generator().manual_seed(seed)
    n, k, m = 320, 512, 40
    a = q.adapters(6, 16, n, k)
    for i in range(6):
        q.adapters_load(a, i, torch.randn(16, k, generator=g).cuda(), torch.randn(n, 16, generator=g).cuda(), 0.5)
    return (q, state(q), a, torch.randn(m, k, generator=g).cuda(), torch.randn(m, n, generator=g).cuda(),
            torch.randint(-1, 6, (m,), generator=g, dtype=I32).cuda(), torch.randn(12, 333, generator=g).cuda(), rules())


def test_two_streams_at_once():
    q = lib()
    both = [steps(q, i) for i in range(2)]
    want = [step(*b) for b in both]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for b, stream, out in zip(both, streams, got):
            with torch.cuda.stream(stream):
                out.append(step(*b))
    torch.cuda.synchronize()
    for w, out in zip(want, got):
        for one in out:
            assert all(torch.equal(x, y) for x, y in zip(w, one))


def test_two_threads_at_once():
    import threading
    q = lib()
    both = [steps(q, i) for i in range(2)]
    want = [step(*b) for b in both]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i].append(step(*both[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:                                     # shown by the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for w, out in zip(want, got):
        assert len(out) == 20
        for one in out:
            assert all(torch.equal(x, y) for x, y in zip(w, one))


def test_captured_without_outputs():
    """Outputs and workspaces that the calls allocate themselves live in the graph's memory."""
    q = lib()
    args = steps(q, 4)
    want = step(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*args)
    for _ in range(3):
        for x in got:
            x.zero_()
        junk = torch.randn(1 << 20, device="cuda")                 # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        del junk
