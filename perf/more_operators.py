"""Operators of a serving step with drafted tokens and many adapters, as cases to time and compare.

Four operators beside the 4-bit linear layer and the paged 4-bit cache (pages of tokens, fp16 scale
per run of 32 channels, see _quantise):

  tree      attention of a tree of drafted tokens over the cache: the newest m tokens of a sequence of n
            are nodes of a tree (parents[i] < i in the sequence's own count, anything else: a root).  A
            node sees the n - m tokens before the tree, its ancestors and itself; with a window w only
            those whose position is above its own minus w, a node's position being n - m + its depth.
  keep      the accepted path of each tree in a row: the nodes on the way to leaf[b] move to places n - m,
            n - m + 1, ... of the cache, in the caches of several layers at once.  A pass stores the
            drafts' keys and values first, as a step does, and reads them back at the end.
  adapters  y[m] = x[m] W^T + alpha_s (x[m] A_s^T) B_s^T, s = slot[m]: low-rank adapters of many requests
            beside one 4-bit weight ("fwd"), or added to a projection that was computed otherwise ("add").
  logits    logits of single tokens or of a tree's nodes: tokens seen so far divided (or multiplied) by
            a penalty, generated ones lowered by their count, biases added, a grammar's mask applied.

`run` takes plain torch operations where `own` is false and the package's calls where it is true.
"""
import random

import torch

own = False

P = 64                      # tokens per cache page
G = 32                      # channels per scale of the cache, columns per scale of a weight
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---- cases -----------------------------------------------------------------------------------
def _tree(name, batch, nodes, ctx, hq, hkv, dim, dtype, ragged=False, window=0, cap=0.0):
    return dict(name=name, op="tree", batch=batch, nodes=nodes, ctx=ctx, hq=hq, hkv=hkv, dim=dim, dtype=dtype,
                ragged=ragged, window=window, cap=cap)


def _keep(name, batch, nodes, ctx, hkv, dim, dtype, caches, ragged=False):
    return dict(name=name, op="keep", batch=batch, nodes=nodes, ctx=ctx, hkv=hkv, dim=dim, dtype=dtype, caches=caches,
                ragged=ragged)


def _adapters(name, how, rows, cols, outs, rank, slots, xtype, ftype, runs=False):
    return dict(name=name, op="adapters", how=how, rows=rows, cols=cols, outs=outs, rank=rank, slots=slots, xtype=xtype,
                ftype=ftype, runs=runs)


def _logits(name, batch, nodes, vocab, history, dtype, bias=0, mask=False, ragged=False):
    return dict(name=name, op="logits", batch=batch, nodes=nodes, vocab=vocab, history=history, dtype=dtype, bias=bias,
                mask=mask, ragged=ragged)


def listed():
    return [
        # one user, a small tree, a short conversation, in the geometry of the QKV triple 2048 / 512 / 512: latency
        _tree("tree_one", 1, 13, 521, 32, 8, 64, "bf16"),
        # a server's batch of unlike lengths, trees of up to 16 nodes
        _tree("tree_batch", 16, 16, 4096, 32, 8, 128, "fp16", ragged=True),
        # two long documents with wide trees: the cache's length has to be split
        _tree("tree_long", 2, 64, 131072, 32, 8, 128, "bf16"),
        # wide heads, a sliding window and capped scores
        _tree("tree_window", 8, 26, 8191, 16, 4, 256, "bf16", ragged=True, window=1024, cap=50.0),
        # the accepted paths of a few sequences in two layers' caches
        _keep("keep_few", 4, 13, 700, 8, 64, "bf16", 2),
        # a large batch with wide trees, in four layers' caches
        _keep("keep_batch", 64, 61, 4099, 8, 128, "fp16", 4, ragged=True),
        # one token of one request: the latency of a call
        _adapters("adapters_one", "fwd", 1, 2048, 2048, 16, 8, "bf16", "bf16"),
        # one token each of 64 requests with 32 adapters among them, at the MLP's up projection
        _adapters("adapters_batch", "fwd", 64, 2048, 8192, 16, 32, "bf16", "bf16"),
        # the same beside a projection of int8 rows, whose norm's rows are fp32
        _adapters("adapters_beside", "add", 61, 8192, 2048, 32, 48, "fp32", "fp16"),
        # prompts of four requests, packed one after the other
        _adapters("adapters_prompt", "fwd", 2048, 2048, 8192, 16, 4, "bf16", "bf16", runs=True),
        # greedy decoding of a small batch: fp32 logits of the int8 linear over a small vocabulary
        _logits("logits_step", 8, 1, 32000, 600, "fp32"),
        # trees over a large vocabulary, with grammars and biased tokens
        _logits("logits_tree", 8, 16, 128256, 4096, "fp32", bias=40, mask=True, ragged=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "keep", "adapters", "adapters", "adapters", "logits", "logits"])
    dtype = rng.choice(["bf16", "fp16"])
    hkv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 64, 96, 128, 128, 128, 192, 256])
    group = rng.choice([1, 2, 3, 4, 4, 6, 8])
    window = rng.choice([0, 0, 0, _spread(rng, 4, 4096)])
    cap = rng.choice([0.0, 0.0, 0.0, 30.0, 50.0])
    ragged = rng.random() < 0.7
    if kind == "tree":
        nodes = _spread(rng, 1, 200)
        ctx = nodes + rng.choice([0, _spread(rng, 1, 131072), _spread(rng, 1, 131072)])
        # products and cache at most a quarter of tree_long's
        while ctx > nodes and nodes * ctx * hkv * group * dim > 64 * 131072 * 32 * 128 // 4:
            ctx = max(nodes, ctx // 2)
        most = min(64 * 131072 * 32 * 128 // 4 // (nodes * ctx * hkv * group * dim), 2 * 131072 * 8 * 128 // (ctx * hkv * dim))
        return _tree("", _spread(rng, 1, max(1, min(64, most))), nodes, ctx, hkv * group, hkv, dim, dtype, ragged, window, cap)
    if kind == "keep":
        nodes = _spread(rng, 1, 200)
        caches = rng.randint(1, 6)
        batch = _spread(rng, 1, max(1, min(64, 64 * 61 * 4 // (nodes * caches))))
        return _keep("", batch, nodes, nodes + _spread(rng, 1, 4000) - 1, hkv, dim, dtype, caches, ragged)
    if kind == "adapters":
        how = rng.choice(["fwd", "add"])
        runs = rng.random() < 0.4
        rows = _spread(rng, 64, 2048) if runs else _spread(rng, 1, 256)
        cols = G * _spread(rng, 4, 256)
        outs = _spread(rng, 100, 8192)
        if rng.random() < 0.6:
            outs = (outs + 63) // 64 * 64
        rank = rng.choice([4, 8, 8, 16, 16, 16, 24, 32, 64])
        slots = _spread(rng, 1, 64)
        while rows * outs > 2048 * 8192 // 2:
            outs //= 2
        # the linear of fp16 rows has its own rounding of scales into fp16 weights: those rows are added beside
        xtype = rng.choice(["bf16", "fp32"] if how == "fwd" else ["bf16", "fp32", "fp16"])
        return _adapters("", how, rows, cols, outs, rank, slots, xtype, dtype, runs)
    nodes = rng.choice([1, 1, _spread(rng, 2, 64)])
    batch = _spread(rng, 1, max(1, min(64, 128 // nodes)))
    vocab = _spread(rng, 500, 160000)
    while batch * nodes * vocab > 8 * 16 * 128256 // 2:
        vocab //= 2
    return _logits("", batch, nodes, vocab, rng.choice([0, _spread(rng, 1, 8192)]), rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                   rng.choice([0, rng.randint(1, 200)]), rng.random() < 0.5, ragged)


def _lens(case):
    """(nodes, tokens in the cache with them) of every sequence: all alike, or unlike with the first as
    long as the case says."""
    new, ctx = [case["nodes"]] * case["batch"], [case.get("ctx", 0)] * case["batch"]
    if case["ragged"]:
        r = random.Random(f"{case['batch']} {case['nodes']} {case.get('ctx')}")
        for b in range(1, case["batch"]):
            new[b] = r.randint((case["nodes"] + 1) // 2, case["nodes"])
            ctx[b] = r.randint(max(new[b], case.get("ctx", 0) // 4), max(new[b], case.get("ctx", 0)))
    return new, ctx


def _forest(case, seed):
    """Parents of every sequence's nodes: node 0 the token sampled last, each later one behind one of the
    eight nodes before it, now and then a second root."""
    r = random.Random(f"tree {seed}")
    new, _ = _lens(case)
    return [[-1 if i == 0 or r.random() < 0.02 else i - r.randint(1, min(i, 8)) for i in range(m)] for m in new]


def _path(parents, leaf):
    path = []
    while leaf >= 0:
        path.append(leaf)
        leaf = parents[leaf]
    return path[::-1]


def _history(case):
    """(tokens, of them prompt) that each sequence has behind it."""
    r = random.Random(f"history {case['batch']} {case['history']}")
    n = [case["history"] if b == 0 or not case["ragged"] else r.randint(case["history"] // 4, case["history"])
         for b in range(case["batch"])]
    return n, [x * 3 // 4 for x in n]


def _slots(case, seed):
    """The adapter of every row: prompts one after the other, or single tokens as they come; -1: none."""
    r = random.Random(f"slots {seed}")
    m, n = case["rows"], case["slots"]
    if not case["runs"]:
        return [-1 if r.random() < 0.03 else r.randrange(n) for _ in range(m)]
    parts = min(n, 8)
    cut = [0] + sorted(r.randrange(m + 1) for _ in range(parts - 1)) + [m]
    order = r.sample(range(n), parts)
    return [order[j] for j in range(parts) for _ in range(cut[j], cut[j + 1])]


def work(case):
    if case["op"] == "adapters":
        m, k, n, r = case["rows"], case["cols"], case["outs"], case["rank"]
        used = len(set(_slots(case, 1)) - {-1})
        # x, the used factors, y; with the weight's codes and scales, or the projection it is added to
        base = n * k * (0.5 + 2 / G) if case["how"] == "fwd" else 4 * m * n
        return {"bytes": int(m * k * SIZE[case["xtype"]] + used * r * (k + n) * 2 + base + 4 * m * n),
                "flops": 2 * m * r * (k + n) + (2 * m * n * k if case["how"] == "fwd" else 0)}
    new, ctx = _lens(case)
    if case["op"] == "logits":
        rows = sum(new)
        size = rows * case["vocab"]
        return {"bytes": int(size * (2 * SIZE[case["dtype"]] + (1 / 8 if case["mask"] else 0)) + 4 * sum(_history(case)[0])
                             + 8 * case["batch"] * case["bias"]), "flops": 6 * size}
    row = case["hkv"] * case["dim"] * 2           # elements of one token's keys and values
    if case["op"] == "keep":
        paths = [len(_path(f, len(f) - 1)) for f in _forest(case, 1)]
        n = sum(new) * row
        # the drafts in and, as fp32, out again; a path's codes read and written
        return {"bytes": int(case["caches"] * (n * (SIZE[case["dtype"]] + 0.5 + 2 / G + 4) + 2 * sum(paths) * row * (0.5 + 2 / G))),
                "flops": 6 * case["caches"] * n}
    keys = pairs = 0
    for m, n in zip(new, ctx):
        first = max(0, n - m + 1 - case["window"]) if case["window"] else 0
        keys += n - first
        pairs += m * (n - m - first) + 4 * m
    io = 2 * sum(new) * case["hq"] * case["dim"] * SIZE[case["dtype"]]
    return {"bytes": int(keys * row * (0.5 + 2 / G)) + io + 4 * sum(new), "flops": 4 * pairs * case["hq"] * case["dim"]}


# ---- inputs ----------------------------------------------------------------------------------
def _gen(seed, b):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 7919 * b + 1)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _keys_values(case, seed, b, n):
    """n tokens of keys (a few channels larger than the others, as keys have them) and values."""
    g = _gen(seed, b)
    h, d = case["hkv"], case["dim"]
    channel = 0.5 + torch.rand(h, d, generator=g, device="cuda")
    channel = torch.where(torch.rand(h, d, generator=g, device="cuda") < 0.03, 5 * channel, channel)
    k = (_randn(g, n, h, d) * channel).to(DT[case["dtype"]])
    return k, _randn(g, n, h, d).to(DT[case["dtype"]])


def _quantise(x):
    """(code - 8 as int8 [.., dim], scale fp16 [.., dim / 32]) of rows of keys or values."""
    g = x.float().unflatten(-1, (-1, G))
    amax = g.abs().amax(-1)
    s = (amax / torch.full_like(amax, 7.0)).clamp(max=8188.0).half()
    inv = (1.0 / s.float()).unsqueeze(-1)
    c = torch.where(s.unsqueeze(-1) > 0, (g * inv).round().clamp(-8, 7), torch.zeros_like(g))
    return c.to(torch.int8).flatten(-2), s


def _values(codes, scale):
    return (codes.unflatten(-1, (-1, G)).float() * scale.float().unsqueeze(-1)).flatten(-2)


class _Pool:
    """The plain form's cache: int8 code - 8 and scales of every page's tokens."""

    def __init__(self, pages, h, d):
        self.k, self.v = (torch.zeros(pages, P, h, d, dtype=torch.int8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.zeros(pages, P, h, d // G, dtype=torch.float16, device="cuda") for _ in range(2))

    def store(self, k, v, page, slot):
        self.k[page, slot], self.ks[page, slot] = _quantise(k)
        self.v[page, slot], self.vs[page, slot] = _quantise(v)


def _factors(case, seed):
    """(A [slots, rank, cols], B [slots, outs, rank], alpha) of every adapter."""
    g = _gen(seed, -2)
    n, r = case["slots"], case["rank"]
    a = (_randn(g, n, r, case["cols"]) * case["cols"] ** -0.5).to(DT[case["ftype"]])
    b = (_randn(g, n, case["outs"], r) * 0.3).to(DT[case["ftype"]])
    return a, b, [2.0 * (1 + s % 3) / r for s in range(n)]


def _rows(case, seed):
    """(x, the 4-bit weight's codes and scales, or the projection to add to)."""
    g = _gen(seed, -3)
    m, k, n = case["rows"], case["cols"], case["outs"]
    x = _randn(g, m, k).to(DT[case["xtype"]])
    if case["how"] == "add":
        return x, _randn(g, m, n), None
    codes = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    return x, codes, ((0.8 + 0.4 * torch.rand(k // G, n, generator=g, device="cuda")) / (4.6 * k ** 0.5)).half()


def _prepare_adapters(case, seed):
    x, w, scales = _rows(case, seed)
    a, b, alpha = _factors(case, seed)
    s = dict(case=case, x=x, slots=_ints(_slots(case, seed)))
    if own:
        import bit_group_quantized_q4gsw_amd as q4
        s.update(q4=q4, set=q4.adapters(case["slots"], case["rank"], case["outs"], case["cols"], DT[case["ftype"]], "cuda"),
                 out=torch.empty(case["rows"], case["outs"], dtype=torch.float32, device="cuda"))
        for i in range(case["slots"]):
            q4.adapters_load(s["set"], i, a[i], b[i], alpha[i])
        if case["how"] == "fwd":
            s.update(w=q4.pack(w, scales, G))
            need = q4.adapters_workspace_bytes(s["set"], case["rows"], x.dtype, s["w"])
        else:
            s.update(base=w)
            need = q4.adapters_workspace_bytes(s["set"], case["rows"], x.dtype)
        s.update(workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    else:
        s.update(w=w, scales=scales, a=a, b=b, alpha=torch.tensor(alpha, dtype=torch.float32).cuda())
    return s


def _prepare_logits(case, seed):
    new, _ = _lens(case)
    b, v = case["batch"], case["vocab"]
    g = _gen(seed, 0)
    n, prompt = _history(case)
    ids = lambda *shape: torch.randint(0, v, shape, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    s = dict(case=case, logits=(3 * _randn(g, sum(new), v)).to(DT[case["dtype"]]),
             # common tokens come again and again
             history=torch.where(torch.rand(b, max(1, case["history"]), generator=g, device="cuda") < 0.5,
                                 ids(b, max(1, case["history"])) % min(v, 300), ids(b, max(1, case["history"]))),
             history_lens=_ints(n), prompt_lens=_ints(prompt), ids=None, parents=None, cu=None, bias_ids=None, bias=None,
             mask=None, max_new=max(new))
    s.update(repetition=1 + 0.5 * torch.rand(b, generator=g, device="cuda"),
             presence=torch.rand(b, generator=g, device="cuda"), frequency=0.3 * torch.rand(b, generator=g, device="cuda"))
    if case["nodes"] > 1:
        s.update(cu=_ints([sum(new[:i]) for i in range(b + 1)]), ids=ids(sum(new)),
                 parents=_ints([p for f in _forest(case, seed) for p in f]))
    if case["bias"]:
        # no token twice in a sequence's list
        first = ids(b, 1)
        s.update(bias_ids=((first + torch.arange(case["bias"], device="cuda", dtype=torch.int32) * max(1, v // 256)) % v)
                 .to(torch.int32).contiguous(), bias=3 * _randn(g, b, case["bias"]))
    if case["mask"]:
        s.update(mask=torch.randint(-2 ** 31, 2 ** 31, (sum(new), (v + 31) // 32), generator=g, device="cuda").to(torch.int32))
    if own:
        import bit_group_quantized_q4gsw_amd as q4
        s.update(q4=q4, out=torch.empty_like(s["logits"]))
    return s


def prepare(case, seed):
    if case["op"] == "adapters":
        return _prepare_adapters(case, seed)
    if case["op"] == "logits":
        return _prepare_logits(case, seed)
    new, ctx = _lens(case)
    h, d = case["hkv"], case["dim"]
    need = [(n + P - 1) // P for n in ctx]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 1)).tolist()
    table = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
        order = order[n:]
    forest = _forest(case, seed)
    s = dict(case=case, batch=len(new), max_new=max(new), max_ctx=max(ctx), tokens=sum(new), table=table.cuda(),
             cu=_ints([sum(new[:b]) for b in range(len(new) + 1)]), lens=_ints(ctx),
             parents=_ints([p for f in forest for p in f]))
    caches = case.get("caches", 1)
    if own:
        import bit_group_quantized_q4gsw_amd as q4
        s.update(q4=q4, caches=[q4.kv_cache(pages, P, h, d, "cuda") for _ in range(caches)])
    else:
        s.update(caches=[_Pool(pages, h, d) for _ in range(caches)])

    if case["op"] == "keep":
        kv = [[_keys_values(case, seed, b + 1000 * c, m) for b, m in enumerate(new)] for c in range(caches)]
        s.update(k=[torch.cat([k for k, _ in one]) for one in kv], v=[torch.cat([v for _, v in one]) for one in kv],
                 leaf=_ints([len(f) - 1 for f in forest]))
        return s

    g = _gen(seed, -1)
    # scores of a spread of two to three, as trained heads have them
    s["q"] = (1.6 * _randn(g, sum(new), case["hq"], d)).to(DT[case["dtype"]])
    for b, n in enumerate(ctx):
        k, v = _keys_values(case, seed, b, n)
        if own:
            one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            s["q4"].kv_append(s["caches"][0], k, v, s["table"][b:b + 1], one, s["lens"][b:b + 1])
        else:
            t = torch.arange(n, device="cuda")
            s["caches"][0].store(k, v, s["table"][b].long()[t // P], t % P)
    if own:
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = torch.empty(
            q4.kv_tree_attention_workspace_bytes(s["caches"][0], len(ctx), sum(new), case["hq"], max(new), max(ctx)),
            dtype=torch.uint8, device="cuda")
    return s


# ---- the operators ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"tree": _own_tree, "keep": _own_keep, "adapters": _own_adapters, "logits": _own_logits}[op](s)
    return {"tree": _plain_tree, "keep": _plain_keep, "adapters": _plain_adapters, "logits": _plain_logits}[op](s)


def _own_tree(s):
    c = s["case"]
    return s["q4"].kv_tree_attention(s["caches"][0], s["q"], s["parents"], s["table"], s["cu"], s["lens"], s["max_new"],
                                     s["max_ctx"], window=c["window"], softcap=c["cap"], out=s["out"],
                                     workspace=s["workspace"])


def _own_keep(s):
    q4, where = s["q4"], (s["table"], s["cu"], s["lens"])
    for cache, k, v in zip(s["caches"], s["k"], s["v"]):
        q4.kv_append(cache, k, v, *where)
    kept, path = q4.kv_keep(s["caches"], s["parents"], s["leaf"], *where, s["max_new"])
    return kept, path, [q4.kv_read(cache, *where, s["tokens"]) for cache in s["caches"]]


def _own_adapters(s):
    if s["case"]["how"] == "fwd":
        return s["q4"].adapters_fwd(s["w"], s["x"], s["set"], s["slots"], out=s["out"], workspace=s["workspace"])
    return s["q4"].adapters_add(s["base"], s["x"], s["set"], s["slots"], out=s["out"], workspace=s["workspace"])


def _own_logits(s):
    return s["q4"].logits_adjust(s["logits"], cu=s["cu"], max_new=s["max_new"], history=s["history"],
                                 history_lens=s["history_lens"], prompt_lens=s["prompt_lens"], ids=s["ids"],
                                 parents=s["parents"], repetition=s["repetition"], presence=s["presence"],
                                 frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"],
                                 out=s["out"])


def _ancestors(parents, cu, batch, most):
    """bool [batch, most, most]: node j is an ancestor of node i or itself."""
    token = torch.arange(parents.numel(), device="cuda")
    seq = torch.searchsorted(cu[1:].long(), token, right=True)
    node, up = token - cu[seq], parents.long()
    reach = torch.zeros(batch, most + 1, most + 1, device="cuda")
    reach[seq, node, torch.where((up >= 0) & (up < node), up, most)] = 1.0
    reach = (reach[:, :most, :most] + torch.eye(most, device="cuda")).contiguous()
    for _ in range((most - 1).bit_length()):               # ways of twice as many steps
        reach = (torch.matmul(reach, reach) > 0).float()
    return reach > 0, seq, node


def _plain_tree(s):
    c, pool = s["case"], s["caches"][0]
    hkv, d, group = c["hkv"], c["dim"], c["hq"] // c["hkv"]
    batch, m, n = s["batch"], s["max_new"], s["max_ctx"]
    reach, seq, node = _ancestors(s["parents"], s["cu"], batch, m)
    t = torch.arange(n, device="cuda")
    before = (s["lens"] - (s["cu"][1:] - s["cu"][:-1])).long()[:, None]
    page, slot = s["table"][:, t // P].long().clamp(min=0), (t % P).expand(batch, n)
    k = _values(pool.k[page, slot], pool.ks[page, slot]).permute(0, 2, 3, 1).reshape(batch * hkv, d, n)
    v = _values(pool.v[page, slot], pool.vs[page, slot]).transpose(1, 2).reshape(batch * hkv, n, d)
    q = torch.zeros(batch, m, c["hq"], d, device="cuda")
    q[seq, node] = s["q"].float()
    q = q.view(batch, m, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch * hkv, group * m, d)
    x = torch.matmul(q, k.contiguous()) * d ** -0.5
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    inside = (t >= before) & (t < s["lens"][:, None])
    at = (t - before).clamp(0, m - 1)
    seen = torch.where(inside[:, None], reach.gather(2, at[:, None].expand(batch, m, n)), (t < before)[:, None])
    if c["window"]:
        depth = reach.sum(2) - 1
        position = torch.where(inside, before + depth.gather(1, at), t)
        seen &= position[:, None] > (before + depth)[:, :, None] - c["window"]
    seen |= (torch.arange(m, device="cuda") >= (s["cu"][1:] - s["cu"][:-1])[:, None])[:, :, None]    # rows of no node
    x = x.view(batch, hkv, group, m, n).masked_fill(~seen[:, None, None], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p.view(batch * hkv, group * m, n), v.contiguous()).view(batch, hkv, group, m, d) / p.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(batch, m, c["hq"], d)[seq, node].to(s["q"].dtype)


def _plain_keep(s):
    m = s["max_new"]
    reach, seq, node = _ancestors(s["parents"], s["cu"], s["batch"], m)
    before = (s["lens"] - (s["cu"][1:] - s["cu"][:-1])).long()
    on = reach[torch.arange(s["batch"], device="cuda"), s["leaf"].long()]          # [batch, m]: on the path
    count = on.sum(1)
    kept = (before + count).to(torch.int32)
    order = torch.where(on, torch.arange(m, device="cuda"), m).sort(1).values
    path = torch.where(order < m, order, -1).to(torch.int32)
    pos = before[seq] + node
    source = before[seq] + torch.where(node < count[seq], order[seq, node], node)
    page, slot = s["table"][seq, pos // P].long(), pos % P
    from_page, from_slot = s["table"][seq, source // P].long(), source % P
    out = []
    for pool, k, v in zip(s["caches"], s["k"], s["v"]):
        pool.store(k, v, page, slot)
        moved = [x[from_page, from_slot] for x in (pool.k, pool.ks, pool.v, pool.vs)]
        for x, y in zip((pool.k, pool.ks, pool.v, pool.vs), moved):
            x[page, slot] = y
        out.append((_values(pool.k[page, slot], pool.ks[page, slot]), _values(pool.v[page, slot], pool.vs[page, slot])))
    return kept, path, out


def _plain_adapters(s):
    c = s["case"]
    n, r = c["slots"], c["rank"]
    x = s["x"].float()
    if c["how"] == "fwd":
        w = (s["w"].float() - 8).unflatten(1, (-1, G)) * s["scales"].float().t().unsqueeze(-1)
        y = torch.matmul(x, w.flatten(1).t())
    else:
        y = s["w"]
    used = s["slots"].long()[:, None] == torch.arange(n, device="cuda")              # [rows, slots]
    t = torch.matmul(x, s["a"].float().view(n * r, -1).t()).view(-1, n, r)
    t = torch.where(used[:, :, None], t * s["alpha"][:, None], torch.zeros_like(t)).view(-1, n * r)
    return y + torch.matmul(t, s["b"].float().transpose(1, 2).reshape(n * r, -1))


def _plain_logits(s):
    c = s["case"]
    b, v = c["batch"], c["vocab"]
    x = s["logits"].float()
    rows = x.shape[0]
    at = torch.arange(s["history"].shape[1], device="cuda")
    held, prompt = at < s["history_lens"][:, None], at < s["prompt_lens"][:, None]
    ids = s["history"].long()
    seen = torch.zeros(b, v, device="cuda").scatter_add(1, ids, held.float())
    made = torch.zeros(b, v, device="cuda").scatter_add(1, ids, (held & ~prompt).float())
    if s["cu"] is None:
        seq = torch.arange(rows, device="cuda")
    else:
        reach, seq, node = _ancestors(s["parents"], s["cu"], b, s["max_new"])
        token = torch.zeros(b, s["max_new"], dtype=torch.long, device="cuda")
        token[seq, node] = s["ids"].long()
        path = torch.zeros(rows, v, device="cuda").scatter_add(1, token[seq], reach[seq, node].float())
    seen, made = seen[seq], made[seq]
    if s["cu"] is not None:
        seen, made = seen + path, made + path
    rep = s["repetition"][seq][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = torch.where(made > 0, x - s["frequency"][seq][:, None] * made - s["presence"][seq][:, None], x)
    if s["bias"] is not None:
        x = x + torch.zeros(b, v, device="cuda").scatter(1, s["bias_ids"].long(), s["bias"])[seq]
    if s["mask"] is not None:
        token = torch.arange(v, device="cuda")
        x = x.masked_fill((s["mask"][:, token // 32] >> (token % 32) & 1) == 0, float("-inf"))
    return x.to(s["logits"].dtype)


# ---- the definitions in 64 bits --------------------------------------------------------------
def _f32(x):
    return x.to(torch.float32).double()


def _stored(x):
    """What the cache stands for, in 64 bits; the definition's roundings to 16 and 32 bits kept."""
    n, h, d = x.shape
    x = x.double().view(n, h, d // G, G)
    step = _f32(x.abs().max(dim=-1, keepdim=True).values / 7).clamp(max=8188.0).to(torch.float16).double()
    code = torch.round(_f32(x * _f32(1 / step.clamp(min=2.0 ** -24)))).clamp(-8, 7)
    return (code * step).view(n, h, d)


def _exact_adapters(case, seed):
    x, w, scales = _rows(case, seed)
    a, b, alpha = _factors(case, seed)
    x = x.double()
    if case["how"] == "fwd":
        w = (w.double() - 8) * scales.double().T.repeat_interleave(G, dim=1)
        y = x @ w.T
    else:
        y = w.double()
    slots = torch.tensor(_slots(case, seed), device="cuda")
    for i in range(case["slots"]):
        mine = (slots == i).nonzero()[:, 0]
        if len(mine):
            factor = float(torch.tensor(alpha[i], dtype=torch.float32))
            y[mine] += factor * ((x[mine] @ a[i].double().T) @ b[i].double().T)
    return y


def _exact_logits(case, seed):
    s = _prepare_logits(case, seed)
    new, _ = _lens(case)
    held, prompt = _history(case)
    out, at = s["logits"].double(), 0
    forest = _forest(case, seed) if s["cu"] is not None else [[-1]] * case["batch"]
    for b, m in enumerate(new):
        told = s["history"][b, :held[b]].tolist()
        rep, pres, freq = (float(s[k][b]) for k in ("repetition", "presence", "frequency"))
        base = torch.bincount(torch.tensor(told[prompt[b]:], dtype=torch.long), minlength=case["vocab"])
        had = torch.bincount(torch.tensor(told, dtype=torch.long), minlength=case["vocab"]) > 0
        tokens = s["ids"][at:at + m].tolist() if s["ids"] is not None else None
        for i in range(m):
            made, seen = base.clone(), had.clone()
            for j in _path(forest[b], i) if tokens else []:
                made[tokens[j]] += 1
                seen[tokens[j]] = True
            made, seen = made.cuda(), seen.cuda()
            x = out[at + i]
            x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
            x = x - freq * made - pres * (made > 0)
            if s["bias"] is not None:
                x[s["bias_ids"][b].long()] += s["bias"][b].double()
            if s["mask"] is not None:
                bits = (s["mask"][at + i].long()[:, None] >> torch.arange(32, device="cuda")) & 1
                x[bits.flatten()[:case["vocab"]] == 0] = -float("inf")
            out[at + i] = x
        at += m
    return out


def exact(case, seed):
    if case["op"] == "adapters":
        return _exact_adapters(case, seed)
    if case["op"] == "logits":
        return _exact_logits(case, seed)
    new, ctx = _lens(case)
    forest = _forest(case, seed)
    if case["op"] == "keep":
        paths = [_path(f, len(f) - 1) for f in forest]
        out = []
        for c in range(case["caches"]):
            ks, vs = [], []
            for b, m in enumerate(new):
                k, v = (_stored(x) for x in _keys_values(case, seed, b + 1000 * c, m))
                order = paths[b] + list(range(len(paths[b]), m))
                ks.append(k[order])
                vs.append(v[order])
            out.append((torch.cat(ks), torch.cat(vs)))
        kept = _ints([n - m + len(p) for n, m, p in zip(ctx, new, paths)])
        return kept, _ints([p + [-1] * (max(new) - len(p)) for p in paths]), out

    group, win, cap = case["hq"] // case["hkv"], case["window"], case["cap"]
    q = (1.6 * _randn(_gen(seed, -1), sum(new), case["hq"], case["dim"])).to(DT[case["dtype"]]).double()
    out, at = torch.zeros_like(q), 0
    for b, (m, n) in enumerate(zip(new, ctx)):
        k, v = _keys_values(case, seed, b, n)
        gone = torch.ones(m, n, dtype=torch.bool)
        for i in range(m):
            path = _path(forest[b], i)
            first = max(0, n - m + len(path) - win) if win else 0
            gone[i, first:n - m] = False
            for j in path[-win:] if win else path:
                gone[i, n - m + j] = False
        gone = gone.cuda()
        for kvh in range(case["hkv"]):
            ks, vs = _stored(k[:, kvh:kvh + 1])[:, 0], _stored(v[:, kvh:kvh + 1])[:, 0]
            for hq in range(kvh * group, (kvh + 1) * group):
                x = q[at:at + m, hq] @ ks.T / case["dim"] ** 0.5
                if cap:
                    x = cap * torch.tanh(x / cap)
                x[gone] = -float("inf")
                out[at:at + m, hq] = torch.softmax(x, dim=1) @ vs
        at += m
    return out
