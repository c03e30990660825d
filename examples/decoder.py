"""A small decoder served with 4-bit weights, int8 activations and a 4-bit key/value cache.

Every layer is
    h, rows = h + y, int8 rows of rmsnorm(h)       rmsnorm_dq8ca
    q, k, v = rows . W^T                           linear_dq8ca_rows, three weights on one set of rows
    cache  <- k, v;  y = attention(q, cache)       kv_append, kv_attention
    h, rows = h + y . Wo^T, int8 rows of its norm  linear_fwd, rmsnorm_dq8ca
    y = (silu(g) * u) . Wd^T, [g u] = rows . Wu^T  linear_dq8ca_rows, linear_fwd
on random weights, without positions (nothing rotates q and k on their way).  Run as a command it
takes a batch of prompts of unlike lengths in one call and then decodes from a captured HIP graph:

    python examples/decoder.py [--layers 4] [--batch 8] [--prompt 512] [--tokens 64] [--adapters 4] [--draft]

With --adapters every sequence takes one of so many low-rank adapters beside the projections
(adapters_add, adapters_fwd).  With --draft a step checks a tree of drafted tokens at once: attention
over the tree (kv_tree_attention), rules on the logits of every node (logits_adjust), and the accepted path's
keys and values moved together (kv_keep).
"""
import argparse
import copy
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_group_quantized_q4gsw_amd as q  # noqa: E402

EPS = 1e-6
PAGE = 64


class Config:
    def __init__(self, hidden=2048, ffn=8192, heads=32, kv_heads=8, dim=64, layers=4, vocab=32000, group=32):
        self.hidden, self.ffn, self.heads, self.kv_heads, self.dim = hidden, ffn, heads, kv_heads, dim
        self.layers, self.vocab, self.group = layers, vocab, group


def random_weight(n, k, group, gen):
    """Codes and scales of a [n, k] weight with rows of norm about one."""
    codes = torch.randint(0, 16, (n, k), generator=gen, dtype=torch.uint8)
    scales = ((0.8 + 0.4 * torch.rand(k // group, n, generator=gen)) / (4.6 * k ** 0.5)).half()
    return q.pack(codes.cuda(), scales.cuda(), group)


class Layer:
    def __init__(self, c, gen):
        weight = lambda n, k: random_weight(n, k, c.group, gen)
        self.wq, self.wk, self.wv = (weight(n * c.dim, c.hidden) for n in (c.heads, c.kv_heads, c.kv_heads))
        self.wo = weight(c.hidden, c.heads * c.dim)
        self.wu, self.wd = weight(2 * c.ffn, c.hidden), weight(c.hidden, c.ffn)
        self.norm1, self.norm2 = (1 + 0.1 * torch.randn(c.hidden, generator=gen).cuda() for _ in range(2))


class LayerAdapters:
    """Adapters of a layer's query, value, output and down projections, one slot a tenant."""

    def __init__(self, c, slots, rank, gen):
        inner = c.heads * c.dim
        shapes = dict(q=(inner, c.hidden), v=(c.kv_heads * c.dim, c.hidden), o=(c.hidden, inner), d=(c.hidden, c.ffn))
        for name, (n, k) in shapes.items():
            s = q.adapters(slots, rank, n, k)
            for i in range(slots):
                q.adapters_load(s, i, torch.randn(rank, k, generator=gen).cuda() * k ** -0.5,
                                torch.randn(n, rank, generator=gen).cuda() * (0.1 * rank ** -0.5), 1.0)
            setattr(self, name, s)


class Decoder:
    def __init__(self, c, seed=0, adapters=0, rank=16):
        gen = torch.Generator().manual_seed(seed)
        self.c = c
        self.embed = random_weight(c.vocab, c.hidden, c.group, gen)      # also the output weight
        self.layers = [Layer(c, gen) for _ in range(c.layers)]
        self.norm = 1 + 0.1 * torch.randn(c.hidden, generator=gen).cuda()
        for layer in self.layers:
            layer.adapters = LayerAdapters(c, adapters, rank, gen) if adapters else None

    def hidden(self, h, state, max_new, max_ctx, last):
        """The normalised rows `last` of the final stream for the embedded new tokens h [tokens, hidden]."""
        c, T = self.c, h.shape[0]
        y = torch.zeros_like(h)
        slots = state.row_slots(T)
        for layer, cache in zip(self.layers, state.caches):
            a = layer.adapters if slots is not None else None
            rows, h, x = q.rmsnorm_dq8ca(y, layer.norm1, EPS, residual=h, values=torch.empty_like(h) if a else None)
            xq, xk, xv = (q.linear_dq8ca_rows(w, rows) for w in (layer.wq, layer.wk, layer.wv))
            if a:
                q.adapters_add(xq, x, a.q, slots, out=xq)
                q.adapters_add(xv, x, a.v, slots, out=xv)
            xq, xk, xv = (x.view(T, -1, c.dim) for x in (xq, xk, xv))
            q.kv_append(cache, xk, xv, state.table, state.cu, state.lens)
            if state.parents is None:
                y = q.kv_attention(cache, xq, state.table, state.cu, state.lens, max_new, max_ctx)
            else:
                y = q.kv_tree_attention(cache, xq, state.parents, state.table, state.cu, state.lens, max_new, max_ctx)
            y = y.view(T, -1)
            y = q.adapters_fwd(layer.wo, y, a.o, slots) if a else q.linear_fwd(layer.wo, y)
            rows, h, _ = q.rmsnorm_dq8ca(y, layer.norm2, EPS, residual=h)
            g, u = q.linear_dq8ca_rows(layer.wu, rows).chunk(2, 1)
            y = torch.nn.functional.silu(g) * u
            y = q.adapters_fwd(layer.wd, y, a.d, slots) if a else q.linear_fwd(layer.wd, y)
        return q.rmsnorm_dq8ca(y[last], self.norm, EPS, residual=h[last])[0]

    def logits(self, ids, state, max_new, max_ctx, last):
        h = q.embedding(self.embed, ids) * self.c.hidden ** 0.5
        return q.linear_dq8ca_rows(self.embed, self.hidden(h, state, max_new, max_ctx, last))


class State:
    """The sequences of a batch: a cache per layer, the page table, and the lengths with the call's
    new tokens.  The tensors stay where they are: a captured graph holds their addresses."""

    def __init__(self, c, capacity):
        need = [(n + PAGE - 1) // PAGE for n in capacity]
        pages, at = sum(need), 0
        table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
            at += n
        self.table = table.cuda()
        self.caches = [q.kv_cache(pages, PAGE, c.kv_heads, c.dim) for _ in range(c.layers)]
        self.lens = torch.zeros(len(need), dtype=torch.int32, device="cuda")
        self.cu = torch.zeros(len(need) + 1, dtype=torch.int32, device="cuda")
        self.capacity, self.held = list(capacity), [0] * len(need)
        self.parents = None          # of the new tokens, where they form trees
        self.slots = None            # int32 [batch]: the adapter of every sequence

    def row_slots(self, tokens):
        """The adapters of a call's token rows."""
        if self.slots is None:
            return None
        row = torch.arange(tokens, dtype=torch.int32, device="cuda")
        return self.slots[torch.searchsorted(self.cu[1:], row, right=True).clamp(max=self.slots.numel() - 1)]

    def take(self, news):
        """Count news[b] more tokens of sequence b on the host; ValueError if one has no room for them."""
        held = [n + m for n, m in zip(self.held, news)]
        for b, (n, room) in enumerate(zip(held, self.capacity)):
            if n > room:
                raise ValueError(f"sequence {b} has room for {room} tokens, {n} needed")
        self.held[:] = held

    def advance(self, news):
        """The next call brings news[b] tokens of sequence b."""
        self.take(news)
        self.cu.copy_(torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], dtype=torch.int32))
        self.lens += torch.tensor(news, dtype=torch.int32, device="cuda")


class Stepper:
    """One greedy token of every sequence a replay, from a captured graph.  `ids` holds the next step's
    tokens; between steps the state may take prompt chunks."""

    def __init__(self, model, state, ids, max_ctx):
        self.model, self.state, self.max_ctx = model, state, max_ctx
        self.ids = ids.clone()
        batch = ids.numel()
        self.view = copy.copy(state)             # the state's tensors, with the offsets of single tokens
        self.view.cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
        self.last = torch.arange(batch, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):        # writes the places that the first step writes again
            state.lens.add_(1)
            self.model.logits(self.ids, self.view, 1, max_ctx, self.last)
            state.lens.sub_(1)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = self.launch()

    def launch(self):
        self.state.lens.add_(1)
        out = self.model.logits(self.ids, self.view, 1, self.max_ctx, self.last)
        self.ids.copy_(out.argmax(1))
        return out

    def step(self):
        """The same step without the graph."""
        self.state.take([1] * self.ids.numel())
        return self.launch()

    def __call__(self):
        self.state.take([1] * self.ids.numel())
        self.graph.replay()
        return self.out


class TreeStepper:
    """Drafted tokens checked a tree at a time, from a captured graph.  Node 0 is the token chosen last; node j
    behind node i is drafted from `follow`, int32 [vocab, width]: the tokens seen last behind a token (the
    nodes behind one node take its columns in turn).  A step keeps the longest path whose every token is
    what greedy decoding of its parent gives, which is the token itself after logits_adjust, and at least
    node 0.  `history` holds every sequence's tokens, history_lens of them."""

    def __init__(self, model, state, prompts, ids, parents, follow, max_ctx, penalty=1.0):
        self.model, self.state, self.max_ctx = model, state, max_ctx
        self.follow = torch.cat([follow, follow[:1]])            # the last row takes what is not kept
        batch, nodes = len(prompts), len(parents)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        depth, rank = [0] * nodes, [0] * nodes
        for j, p in enumerate(parents):
            if j:
                depth[j], rank[j] = depth[p] + 1, parents[:j].count(p) % follow.shape[1]
        self.up, self.rank = torch.tensor(parents, device="cuda"), torch.tensor(rank, device="cuda")
        self.depth = torch.tensor(depth, device="cuda")
        self.levels = [torch.tensor([j for j in range(nodes) if depth[j] == d], device="cuda") for d in range(1, max(depth) + 1)]
        self.most = max(depth) + 1                   # tokens that a step keeps at most
        self.view = copy.copy(state)
        self.view.parents = ints(parents * batch)
        self.view.cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * nodes
        self.last = torch.arange(batch * nodes, device="cuda")
        room = max(state.capacity) + 1               # the last column takes what is not kept
        self.history = torch.zeros(batch, room + 1, dtype=torch.int32, device="cuda")
        for b, x in enumerate(prompts):
            self.history[b, :x.numel()] = x
        self.history_lens, self.prompt_lens = (ints([x.numel() for x in prompts]) for _ in range(2))
        self.ids = ids.clone()
        self.penalty = torch.full((batch,), penalty, device="cuda")
        self.kept = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.path = torch.zeros(batch, nodes, dtype=torch.int32, device="cuda")
        keep = [x.clone() for x in self.changing()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):                # writes places that the first step writes again
            self.launch()
        torch.cuda.current_stream().wait_stream(side)
        for x, y in zip(self.changing(), keep):
            x.copy_(y)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.launch()

    def changing(self):
        """What a step changes, but for the caches behind the kept tokens."""
        return [self.state.lens, self.history, self.history_lens, self.ids, self.follow]

    def launch(self):
        state, batch, nodes = self.state, self.ids.numel(), self.up.numel()
        tree = torch.zeros(batch, nodes, dtype=torch.long, device="cuda")
        tree[:, 0] = self.ids
        for at in self.levels:
            tree[:, at] = self.follow[tree[:, self.up[at]], self.rank[at]].long()
        state.lens.add_(nodes)
        out = self.model.logits(tree.flatten(), self.view, nodes, self.max_ctx, self.last)
        tokens = tree.flatten().to(torch.int32)
        out = q.logits_adjust(out, cu=self.view.cu, max_new=nodes, history=self.history, history_lens=self.history_lens,
                              prompt_lens=self.prompt_lens, ids=tokens, parents=self.view.parents, repetition=self.penalty, out=out)
        best = out.argmax(1).view(batch, nodes)
        right = torch.ones(batch, nodes, dtype=torch.bool, device="cuda")
        for at in self.levels:
            right[:, at] = right[:, self.up[at]] & (tree[:, at] == best[:, self.up[at]])
        leaf = torch.where(right, self.depth, -1).argmax(1)
        q.kv_keep(state.caches, self.view.parents, leaf.to(torch.int32), state.table, self.view.cu, state.lens, nodes,
                  kept=self.kept, path=self.path)
        state.lens.copy_(self.kept)
        # the kept tokens go behind the history, what follows each into the table
        kept = self.path >= 0
        chosen = tree.gather(1, self.path.clamp(min=0).long())
        place = self.history_lens[:, None] + torch.arange(nodes, device="cuda")
        place = torch.where(kept, place, self.history.shape[1] - 1)
        self.history.scatter_(1, place.long(), chosen.to(torch.int32))
        self.history_lens.add_(kept.sum(1, dtype=torch.int32))
        after = best.gather(1, self.path.clamp(min=0).long())
        self.follow[:, 0].scatter_(0, torch.where(kept, chosen, self.follow.shape[0] - 1).flatten(), after.flatten().to(torch.int32))
        self.ids.copy_(best.gather(1, leaf[:, None])[:, 0])

    def room(self):
        """Whether every sequence has places for another step's drafts, whatever it keeps."""
        return all(n + self.up.numel() <= c for n, c in zip(self.state.held, self.state.capacity))

    def __call__(self):
        if not self.room():
            raise ValueError("a sequence has no room for the drafts")
        self.state.take([self.most] * self.ids.numel())          # at most
        self.graph.replay()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=512)
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--adapters", type=int, default=0)
    p.add_argument("--draft", action="store_true")
    a = p.parse_args()
    c = Config(layers=a.layers)
    model = Decoder(c, adapters=a.adapters)
    slots = (torch.arange(a.batch, dtype=torch.int32) % a.adapters).cuda() if a.adapters else None
    lens = [a.prompt - (b * a.prompt) // (2 * a.batch) for b in range(a.batch)]
    capacity = a.prompt + a.tokens + 1
    gen = torch.Generator().manual_seed(1)
    ids = torch.randint(0, c.vocab, (sum(lens),), generator=gen).cuda()
    last = (torch.tensor(lens).cumsum(0) - 1).cuda()
    for _ in range(2):                       # the second time is measured
        state = State(c, [n + a.tokens + 1 for n in lens])
        state.slots = slots
        state.advance(lens)
        torch.cuda.synchronize()
        t = time.perf_counter()
        out = model.logits(ids, state, a.prompt, a.prompt, last)
        torch.cuda.synchronize()
        prompt = time.perf_counter() - t
    step = Stepper(model, state, out.argmax(1), capacity)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.tokens):
        step()
    torch.cuda.synchronize()
    decode = time.perf_counter() - t
    if a.draft:
        # two drafts behind each of the first two levels, one behind the next four
        parents = [-1, 0, 0, 1, 1, 2, 2, 3, 4, 5, 6, 7, 8]
        state = State(c, [n + 5 * a.tokens + len(parents) for n in lens])
        state.slots = slots
        state.advance(lens)
        out = model.logits(ids, state, a.prompt, a.prompt, last)
        follow = torch.randint(0, c.vocab, (c.vocab, 2), generator=gen, dtype=torch.int32).cuda()
        tree = TreeStepper(model, state, ids.split(lens), out.argmax(1), parents, follow, max(state.capacity))
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(a.tokens):
            tree()
        torch.cuda.synchronize()
        drafts = time.perf_counter() - t
        kept = int((tree.history_lens - tree.prompt_lens).sum())
        print(f"drafts: {1e3 * drafts / a.tokens:.3f} ms a step, {kept / (a.batch * a.tokens):.2f} tokens kept a step and sequence, "
              f"{kept / drafts:.0f} tokens/s")
    print(f"{c.layers} layers, {a.batch} sequences: prompt of {sum(lens)} tokens {1e3 * prompt:.2f} ms, "
          f"decoding {1e3 * decode / a.tokens:.3f} ms a step, {a.batch * a.tokens / decode:.0f} tokens/s")


if __name__ == "__main__":
    main()
