"""A small decoder served with 4-bit weights, int8 activations and a 4-bit key/value cache.

Every layer is
    h, rows = h + y, int8 rows of rmsnorm(h)       rmsnorm_dq8ca
    q, k, v = rows . W^T                           linear_dq8ca_rows, three weights on one set of rows
    cache  <- k, v;  y = attention(q, cache)       kv_append, kv_attention
    h, rows = h + y . Wo^T, int8 rows of its norm  linear_fwd, rmsnorm_dq8ca
    y = (silu(g) * u) . Wd^T, [g u] = rows . Wu^T  linear_dq8ca_rows, linear_fwd
on random weights, without positions (nothing rotates q and k on their way).  Run as a command it
takes a batch of prompts of unlike lengths in one call and then decodes from a captured HIP graph:

    python examples/decoder.py [--layers 4] [--batch 8] [--prompt 512] [--tokens 64]
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


class Decoder:
    def __init__(self, c, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.c = c
        self.embed = random_weight(c.vocab, c.hidden, c.group, gen)      # also the output weight
        self.layers = [Layer(c, gen) for _ in range(c.layers)]
        self.norm = 1 + 0.1 * torch.randn(c.hidden, generator=gen).cuda()

    def hidden(self, h, state, max_new, max_ctx, last):
        """The normalised rows `last` of the final stream for the embedded new tokens h [tokens, hidden]."""
        c, T = self.c, h.shape[0]
        y = torch.zeros_like(h)
        for layer, cache in zip(self.layers, state.caches):
            rows, h, _ = q.rmsnorm_dq8ca(y, layer.norm1, EPS, residual=h)
            xq, xk, xv = (q.linear_dq8ca_rows(w, rows).view(T, -1, c.dim) for w in (layer.wq, layer.wk, layer.wv))
            q.kv_append(cache, xk, xv, state.table, state.cu, state.lens)
            a = q.kv_attention(cache, xq, state.table, state.cu, state.lens, max_new, max_ctx)
            y = q.linear_fwd(layer.wo, a.view(T, -1))
            rows, h, _ = q.rmsnorm_dq8ca(y, layer.norm2, EPS, residual=h)
            g, u = q.linear_dq8ca_rows(layer.wu, rows).chunk(2, 1)
            y = q.linear_fwd(layer.wd, torch.nn.functional.silu(g) * u)
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


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=512)
    p.add_argument("--tokens", type=int, default=64)
    a = p.parse_args()
    c = Config(layers=a.layers)
    model = Decoder(c)
    lens = [a.prompt - (b * a.prompt) // (2 * a.batch) for b in range(a.batch)]
    capacity = a.prompt + a.tokens + 1
    gen = torch.Generator().manual_seed(1)
    ids = torch.randint(0, c.vocab, (sum(lens),), generator=gen).cuda()
    last = (torch.tensor(lens).cumsum(0) - 1).cuda()
    for _ in range(2):                       # the second time is measured
        state = State(c, [n + a.tokens + 1 for n in lens])
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
    print(f"{c.layers} layers, {a.batch} sequences: prompt of {sum(lens)} tokens {1e3 * prompt:.2f} ms, "
          f"decoding {1e3 * decode / a.tokens:.3f} ms a step, {a.batch * a.tokens / decode:.0f} tokens/s")


if __name__ == "__main__":
    main()
