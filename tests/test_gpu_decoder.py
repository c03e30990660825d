"""The decoder example: its layer against a plain 64-bit model, decoding against the prompt pass, and
the captured step against eager calls.

What separates the layer from its model are the documented roundings of attention (2^-9 rms), of the
linears (below 2^-9) and what they do to int8 codes further on: a value that is off by d crosses a border of
its code with probability d / step and is then off by a step, sqrt(d step) rms.  With rows that span 8 sigma
a step is 2^-5 sigma, so 2^-8 off (both roundings, on the branch's share of the stream) gives 2^-6.5
rms; 2^-5 leaves the two norms of a layer and the final one their sum.  Keys and values of the first layer
depend on the ids alone, so their 4-bit codes are decided by fp32 roundings only.
"""
import pytest
import torch

from tests.gpu_helpers import lib
from tests.serving_model import attention, kv_values, norm_rows

pytestmark = pytest.mark.gpu
RMS = 2.0 ** -5


def example():
    lib()
    from examples import decoder
    return decoder


def small(d, layers):
    return d.Config(hidden=256, ffn=512, heads=8, kv_heads=2, dim=64, layers=layers, vocab=512, group=32)


def dense(w, d):
    codes, scales = d.q.unpack(w)
    s = scales.cpu().double().repeat_interleave(w.group_size, 0).T
    return (codes.cpu().double() - 8) * s


def reference(model, d, ids, lens):
    """Logits [tokens, vocab] of a one-layer model in 64 bits, int8 rows and 4-bit cache as defined."""
    c, layer = model.c, model.layers[0]
    at = [sum(lens[:b]) for b in range(len(lens) + 1)]
    norm = lambda y, h, w: norm_rows(y.float(), h.float(), w.cpu(), d.EPS)
    e = dense(model.embed, d)
    h = e[ids.cpu()] * c.hidden ** 0.5
    h, _, _, _, rows = norm(torch.zeros_like(h), h, layer.norm1)
    xq, xk, xv = ((rows @ dense(w, d).T).float().view(len(h), -1, c.dim) for w in (layer.wq, layer.wk, layer.wv))
    cut = lambda x: [kv_values(x[a:b]) for a, b in zip(at, at[1:])]
    y, _ = attention(xq, cut(xk), cut(xv), lens, lens)
    h, _, _, _, rows = norm(y.flatten(1) @ dense(layer.wo, d).T, h, layer.norm2)
    g, u = (rows @ dense(layer.wu, d).T).chunk(2, 1)
    y = (torch.nn.functional.silu(g) * u) @ dense(layer.wd, d).T
    return norm(y, h, model.norm)[4] @ e.T


def rms(got, want):
    return float((got.cpu().double() - want).square().mean().sqrt() / want.square().mean().sqrt())


@pytest.mark.parametrize("lens", [[1], [40, 7, 70], [200, 129]])
def test_layer_against_its_model(lens):
    d = example()
    print(f"decoder layer lens={lens}", flush=True)
    c = small(d, 1)
    model, state = d.Decoder(c), d.State(c, lens)
    ids = torch.randint(0, c.vocab, (sum(lens),), generator=torch.Generator().manual_seed(2)).cuda()
    state.advance(lens)
    got = model.logits(ids, state, max(lens), max(lens), torch.arange(sum(lens), device="cuda"))
    err = rms(got, reference(model, d, ids, lens))
    print(f"  rms {err:.2e}")
    assert err <= RMS


def test_decoding_follows_the_prompt():
    """Tokens fed one at a time behind a prompt give the logits of one call over all of them."""
    d = example()
    print("decoder one by one", flush=True)
    c = small(d, 1)
    model = d.Decoder(c)
    lens, more = [50, 33], 20
    ids = [torch.randint(0, c.vocab, (n + more,), generator=torch.Generator().manual_seed(n)).cuda() for n in lens]
    want = reference(model, d, torch.cat(ids), [n + more for n in lens])
    state = d.State(c, [n + more for n in lens])
    state.advance(lens)
    model.logits(torch.cat([x[:n] for x, n in zip(ids, lens)]), state, max(lens), max(lens), torch.arange(2, device="cuda"))
    for i in range(more):
        state.advance([1, 1])
        out = model.logits(torch.stack([x[n + i] for x, n in zip(ids, lens)]), state, 1, max(lens) + more,
                           torch.arange(2, device="cuda"))
        rows = torch.tensor([lens[0] + i, lens[0] + more + lens[1] + i])
        assert rms(out, want[rows]) <= RMS, f"token {i}"


def test_captured_steps_equal_eager_ones():
    d = example()
    print("decoder graph", flush=True)
    c = small(d, 2)
    model, lens, steps = d.Decoder(c), [70, 5, 31], 6
    ids = torch.randint(0, c.vocab, (sum(lens),), generator=torch.Generator().manual_seed(2)).cuda()
    last = (torch.tensor(lens).cumsum(0) - 1).cuda()
    runs = []
    for captured in (False, True):
        state = d.State(c, [n + steps + 1 for n in lens])
        state.advance(lens)
        first = model.logits(ids, state, max(lens), max(lens), last)
        outs = [first.clone()]
        step = d.Stepper(model, state, first.argmax(1), max(lens) + steps)
        for _ in range(steps):
            outs.append((step() if captured else step.step()).clone())
            torch.cuda.synchronize()
        runs.append(outs)
    for i, (a, b) in enumerate(zip(*runs)):
        assert torch.equal(a, b), f"step {i}"
