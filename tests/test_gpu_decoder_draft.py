"""The decoder example with drafted trees and with adapters: what a step chooses against a plain 64-bit model,
captured steps, and adapters against one merged model each.

Bounds.  A chosen token is the greedy one of logits that are off by RMS of the logits' own rms (test_gpu_decoder):
in 512 logits the largest of normal errors is below 5 times that, and the difference of two such is what may
turn a choice."""
import pytest
import torch

from tests.test_gpu_decoder import RMS, dense, example, reference, rms, small

pytestmark = pytest.mark.gpu
TREE = [-1, 0, 0, 1, 1, 2, 3, 3, 6]


def start(d, model, c, lens, room, slots=None):
    ids = [torch.randint(0, c.vocab, (n,), generator=torch.Generator().manual_seed(n)).cuda() for n in lens]
    state = d.State(c, [n + room for n in lens])
    state.slots = slots
    state.advance(lens)
    out = model.logits(torch.cat(ids), state, max(lens), max(lens), (torch.tensor(lens).cumsum(0) - 1).cuda())
    return ids, state, out.argmax(1)


def greedy(d, model, c, lens, steps):
    """Tokens of plain greedy decoding, [batch][steps]."""
    ids, state, first = start(d, model, c, lens, steps + 1)
    step, out = d.Stepper(model, state, first, max(lens) + steps), [first]
    for _ in range(steps):
        out.append(step().argmax(1).clone())
    return ids, torch.stack(out, 1)


@pytest.mark.parametrize("known", [False, True])
def test_drafted_steps_choose_greedy_tokens(known):
    """With a table of random drafts, and with one that knows plain decoding's tokens (several are kept a step)."""
    d = example()
    c = small(d, 1)
    model, lens, steps = d.Decoder(c), [50, 33, 7], 10
    gen = torch.Generator().manual_seed(4)
    follow = torch.randint(0, c.vocab, (c.vocab, 2), generator=gen, dtype=torch.int32).cuda()
    if known:
        _, told = greedy(d, model, c, lens, 40)
        follow[told[:, :-1].flatten(), 1] = told[:, 1:].flatten().to(torch.int32)
    ids, state, first = start(d, model, c, lens, 120)
    tree = d.TreeStepper(model, state, ids, first, TREE, follow, max(lens) + 120)
    for _ in range(steps):
        tree()
    torch.cuda.synchronize()
    n = tree.history_lens.tolist()
    assert state.lens.tolist() == n
    made = [b - a for a, b in zip(lens, n)]
    print(f"drafts known={known}: {made} tokens in {steps} steps", flush=True)
    assert min(made) >= steps
    if known:
        assert max(made) > steps
    told = [tree.history[b, :k].long() for b, k in enumerate(n)]
    want = reference(model, d, torch.cat(told), n)
    size = float(want.square().mean().sqrt())
    at = 0
    for b, k in enumerate(n):
        rows = want[at + lens[b] - 1:at + k]
        then = torch.cat([told[b][lens[b]:], tree.ids[b:b + 1]]).cpu()
        short = rows.max(1).values - rows.gather(1, then[:, None])[:, 0]
        assert float(short.max()) <= 2 * 5 * RMS * size, f"sequence {b}: a token {float(short.max()):.3f} below the best"
        at += k
    # and the cache holds what a prompt pass over the kept tokens stores
    state2 = d.State(c, [k + 9 for k in n])
    state2.advance(n)
    model.logits(torch.cat(told), state2, max(n), max(n), torch.zeros(1, dtype=torch.long, device="cuda"))
    cu = torch.tensor([sum(n[:b]) for b in range(4)], dtype=torch.int32, device="cuda")
    for x, y in zip(d.q.kv_read(state.caches[0], state.table, cu, state.lens, sum(n)),
                    d.q.kv_read(state2.caches[0], state2.table, cu, state2.lens, sum(n))):
        # the first layer's keys and values depend on the ids alone: fp32 sums in another order decide few codes otherwise
        assert float((x != y).float().mean()) < 0.01


def test_a_penalty_forbids_what_was_said():
    """A huge repetition penalty turns positive logits of said tokens to nothing and drives negative ones far
    down: no token comes twice."""
    d = example()
    c = small(d, 1)
    model, lens = d.Decoder(c), [20, 11]
    follow = torch.randint(0, c.vocab, (c.vocab, 2), generator=torch.Generator().manual_seed(4), dtype=torch.int32).cuda()
    ids, state, first = start(d, model, c, lens, 120)
    tree = d.TreeStepper(model, state, ids, first, TREE, follow, 140, penalty=1e6)
    for _ in range(12):
        tree()
    torch.cuda.synchronize()
    for b, k in enumerate(tree.history_lens.tolist()):
        said = tree.history[b, lens[b]:k].tolist()
        # the first one was chosen by the prompt's pass, without the rules
        assert len(set(said[1:])) == len(said) - 1
        assert not set(said[1:]) & set(ids[b].tolist())


def test_no_room():
    d = example()
    c = small(d, 1)
    model = d.Decoder(c)
    follow = torch.zeros(c.vocab, 2, dtype=torch.int32, device="cuda")
    ids, state, first = start(d, model, c, [20], 30)
    tree = d.TreeStepper(model, state, ids, first, TREE, follow, 50)
    with pytest.raises(ValueError):
        for _ in range(30):
            tree()
    torch.cuda.synchronize()
    assert 20 < int(state.lens) <= 50


def test_adapters():
    """A batch with an adapter of its own for every sequence, and one without, gives each sequence what a model
    with that adapter merged into its weights gives (64 bits, the base's 4-bit weights as they are)."""
    d = example()
    c = small(d, 1)
    model, lens = d.Decoder(c, adapters=3, rank=8), [40, 7, 70, 12]
    ids, state, _ = start(d, model, c, lens, 9, torch.tensor([2, 0, 1, -1], dtype=torch.int32, device="cuda"))
    state = d.State(c, lens)
    state.slots = torch.tensor([2, 0, 1, -1], dtype=torch.int32, device="cuda")
    state.advance(lens)
    got = model.logits(torch.cat(ids), state, max(lens), max(lens), torch.arange(sum(lens), device="cuda")).cpu().double()
    layer, eye, at = model.layers[0], torch.eye, 0
    plain = dense
    for n, x, slot in zip(lens, ids, state.slots.tolist()):
        change = {}
        for w, s in ((layer.wq, layer.adapters.q), (layer.wv, layer.adapters.v), (layer.wo, layer.adapters.o), (layer.wd, layer.adapters.d)):
            one = torch.full((s.K,), slot, dtype=torch.int32, device="cuda")
            # the set's own term on unit rows: alpha (B A)^T
            change[id(w)] = d.q.adapters_add(torch.zeros(s.K, s.N, device="cuda"), eye(s.K, device="cuda"), s, one).cpu().double().T
        import tests.test_gpu_decoder as base
        base.dense = lambda w, d: plain(w, d) + change.get(id(w), 0.0)
        try:
            want = reference(model, d, x, [n])
        finally:
            base.dense = plain
        err = rms(got[at:at + n], want)
        print(f"adapter {slot}: rms {err:.2e}", flush=True)
        assert err <= RMS
        if slot >= 0:
            # the adapters' terms have a tenth of their projections' size: the model without them has to be further off
            assert 4 * err < rms(got[at:at + n], reference(model, d, x, [n]))
        at += n
