"""The decoder example's sequences between captured steps: prompt chunks, the offsets a graph keeps, and
the capacity.  The bound is test_gpu_decoder's."""
import pytest
import torch

from tests.test_gpu_decoder import RMS, example, reference, rms, small

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_a_chunk_between_steps(captured):
    """Single tokens, a chunk of several, single tokens again: each gives the logits of one call over all
    tokens, whatever other work has reused the memory of the chunk's arguments."""
    d = example()
    print(f"decoder chunk between steps captured={captured}", flush=True)
    c = small(d, 1)
    model = d.Decoder(c)
    lens, singles, chunk = [50, 33, 5], 3, [4, 1, 9]
    total = [n + 2 * singles + m for n, m in zip(lens, chunk)]
    ids = [torch.randint(0, c.vocab, (n,), generator=torch.Generator().manual_seed(n)).cuda() for n in total]
    want = reference(model, d, torch.cat(ids), total)
    row = [sum(total[:b]) for b in range(3)]
    state, at = d.State(c, total), [0, 0, 0]

    def take(news):
        out = torch.cat([x[a:a + m] for x, a, m in zip(ids, at, news)])
        for b, m in enumerate(news):
            at[b] += m
        return out

    def check(out, label):
        torch.cuda.synchronize()
        err = rms(out, want[torch.tensor([r + a - 1 for r, a in zip(row, at)])])
        print(f"  {label}: rms {err:.2e}", flush=True)
        assert err <= RMS, label

    def prompt(news):
        state.advance(news)
        last = torch.tensor(news).cumsum(0).cuda() - 1
        return model.logits(take(news), state, max(news), max(total), last)

    check(prompt(lens), "prompt")
    step = d.Stepper(model, state, torch.zeros(3, dtype=torch.int64, device="cuda"), max(total))

    def single(label):
        step.ids.copy_(take([1, 1, 1]))
        check(step() if captured else step.step(), label)

    for i in range(singles):
        single(f"token {i}")
    check(prompt(chunk), "chunk")
    keep = [torch.full((n,), 7, dtype=torch.int32, device="cuda") for n in (3, 4, 4, 4, 4, 128) for _ in range(20)]
    for i in range(singles):
        single(f"token {i} behind the chunk")
    assert len(keep) == 120


def test_capacity():
    """Tokens past a sequence's capacity are refused before anything is launched."""
    d = example()
    print("decoder capacity", flush=True)
    c = small(d, 1)
    model, state = d.Decoder(c), d.State(c, [40, 20])
    with pytest.raises(ValueError):
        state.advance([41, 1])
    state.advance([38, 20 - 2])
    ids = torch.zeros(56, dtype=torch.int64, device="cuda")
    model.logits(ids, state, 38, 38, torch.tensor([37, 55]).cuda())
    step = d.Stepper(model, state, ids[:2], 40)
    step()
    step.step()
    for call in (step, step.step):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert state.lens.tolist() == [40, 20]
