"""The example layer: packed training with gradients for every parameter, and
token by token what the whole sequence gives."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("mixing_layer", os.path.join(ROOT, "examples", "mixing_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_continue_a_prompt(example):
    """A prompt's states, then steps, against the scan of the whole.  float32:
    both ways hold sums of the same terms, at most 90 of them, in 32 bits; the
    projections' roundings are the same rows' in other tilings.  2e-4 of the
    largest output is 90 terms * 2^-24 * 4 stages * a factor 9 for the norms."""
    torch.manual_seed(3)
    layer = example.MixingLayer(128, heads=4, key_heads=2, key_width=32, value_width=40, dtype=torch.float32)
    lengths, more = [37, 1, 70], 20
    x = torch.randn(sum(lengths) + 3 * more, 128, device="cuda")
    full_off, full_pos = example.pack([n + more for n in lengths])
    starts = full_off[:-1].tolist()
    with torch.no_grad():
        want, end = layer(x, full_pos, full_off)
        head = torch.cat([x[s:s + n] for s, n in zip(starts, lengths)])
        off, pos = example.pack(lengths)
        got, states = layer(head, pos, off)
        rows = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, lengths)]).cuda()
        big = float(want.abs().max())
        assert float((got - want[rows]).abs().max()) <= 2e-4 * big
        slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
        pool = torch.full((5, *states.shape[1:]), 7.0, device="cuda")
        pool[slots.long()] = states
        at = torch.tensor(lengths, device="cuda")
        first = torch.tensor(starts, device="cuda")
        for _ in range(more):
            y = layer.step(x[first + at], at, pool, slots)
            assert float((y - want[first + at]).abs().max()) <= 2e-4 * big
            at = at + 1
        assert float((pool[slots.long()] - end).abs().max()) <= 2e-4 * float(end.abs().max())
        assert bool((pool[[1, 3]] == 7.0).all())  # nobody else's states


def test_training_learns_and_reaches_every_parameter(example):
    torch.manual_seed(5)
    gen = torch.Generator().manual_seed(6)
    model = example.Model()
    losses = example.train(model, 60, gen)
    assert all(p.grad is not None and bool(p.grad.abs().sum() > 0) for p in model.parameters())
    # 64 tokens by chance: 4.16; of a cycle of 16 only the first 16 of a sequence cannot be known:
    # 16 / 120 of the tokens at up to ln 64 leave 0.55
    assert losses[0] > 3.5 and losses[-1] < 2.0
