"""The operators together, as the example uses them: gradients for every parameter
against a plain form of the model, and token by token what the whole sequence gives."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("language_model", os.path.join(ROOT, "examples", "language_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def small(example, dtype):
    torch.manual_seed(3)
    return example.LanguageModel(vocabulary=50, width=64, inner=72, layers=2, dtype=dtype, heads=2, key_heads=1,
                                 key_width=32, value_width=24)


def batch(example, lengths=(37, 1, 70)):
    offsets, positions = example.pack(lengths)
    gen = torch.Generator().manual_seed(4)
    tokens = torch.randint(0, 50, (sum(lengths),), generator=gen).cuda()
    target = torch.roll(tokens, -1)
    target[(offsets[1:] - 1).long()] = -100
    return tokens, target, positions, offsets


def test_gradients(example, monkeypatch):
    """float32, against the same model with the three operators in torch's own elementary
    operations.  Both have fp32 roundings of sums of at most 108 terms through 2 layers of
    6 products each: 2^-24 sqrt(108) for each, a factor 20 for the norms between."""
    model = small(example, torch.float32)
    model.loss(*batch(example)).backward()
    got = {n: p.grad.clone() for n, p in model.named_parameters()}
    gs = example.gs

    def embed(table, tokens, scale=1.0, dtype=None):
        return table[tokens] * scale

    def gated(x, wg, wu):
        a = x @ wg.T
        return a * torch.sigmoid(a) * (x @ wu.T)

    def entropy(h, w, target):
        z = torch.log_softmax(h @ w.T, -1)
        return -z[target >= 0, target[target >= 0]].mean()

    monkeypatch.setattr(gs, "embed", embed)
    monkeypatch.setattr(gs, "gated_projection", gated)
    monkeypatch.setattr(gs, "linear_cross_entropy", entropy)
    model.zero_grad()
    model.loss(*batch(example)).backward()
    for name, p in model.named_parameters():
        assert float((got[name] - p.grad).norm()) <= 12 * 20 * 2.0 ** -24 * 11 * float(p.grad.norm()), name


def test_steps_continue_a_prompt(example):
    """float32: the same sums in other orders, as above; largest element."""
    model = small(example, torch.float32)
    tokens, _, positions, offsets = batch(example)
    starts, lengths = offsets[:-1].tolist(), (offsets[1:] - offsets[:-1]).tolist()
    with torch.no_grad():
        want = model.logits(model(tokens, positions, offsets)[0])
        pools = [torch.zeros(4, 2, 32, 24, device="cuda") for _ in range(2)]
        slots = torch.tensor([2], dtype=torch.int32, device="cuda")
        before = torch.zeros(1, dtype=torch.int64, device="cuda")
        for i in range(lengths[2]):
            at, token = torch.tensor([i], device="cuda"), tokens[starts[2] + i].view(1)
            y = model.step(token, before, at, pools, slots)
            before = token
            assert float((y[0] - want[starts[2] + i]).abs().max()) <= 4 * 12 * 20 * 2.0 ** -24 * 11 * float(want.abs().max())


def test_runs_in_bfloat16(example):
    torch.manual_seed(5)
    model = example.LanguageModel(layers=1)
    losses = example.train(model, 3, torch.Generator().manual_seed(6))
    assert all(l == l and l < 100 for l in losses)
    assert all(p.grad is not None and bool(p.grad.abs().sum() > 0) for p in model.parameters())
    made = example.generate(model, [torch.arange(1, 9), torch.arange(3, 40)], 5, pool_size=3)
    assert made.shape == (2, 5) and int(made.min()) >= 0 and int(made.max()) < 64
