"""The 64-bit forms' gradients against central differences (CPU)."""
import pytest
import torch

from tests import lm_ref as ref


def differences(f, x, step=1e-5):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros(x.numel(), dtype=x.dtype)
        d[i] = step
        d = d.view_as(x)
        g.view(-1)[i] = (f(x + d) - f(x - d)) / (2 * step)
    return g


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gate(name):
    torch.manual_seed(1)
    x, wg, wu = (torch.randn(*s, dtype=torch.float64) for s in ((3, 5), (4, 5), (4, 5)))
    d = torch.randn(3, 4, dtype=torch.float64)
    dx, dg, du = ref.gate_grad(x, wg, wu, d, name)
    for got, f, at in ((dx, lambda v: (ref.gate(v, wg, wu, name) * d).sum(), x),
                       (dg, lambda v: (ref.gate(x, v, wu, name) * d).sum(), wg),
                       (du, lambda v: (ref.gate(x, wg, v, name) * d).sum(), wu)):
        assert float((got - differences(f, at)).abs().max()) < 1e-8


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_loss(reduction):
    torch.manual_seed(2)
    h, w = torch.randn(5, 4, dtype=torch.float64), torch.randn(7, 4, dtype=torch.float64)
    target = torch.tensor([3, -100, 0, 6, 7])
    d = torch.rand(5, dtype=torch.float64) if reduction == "none" else torch.tensor(0.7, dtype=torch.float64)
    dh, dw = ref.loss_grad(h, w, target, d, 0.6, reduction)
    for got, f, at in ((dh, lambda v: (ref.loss(v, w, target, 0.6, reduction)[0] * d).sum(), h),
                       (dw, lambda v: (ref.loss(h, v, target, 0.6, reduction)[0] * d).sum(), w)):
        assert float((got - differences(f, at)).abs().max()) < 1e-8
    assert float(dh[1].abs().sum()) == 0.0 and float(dh[4].abs().sum()) == 0.0


def test_embed():
    table, tokens = torch.arange(12.0).view(4, 3), torch.tensor([[2, -1], [4, 2]])
    y = ref.embed(table, tokens, 2.0)
    assert y[0, 0].tolist() == [12.0, 14.0, 16.0] and float(y[0, 1].abs().sum() + y[1, 0].abs().sum()) == 0.0
    g = ref.embed_grad(torch.ones(2, 2, 3), tokens, 4, 0.5)
    assert g[2].tolist() == [1.0, 1.0, 1.0] and float(g.sum()) == 3.0
