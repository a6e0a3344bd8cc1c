"""Gradients of the cross entropy where no token counts: sums over no tokens, zero
whatever reaches the loss (a sum divided by the number of tokens that count brings an
infinity or a NaN)."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 1.0])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("n", [0, 5, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_zero(dtype, n, reduction, value):
    gen = torch.Generator().manual_seed(4)
    h = torch.randn(n, 264, generator=gen).to(dtype).to(DEV)
    w = torch.randn(333, 264, generator=gen).to(dtype).to(DEV)
    target = torch.full((n,), -100, device=DEV)
    loss, lse = gs.linear_cross_entropy_forward(h, w, target, reduction=reduction)
    assert bool((loss == 0).all()) and bool((lse == 0).all())
    d = torch.full(loss.shape, value, device=DEV)
    dh, dw = gs.linear_cross_entropy_backward(h, w, target, lse, d, reduction=reduction)
    assert bool((dh == 0).all()) and bool((dw == 0).all())


def test_mean_taken_by_the_caller():
    h = torch.ones(40, 16, device=DEV, requires_grad=True)
    w = torch.ones(9, 16, device=DEV, requires_grad=True)
    target = torch.full((40,), -1, device=DEV)
    (gs.linear_cross_entropy(h, w, target, reduction="sum") / (target >= 0).sum()).backward()
    assert bool((h.grad == 0).all()) and bool((w.grad == 0).all())
