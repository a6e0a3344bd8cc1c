"""gated_projection, linear_cross_entropy and embed on rows further apart than the
library reads them: the last token of each long sequence, weights in such a layout, and
upstream gradients that come as slices of a stacked batch.  The results are those of
dense copies, bit for bit; the calls under them refuse."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
T, D = 2 ** 18 + 1, 8  # T * D is past 2^21
GEN = torch.Generator()


def normal(*shape, dtype):
    return torch.randn(*shape, generator=GEN).to(dtype).to(DEV)


def last_of(dense):
    """dense [n, D] as the last tokens of n sequences."""
    x = torch.zeros(len(dense), T, D, dtype=dense.dtype, device=DEV)
    x[:, -1] = dense
    return x.requires_grad_()


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_gated_projection(n, dtype):
    GEN.manual_seed(1)
    x, wg, wu, d = (normal(*s, dtype=dtype) for s in ((n, D), (16, D), (16, D), (n, 16)))
    leaves = last_of(x), last_of(wg), last_of(wu)
    slices = [t[:, -1] for t in leaves]
    assert all(t.stride(0) > 2 ** 21 for t in slices)
    y = gs.gated_projection(*slices)
    assert torch.equal(y, gs.gated_projection_forward(x, wg, wu))
    y.backward(d)
    for leaf, g in zip(leaves, gs.gated_projection_backward(x, wg, wu, d)):
        assert torch.equal(leaf.grad[:, -1], g) and float(leaf.grad[:, :-1].abs().max()) == 0.0
    with pytest.raises(gs.GScanError):
        gs.gated_projection_forward(slices[0].detach(), wg, wu)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_linear_cross_entropy(n, dtype):
    GEN.manual_seed(2)
    h, w = normal(n, D, dtype=dtype), normal(21, D, dtype=dtype)
    target = torch.randint(-2, 21, (n,), generator=GEN).to(DEV)
    leaves = last_of(h), last_of(w)
    loss = gs.linear_cross_entropy(leaves[0][:, -1], leaves[1][:, -1], target)
    want, lse = gs.linear_cross_entropy_forward(h, w, target)
    assert torch.equal(loss.detach(), want)
    loss.backward()
    for leaf, g in zip(leaves, gs.linear_cross_entropy_backward(h, w, target, lse, torch.ones((), device=DEV))):
        assert torch.equal(leaf.grad[:, -1], g) and float(leaf.grad[:, :-1].abs().max()) == 0.0
    with pytest.raises(gs.GScanError):
        gs.linear_cross_entropy_forward(leaves[0][:, -1].detach(), w, target)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_upstream_gradients_that_are_slices(dtype):
    """Each step's output is stacked with others of its batch: its gradient comes back as a
    view whose rows are a whole sequence apart."""
    GEN.manual_seed(3)
    steps, F = 1030, 2048  # steps * F is past 2^21
    x, wg, wu = (normal(*s, dtype=dtype).requires_grad_() for s in ((4, D), (F, D), (F, D)))
    d = torch.zeros(4, steps, F, dtype=dtype, device=DEV)
    d[:, 5] = normal(4, F, dtype=dtype)
    seen = []
    y = gs.gated_projection(x, wg, wu)
    y.register_hook(lambda g: seen.append(g.stride()))
    rest = torch.zeros(4, F, dtype=dtype, device=DEV)
    torch.stack([rest] * 5 + [y] + [rest] * (steps - 6), 1).backward(d)
    assert seen[0][0] == steps * F  # (else nothing was tested)
    for t, g in zip((x, wg, wu), gs.gated_projection_backward(x.detach(), wg.detach(), wu.detach(),
                                                              d[:, 5].contiguous())):
        assert torch.equal(t.grad, g)


def test_numbers_are_refused():
    x, w, t = torch.ones((), device=DEV), torch.ones(8, 8, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    for call in (lambda: gs.embed(x, t), lambda: gs.gated_projection(x, w, w), lambda: gs.gated_projection(w, x, w),
                 lambda: gs.linear_cross_entropy(x, w, t), lambda: gs.linear_cross_entropy(w, x, t)):
        with pytest.raises(ValueError):
            call()
