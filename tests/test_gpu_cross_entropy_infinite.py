"""Logits of plus infinity: the log-sum is infinite, as log sum exp is, and so is the
loss of any other class; that of the infinite one is inf - inf, NaN."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests import lm_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("n", [1, 7, 32, 33, 300])
@pytest.mark.parametrize("V,bad", [(1, 0), (40, 7), (3001, 0), (3001, 1500), (3001, 3000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_log_sum(dtype, V, bad, n):
    gen = torch.Generator().manual_seed(5)
    h, w = torch.randn(n, 72, generator=gen).to(dtype), (torch.randn(V, 72, generator=gen) * 0.3).to(dtype)
    h[:, 3] = torch.where(h[:, 3] >= 0, h[:, 3] + 1, h[:, 3] - 1)  # no zero
    target = torch.randint(0, V, (n,), generator=gen)
    target[::2] = bad
    # the class's logit is plus infinity for tokens with h > 0, minus infinity for the others
    w[bad, 3] = float("inf")
    loss, lse = gs.linear_cross_entropy_forward(h.to(DEV), w.to(DEV), target.to(DEV), reduction="none")
    z = h.double() @ w.double().T
    above, hit = h[:, 3] > 0, target == bad
    want, lse, loss = torch.logsumexp(z, -1), lse.double().cpu(), loss.double().cpu()
    assert bool((lse[above] == float("inf")).all())
    assert bool((loss[above & ~hit] == float("inf")).all()) and bool(torch.isnan(loss[above & hit]).all())
    # minus infinity: no part in the sum; alone it is the sum
    if V == 1:
        assert bool((lse[~above] == -float("inf")).all()) and bool(torch.isnan(loss[~above]).all())
        return
    top = float(z.masked_fill(torch.isinf(z), 0.0).abs().max())
    tol = (top + 1) * (ref.product(72) + 12 * ref.U) + 80 * ref.U
    if not bool(above.all()):
        assert float((lse - want)[~above].abs().max()) <= tol
    assert bool((loss[~above & hit] == float("inf")).all())
    for reduction in ("sum", "mean"):
        total, again = gs.linear_cross_entropy_forward(h.to(DEV), w.to(DEV), target.to(DEV), reduction=reduction)
        assert torch.equal(again.double().cpu(), lse) and not bool(torch.isfinite(total))


@pytest.mark.parametrize("n", [5, 90])
def test_no_number_beside_infinity(n):
    """NaN is not hidden by an infinite logit, wherever both are."""
    h, w = torch.ones(n, 16, device=DEV), torch.zeros(2000, 16, device=DEV)
    for inf, nan in ((0, 1), (1, 0), (0, 1999), (1999, 0), (700, 701)):
        w.zero_()
        w[inf, 2], w[nan, 2] = float("inf"), float("nan")
        _, lse = gs.linear_cross_entropy_forward(h, w, torch.full((n,), 5, device=DEV))
        assert bool(torch.isnan(lse).all())


@pytest.mark.parametrize("n", [5, 90])
def test_products_past_the_largest_number(n):
    """Finite operands whose product is not."""
    h = torch.full((n, 8), 1e20, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(50, 8, dtype=torch.bfloat16, device=DEV)
    w[9], w[10] = 1e20, 1e-20
    loss, lse = gs.linear_cross_entropy_forward(h, w, torch.full((n,), 10, device=DEV), reduction="none")
    assert bool((lse == float("inf")).all()) and bool((loss == float("inf")).all())
