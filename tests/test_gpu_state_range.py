"""The bf16 backward keeps its chunks' states in 16 bits with a power of two
per tile: that inputs of any magnitude give the same bits, scaled, and that
gradients of gates that remember far are as exact as the operands allow."""
import numpy as np
import pytest
import torch

from gated_linear_recurrence_history_amd import state_scan_backward, state_scan_forward
from . import state_ref as sr

pytestmark = pytest.mark.gpu
DEV = "cuda"


def case(T, H, Dk, Dv, shift, seed, gate=torch.float32):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    q, k, v, do = (t(1, T, H, d).bfloat16() for d in (Dk, Dk, Dv, Dv))
    return q, k, v, (t(1, T, H) + shift).to(gate), do


@pytest.mark.parametrize("power", [-70, -30, 30, 70])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128)])
def test_powers_of_two_pass_through(power, Dk, Dv):
    """v times 2^p: out, the final state, dq, dk and dgate are 2^p times the
    same bits (nothing leaves the range of bf16), dv is the same."""
    q, k, v, a, do = (x.to(DEV) for x in case(300, 2, Dk, Dv, 3.0, 11, torch.bfloat16))
    f = 2.0 ** power
    kw = dict(scale=Dk ** -0.5)
    o, S = state_scan_forward(q, k, v, a, final_state=True, **kw)
    o2, S2 = state_scan_forward(q, k, v * f, a, final_state=True, **kw)
    assert torch.equal(o.float() * f, o2.float()) and torch.equal(S * f, S2)
    g = state_scan_backward(q, k, v, a, do, **kw)
    g2 = state_scan_backward(q, k, v * f, a, do, **kw)
    for i, name in enumerate(("dq", "dk", "dv", "dgate")):
        want = g[i].float() * (1.0 if name == "dv" else f)
        assert torch.equal(want, g2[i].float()), name
    # and of the upstream gradient: all four follow it
    g3 = state_scan_backward(q, k, v, a, do * f, **kw)
    for i, name in enumerate(("dq", "dk", "dv", "dgate")):
        assert torch.equal(g[i].float() * f, g3[i].float()), name


@pytest.mark.parametrize("Dk,Dv", [(128, 64), (64, 128)])
def test_gradient_of_gates_that_remember(Dk, Dv):
    """Gates about sigmoid(7): <S, dS> over the whole width is most of the
    gradient.  Its states have 11 bits (2^-12 / sqrt(3) each, over many terms);
    the chunk's own terms have bf16 states, each part no larger than the whole:
    sqrt(2) 2^-9 / sqrt(3) = 1.6e-3.  Both: below 2e-3 of the norm (with 8 bits in
    the first it was 2.8e-3).  float32 gates: nothing else is rounded."""
    q, k, v, a, do = case(1500, 2, Dk, Dv, 7.0, 5)
    got = state_scan_backward(*(x.to(DEV) for x in (q, k, v, a, do)), scale=Dk ** -0.5)[3]
    x = [t[0].double().numpy() for t in (q, k, v, a)]
    ref = sr.scan_grad(*x, do[0].double().numpy(), Dk ** -0.5, "sigmoid", 0.0)[3]
    err = np.linalg.norm(got[0].double().cpu().numpy() - ref) / np.linalg.norm(ref)
    print(f"  dgate rel {err:.2e}", flush=True)
    assert err <= 2e-3
