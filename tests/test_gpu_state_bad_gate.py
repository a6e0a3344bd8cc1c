"""How far a gate that is no number reaches: forwards its own and later tokens;
backwards dq of its own and later tokens, dk and dv of earlier ones and of the
rest of its chunk (at most 63 tokens), dgate; no other head or sequence."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests.test_gpu_state_scan import BF, F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("form,value", [("sigmoid", float("nan")), ("log", float("nan")), ("log", float("inf"))])
@pytest.mark.parametrize("t", [0, 70, 127, 199])
def test_a_gate_that_is_no_number(t, form, value, dtype):
    print(f"case bad gate: token {t} {form} {value} {dtype}", flush=True)
    c = Case([200] * 2, H=4, Hk=4, Dk=64, Dv=40, dtype=dtype, form=form, shift=0.0 if form == "log" else 1.5,
             state=True)
    ops = [*c.args(), c.dev["do"]]
    bad = [x.clone() for x in ops]
    bad[3][1, t, 2] = value
    clean = (gs.state_scan_forward(*ops[:4], **c.kw()), *gs.state_scan_backward(*ops, **c.kw())[:4])
    got = (gs.state_scan_forward(*bad[:4], **c.kw()), *gs.state_scan_backward(*bad, **c.kw())[:4])
    torch.cuda.synchronize()
    for x, y, name in zip(got, clean, ("out", "dq", "dk", "dv", "dgate")):
        assert torch.equal(x[0], y[0]) and torch.equal(x[:, :, [0, 1, 3]], y[:, :, [0, 1, 3]]), name
        if name in ("out", "dq"):
            assert torch.equal(x[1, :t, 2], y[1, :t, 2]), name
            assert not bool(torch.isfinite(x[1, t, 2]).any()), name
        elif name in ("dk", "dv"):
            assert torch.equal(x[1, t + 64:, 2], y[1, t + 64:, 2]), name
            assert t == 0 or not bool(torch.isfinite(x[1, t - 1, 2]).any()), name
