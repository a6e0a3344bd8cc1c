"""The final state written over the initial one, where sequences are divided
among workgroups of one launch: the same bits as with two arrays, however the
workgroups are scheduled (another stream keeps the GPU busy beside some of the
calls)."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests.test_gpu_state_scan import BF, DEV, F32, Case

pytestmark = pytest.mark.gpu

CASES = {
    "one sequence": dict(lens=[3001], H=2, Hk=1, Dk=128, Dv=64),
    "batch": dict(lens=[2100] * 2, H=3, Hk=3, Dk=64, Dv=128),
    "short last part": dict(lens=[2 * 1024 + 1], H=4, Hk=2, Dk=96, Dv=80),
    "packed": dict(lens=[1700, 0, 5, 2300, 64], H=3, Hk=1, Dk=72, Dv=40, packed=True),
}


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_in_place_states_of_divided_sequences(name, dtype):
    print(f"case in place: {name} {dtype}", flush=True)
    c = Case(dtype=dtype, state=True, shift=4.0, **CASES[name])
    assert gs.state_scan_forward_workspace_bytes(*c.args(), c.off) > 0  # it is divided
    kw = c.kw()
    first = kw.pop("initial_state")
    want = gs.state_scan_forward(*c.args(), **kw, initial_state=first, final_state=True)
    busy, side = torch.randn(2048, 2048, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    for beside in (False, True, True):
        if beside:
            with torch.cuda.stream(side):
                for _ in range(8):
                    busy.mm(busy)
        state = first.clone()
        out, fin = gs.state_scan_forward(*c.args(), **kw, initial_state=state, final_state=state)
        torch.cuda.synchronize()
        assert fin is state and torch.equal(out, want[0]) and torch.equal(state, want[1])
