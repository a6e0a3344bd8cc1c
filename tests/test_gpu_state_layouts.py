"""Layouts and head counts of the matrix-state scan against the recurrence in
64 bits: heads before tokens in memory, gates as slices of wider rows, many
value heads on one key head over many chunks.  Tolerances are those of
test_gpu_state_scan.py, which depend on neither; dgate has the bound of the
coarser of its own type and the operands', whose roundings enter it."""
import numpy as np
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests.test_gpu_state_scan import BF, DEV, F32, Case, close

pytestmark = pytest.mark.gpu


def heads_first(x):
    """The same values, in memory [batch, heads, tokens, ...] (packed: [heads, tokens, ...])."""
    h = 2 if x.dim() == 4 else 1
    return x.transpose(h - 1, h).contiguous().transpose(h - 1, h)


def check(c):
    out, fin = gs.state_scan_forward(*c.args(), **c.kw(), final_state=True)
    g = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw(),
                               d_final_state=None if c.dsT is None else c.dsT.to(DEV))
    torch.cuda.synchronize()
    fwd, bwd = [c.ref(i) for i in range(len(c.lens))], [c.ref(i, grad=True) for i in range(len(c.lens))]
    close(c.flat(out), np.concatenate([r[0] for r in fwd]), c.dtype, "out")
    close(fin, np.stack([r[1] for r in fwd]), F32, "final state")
    for j, what in enumerate(("dq", "dk", "dv", "dgate")):
        dt = BF if what == "dgate" and c.host["a"].dtype == BF else c.dtype
        close(c.flat(g[j]), np.concatenate([r[j] for r in bwd]), dt, what)
    if c.s0 is not None:
        close(g[4], np.stack([r[4] for r in bwd]), F32, "d_initial_state")


@pytest.mark.parametrize("gate_dtype", [F32, BF], ids=["gate f32", "gate bf16"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
def test_heads_before_tokens_and_gates_in_wider_rows(packed, dtype, gate_dtype):
    print(f"case layouts: packed {packed} {dtype} gate {gate_dtype}", flush=True)
    c = Case([150, 3, 81] if packed else [150] * 2, H=6, Hk=2, Dk=64, Dv=40, dtype=dtype, gate_dtype=gate_dtype,
             packed=packed, state=True)
    for n in ("q", "k", "v", "do"):
        c.dev[n] = heads_first(c.dev[n])
        assert not c.dev[n].is_contiguous()
    a = c.dev["a"]
    wide = torch.full((*a.shape[:-1], 37), 9.0, dtype=a.dtype, device=DEV)
    wide[..., 5:5 + 2 * c.host["a"].shape[1]:2] = a  # every other column
    c.dev["a"] = wide[..., 5:5 + 2 * c.host["a"].shape[1]:2]
    check(c)
    if not packed:  # tokens of a head follow each other
        c.dev["a"] = a.transpose(1, 2).contiguous().transpose(1, 2)
        check(c)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("lens,H,Dk,Dv", [([700], 16, 64, 64), ([260, 0, 131, 9], 12, 128, 40)])
def test_many_value_heads_on_one_key_head(lens, H, Dk, Dv, dtype):
    print(f"case one key head: {lens} {H} {Dk} {Dv} {dtype}", flush=True)
    check(Case(lens, H=H, Hk=1, Dk=Dk, Dv=Dv, dtype=dtype, packed=len(lens) > 1, state=len(lens) > 1, shift=3.0))
