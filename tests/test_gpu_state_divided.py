"""The matrix-state scan where the work is divided: long sequences walked in
parts, and more chunks than workgroups, which then take several of them one
after the other.  Tolerances are those of test_gpu_state_scan.py, which do not
depend on lengths: norms of independent roundings against norms of results."""
import numpy as np
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests import test_gpu_qk_norm as qk
from tests import state_ref as sr
from tests.test_gpu_state_scan import BF, DEV, F32, Case, close

pytestmark = pytest.mark.gpu

DIVIDED = {
    "keys of 128": dict(lens=[1501], H=2, Hk=1, Dk=128, Dv=64, shift=4.0),
    "values of 128": dict(lens=[1501] * 2, H=2, Hk=2, Dk=64, Dv=128, state=True, shift=4.0),
    "both of 128": dict(lens=[1100], H=1, Hk=1, Dk=128, Dv=128, state=True, shift=4.0),
    "odd widths": dict(lens=[1301], H=3, Hk=1, Dk=96, Dv=80, state=True, strided=True, shift=4.0),
    "packed": dict(lens=[900, 0, 1, 1210, 64, 65], H=3, Hk=1, Dk=72, Dv=40, packed=True, state=True, shift=4.0),
    "log decays": dict(lens=[1200], H=2, Hk=2, Dk=64, Dv=64, form="log", shift=0.0),
}


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", DIVIDED)
def test_divided_sequences(name, dtype):
    print(f"case divided scan: {name} {dtype}", flush=True)
    c = Case(dtype=dtype, **DIVIDED[name])
    assert gs.state_scan_forward_workspace_bytes(*c.args(), c.off) > 0  # it is divided
    out, fin = gs.state_scan_forward(*c.args(), **c.kw(), final_state=True)
    g = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw(),
                               d_final_state=None if c.dsT is None else c.dsT.to(DEV))
    torch.cuda.synchronize()
    fwd, bwd = [c.ref(i) for i in range(len(c.lens))], [c.ref(i, grad=True) for i in range(len(c.lens))]
    close(c.flat(out), np.concatenate([r[0] for r in fwd]), dtype, "out")
    close(fin, np.stack([r[1] for r in fwd]), F32, "final state")
    for j, what in enumerate(("dq", "dk", "dv", "dgate")):
        close(c.flat(g[j]), np.concatenate([r[j] for r in bwd]), dtype, what)
    if c.s0 is not None:
        close(g[4], np.stack([r[4] for r in bwd]), F32, "d_initial_state")


MANY = {
    "shared heads": dict(lens=[(29 * i) % 83 for i in range(130)], H=8, Hk=4, Dk=40, Dv=24),
    "own heads": dict(lens=[(17 * i) % 140 for i in range(60)], H=5, Hk=5, Dk=128, Dv=64, state=True),
    "full widths": dict(lens=[70, 0, 3, 190, 65] * 8, H=6, Hk=6, Dk=128, Dv=128),
}


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", MANY)
def test_more_chunks_than_workgroups(name, dtype):
    print(f"case many chunks: {name} {dtype}", flush=True)
    c = Case(dtype=dtype, packed=True, **MANY[name])
    chunk = 64 if dtype == BF else 32
    assert sum(-(-n // chunk) for n in c.lens) * c.host["q"].shape[1] > 256
    g = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw(),
                               d_final_state=None if c.dsT is None else c.dsT.to(DEV))
    torch.cuda.synchronize()
    refs = [c.ref(i, grad=True) for i in range(len(c.lens))]
    for j, what in enumerate(("dq", "dk", "dv", "dgate")):
        close(g[j], np.concatenate([r[j] for r in refs]), dtype, what)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("where", ["q", "k", "v", "do", "a"])
def test_one_bad_element_among_many_chunks(where, dtype):
    """An infinity (a NaN gate) in one sequence and head: everything of the other
    sequences, and of the heads that do not share its keys, has the same bits; so
    has the gradient of the tensor itself, which its values do not enter (d_out's
    and the gate's enter all)."""
    c = Case(lens=[100, 64, 130, 7] * 30, H=8, Hk=4, Dk=64, Dv=40, dtype=dtype, packed=True)
    ops = [*c.args(), c.dev["do"]]
    clean = gs.state_scan_backward(*ops, **c.kw())
    i = ["q", "k", "v", "a", "do"].index(where)
    bad = [x.clone() for x in ops]
    t = int(c.spans[46][0]) + 70  # sequence 46 has 130 tokens: its second or third chunk
    head = 1 if where in "qk" else 3  # value heads 2 and 3 share key head 1
    if where == "a":
        bad[i][t, head] = float("nan")
    else:
        bad[i][t, head, 5] = float("inf")
    got = gs.state_scan_backward(*bad, **c.kw())
    torch.cuda.synchronize()
    b, e = (int(x) for x in c.spans[46])
    for x, y, name in zip(got, clean, ("dq", "dk", "dv", "dgate")):
        if name == "d" + where:
            assert torch.equal(x, y), name
            continue
        assert not bool(torch.isfinite(x[b:e]).all()), name
        assert torch.equal(x[:b], y[:b]) and torch.equal(x[e:], y[e:]), name
        others = [0, 2, 3] if x.shape[1] == 4 else [0, 1, 4, 5, 6, 7]
        assert torch.equal(x[b:e, others], y[b:e, others]), name


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_gradients_of_more_tokens_than_workgroups(layout):
    p = dict(n=1500, Hq=30, Hk=10, D=256, rot=64)
    m = qk.make(dtype=F32, **p)
    dy = [x.to(DEV) for x in m["dy"]]
    g = gs.qk_norm_rope_backward(*qk.call_args(m), *dy, eps=1e-5, layout=layout)
    for i in range(2):
        x, w = m["host"][i].double().numpy(), m["w"][i].double().numpy()
        dx, dw = sr.norm_rope_grad(x, w, m["pos"].numpy(), m["freq"].numpy(), m["dy"][i].double().numpy(), 1e-5,
                                   layout, 1.0)
        qk.close(g[i], dx, qk.TOL[F32], f"dx{i}")
        qk.close(g[2 + i], dw, 32 * 2.0 ** -24, f"dw{i}")
