"""The matrix-state scan (gscan_state_scan_*, through the package) against the
recurrence in 64 bits, token by token.

Tolerances, relative 2-norms.  float32: a result is a chain of contractions of
at most 128 + 64 terms per chunk, exponentials of decays that matter (down to
e^-16: error 16 * 2^-24) and a state update per chunk whose errors decay with
it: 32 roundings' worth, 32 * 2^-24 = 1.9e-6.  bfloat16 tensors: the inputs are
exact on both sides; one rounding of the result and one of an operand inside
(decayed scores or state), each at most 2^-8 of its term with signs that do not
conspire: 2 * 2^-8.  float32 states from bfloat16 operands keep the float32
bound.  No element may be off by more than 16 times the bound of the largest."""
import numpy as np
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests import state_ref as sr

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TOL = {torch.float32: 32 * 2.0 ** -24, torch.bfloat16: 2 * 2.0 ** -8}
BF, F32 = torch.bfloat16, torch.float32


def close(got, ref, dtype, what):
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, what
    assert np.all(np.isfinite(got)), what
    if ref.size == 0:
        return
    err, n = np.linalg.norm(got - ref), np.linalg.norm(ref)
    worst = np.max(np.abs(got - ref))
    print(f"  {what}: rel {err / max(n, 1e-300):.2e} max {worst / max(np.max(np.abs(ref)), 1e-300):.2e}",
          flush=True)
    assert err <= TOL[dtype] * n, what
    assert worst <= 16 * TOL[dtype] * np.max(np.abs(ref)), what


class Case:
    def __init__(self, lens, H=4, Hk=4, Dk=32, Dv=32, dtype=F32, packed=False, state=False,
                 form="sigmoid", gate_dtype=None, shift=1.5, seed=1, strided=False):
        r = np.random.default_rng(seed)
        self.lens, self.dtype, self.packed, self.form, self.shift = lens, dtype, packed, form, shift
        self.scale = Dk ** -0.5
        n, N = sum(lens), len(lens)
        gd = gate_dtype or dtype

        def tensor(dt, *shape):
            x = torch.from_numpy(r.standard_normal(shape).astype(np.float32))
            return x.to(dt)

        a = tensor(F32, n, H) + torch.linspace(-1.0, 4.0, H)
        if form == "log":
            a = -torch.nn.functional.softplus(-a)
        self.host = {"q": tensor(dtype, n, Hk, Dk), "k": tensor(dtype, n, Hk, Dk),
                     "v": tensor(dtype, n, H, Dv), "a": a.to(gd), "do": tensor(dtype, n, H, Dv)}
        self.s0 = tensor(F32, N, H, Dk, Dv) if state else None
        self.dsT = tensor(F32, N, H, Dk, Dv) if state else None
        self.dev = {}
        for name, x in self.host.items():
            y = x if packed else x.reshape(N, lens[0], *x.shape[1:])
            if strided and x.dim() == 3:  # a slice of a wider projection, behind 16 other columns
                wide = torch.zeros(*y.shape[:-2], y.shape[-2] * y.shape[-1] + 48, dtype=y.dtype, device=DEV)
                part = wide[..., 16:16 + y.shape[-2] * y.shape[-1]].unflatten(-1, y.shape[-2:])
                part.copy_(y)
                self.dev[name] = part
            else:
                self.dev[name] = y.to(DEV)
        off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.off = torch.from_numpy(off).to(DEV) if packed else None
        self.spans = list(zip(off[:-1], off[1:]))

    def kw(self):
        return dict(scale=self.scale, gate_form=self.form, gate_shift=self.shift,
                    seq_offsets=self.off,
                    initial_state=None if self.s0 is None else self.s0.to(DEV))

    def args(self):
        return tuple(self.dev[n] for n in ("q", "k", "v", "a"))

    def ref(self, i, grad=False):
        b, e = self.spans[i]
        x = [self.host[n][b:e].double().numpy() for n in ("q", "k", "v", "a")]
        s0 = None if self.s0 is None else self.s0[i].double().numpy()
        if not grad:
            o, S = sr.scan(*x, self.scale, self.form, self.shift, s0)
            return o, S[-1]
        dsT = None if self.dsT is None else self.dsT[i].double().numpy()
        return sr.scan_grad(*x, self.host["do"][b:e].double().numpy(), self.scale, self.form, self.shift,
                            s0, dsT)

    def flat(self, x):
        return x if self.packed else x.flatten(0, 1)


FORWARD = {
    "one token": dict(lens=[1]),
    "one token, bf16": dict(lens=[1], dtype=BF, Dk=64, Dv=64),
    "smallest widths": dict(lens=[70], H=1, Hk=1, Dk=8, Dv=8),
    "smallest widths, bf16": dict(lens=[70], H=1, Hk=1, Dk=8, Dv=8, dtype=BF),
    "chunk edges": dict(lens=[31, 32, 33, 63, 64, 65, 127, 128, 129], packed=True, H=2, Hk=2),
    "chunk edges, bf16": dict(lens=[31, 32, 33, 63, 64, 65, 127, 128, 129], packed=True, H=2, Hk=2, dtype=BF),
    "empty sequences": dict(lens=[0, 5, 0, 0, 70, 0], packed=True, state=True),
    "empty sequences, bf16": dict(lens=[0, 5, 0, 0, 70, 0], packed=True, state=True, dtype=BF),
    "many sequences": dict(lens=[(7 * i) % 13 for i in range(150)], packed=True, state=True, H=2, Hk=1),
    "batch": dict(lens=[200] * 3, H=6, Hk=2, Dk=96, Dv=40, state=True),
    "batch, bf16": dict(lens=[200] * 3, H=6, Hk=2, Dk=96, Dv=40, state=True, dtype=BF),
    "widest": dict(lens=[150] * 2, H=2, Hk=2, Dk=128, Dv=128, state=True),
    "widest, bf16": dict(lens=[150] * 2, H=2, Hk=2, Dk=128, Dv=128, state=True, dtype=BF),
    "odd widths, bf16": dict(lens=[90] * 2, H=3, Hk=1, Dk=72, Dv=88, dtype=BF, strided=True),
    "odd widths, strided": dict(lens=[90] * 2, H=3, Hk=1, Dk=72, Dv=88, strided=True, state=True),
    "packed, strided, bf16": dict(lens=[90, 3, 41], H=4, Hk=2, Dk=64, Dv=128, dtype=BF, strided=True,
                                  packed=True),
    "log decays": dict(lens=[140], form="log", shift=0.0),
    "log decays, bf16": dict(lens=[140], form="log", shift=0.0, dtype=BF, Dk=64, Dv=64),
    "float32 gates beside bf16": dict(lens=[140], dtype=BF, gate_dtype=F32, Dk=64, Dv=64),
    "bf16 gates beside float32": dict(lens=[140], gate_dtype=BF),
    "long": dict(lens=[5000], H=2, Hk=1, Dk=16, Dv=16, shift=6.0),
    "long, bf16": dict(lens=[5003, 17], packed=True, H=2, Hk=1, Dk=32, Dv=16, dtype=BF, shift=6.0,
                       state=True),
    "saturated gates": dict(lens=[300], shift=30.0, H=2, Hk=2),
    "nearly closed gates": dict(lens=[300], shift=-30.0, H=2, Hk=2),
}


@pytest.mark.parametrize("name", FORWARD)
def test_forward(name):
    print(f"case state scan forward: {name}", flush=True)
    c = Case(**FORWARD[name])
    out, fin = gs.state_scan_forward(*c.args(), **c.kw(), final_state=True)
    torch.cuda.synchronize()
    assert out.dtype == c.dtype and fin.dtype == F32
    refs = [c.ref(i) for i in range(len(c.lens))]
    close(c.flat(out), np.concatenate([r[0] for r in refs]), c.dtype, "out")
    close(fin, np.stack([r[1] for r in refs]), F32, "final state")


GRAD = {
    "one token": dict(lens=[1], state=True),
    "one token, bf16": dict(lens=[1], dtype=BF, Dk=64, Dv=64),
    "smallest widths": dict(lens=[70], H=1, Hk=1, Dk=8, Dv=8),
    "smallest widths, bf16": dict(lens=[70], H=1, Hk=1, Dk=8, Dv=8, dtype=BF),
    "chunk edges": dict(lens=[31, 32, 33, 63, 64, 65, 129], packed=True, H=2, Hk=2),
    "chunk edges, bf16": dict(lens=[31, 32, 33, 63, 64, 65, 129], packed=True, H=2, Hk=2, dtype=BF),
    "empty sequences": dict(lens=[0, 5, 0, 70, 0], packed=True, state=True),
    "empty sequences, bf16": dict(lens=[0, 5, 0, 70, 0], packed=True, state=True, dtype=BF),
    "many sequences": dict(lens=[(7 * i) % 13 for i in range(90)], packed=True, state=True, H=2, Hk=1),
    "shared heads": dict(lens=[130] * 2, H=6, Hk=2, Dk=96, Dv=40, state=True),
    "shared heads, bf16": dict(lens=[130] * 2, H=6, Hk=2, Dk=96, Dv=40, state=True, dtype=BF),
    "one key head": dict(lens=[100], H=5, Hk=1, Dk=48, Dv=16),
    "widest": dict(lens=[140], H=2, Hk=2, Dk=128, Dv=128, state=True),
    "widest, bf16": dict(lens=[140], H=2, Hk=2, Dk=128, Dv=128, state=True, dtype=BF),
    "wide values": dict(lens=[90], H=2, Hk=1, Dk=40, Dv=128),
    "wide values, bf16": dict(lens=[90], H=2, Hk=1, Dk=40, Dv=128, dtype=BF),
    "wide keys, bf16": dict(lens=[90], H=2, Hk=1, Dk=128, Dv=40, dtype=BF, strided=True),
    "strided": dict(lens=[90] * 2, H=3, Hk=1, Dk=72, Dv=88, strided=True, state=True),
    "log decays": dict(lens=[140], form="log", shift=0.0, state=True),
    "log decays, bf16": dict(lens=[140], form="log", shift=0.0, dtype=BF, Dk=64, Dv=64),
    "bf16 gates beside float32": dict(lens=[140], gate_dtype=BF),
    "long": dict(lens=[1500], H=2, Hk=1, Dk=16, Dv=16, shift=6.0, state=True),
    "long, bf16": dict(lens=[1503, 17], packed=True, H=2, Hk=1, Dk=32, Dv=16, dtype=BF, shift=6.0,
                       state=True),
    "saturated gates": dict(lens=[200], shift=30.0, H=2, Hk=2, gate_dtype=F32),
    "nearly closed gates": dict(lens=[200], shift=-30.0, H=2, Hk=2),
}


@pytest.mark.parametrize("name", GRAD)
def test_backward(name):
    print(f"case state scan backward: {name}", flush=True)
    c = Case(**GRAD[name])
    g = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw(),
                               d_final_state=None if c.dsT is None else c.dsT.to(DEV))
    torch.cuda.synchronize()
    refs = [c.ref(i, grad=True) for i in range(len(c.lens))]
    for j, what in enumerate(("dq", "dk", "dv", "dgate")):
        dt = c.host["a"].dtype if what == "dgate" else c.dtype
        assert g[j].dtype == dt
        close(c.flat(g[j]), np.concatenate([r[j] for r in refs]), dt, what)
    if c.s0 is None:
        assert g[4] is None
    else:
        close(g[4], np.stack([r[4] for r in refs]), F32, "d_initial_state")


def test_gradient_against_differences_of_the_kernel():
    """d loss along a random direction by differences of the forward kernel in
    float32: the loss of ~1e3 terms carries 2^-24 relative noise, the step 2^-6
    a third-order error; agreement to 1e-3 of the derivative's scale."""
    c = Case([70], H=2, Hk=1, Dk=16, Dv=24, state=True, seed=11)
    kw = c.kw()
    s0 = kw.pop("initial_state")
    r = np.random.default_rng(5)
    x = list(c.args()) + [s0]
    d = [torch.from_numpy(r.standard_normal(t.shape).astype(np.float32)).to(DEV) for t in x]

    def loss(step):
        y = [t + step * e for t, e in zip(x, d)]
        o, S = gs.state_scan_forward(*y[:4], **kw, initial_state=y[4], final_state=True)
        return float((o.double() * c.dev["do"].double()).sum() + (S.double() * c.dsT.to(DEV).double()).sum())

    g = gs.state_scan_backward(*c.args(), c.dev["do"], **kw, initial_state=s0, d_final_state=c.dsT.to(DEV))
    want = sum(float((a.double() * b.double()).sum()) for a, b in zip(g, d))
    size = sum(float((a.double() ** 2).sum()) for a in g) ** 0.5
    h = 2.0 ** -6
    # Richardson: removes the third-order error of the central difference
    c1, c2 = (loss(h) - loss(-h)) / (2 * h), (loss(h / 2) - loss(-h / 2)) / h
    assert abs((4 * c2 - c1) / 3 - want) <= 1e-3 * size


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_closed_gate_forgets(dtype):
    """A log gate of minus infinity: what was before does not reach the state,
    the outputs or the gradients, and a decay behind it stays exact."""
    c = Case([200], H=2, Hk=2, dtype=dtype, form="log", shift=0.0, state=True, gate_dtype=F32)
    for t in (0, 50, 51, 64, 130):
        c.host["a"][t] = -np.inf
        c.dev["a"][0, t] = -np.inf
    out, fin = gs.state_scan_forward(*c.args(), **c.kw(), final_state=True)
    o, S = c.ref(0)
    close(out[0], o, dtype, "out")
    close(fin[0], S, F32, "final state")
    g = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw(), d_final_state=c.dsT.to(DEV))
    r = c.ref(0, grad=True)
    for j, what in enumerate(("dq", "dk", "dv")):
        close(g[j][0], r[j], dtype, what)
    assert torch.all(g[4] == 0)  # the first token's gate is closed
    assert torch.all(g[3][0, [0, 50, 51, 64, 130]] == 0)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_value_reaches_no_earlier_token(dtype, value):
    c = Case([150], H=2, Hk=2, Dk=32, Dv=40, dtype=dtype)
    clean = gs.state_scan_forward(*c.args(), **c.kw())
    for name in ("v", "k", "q"):
        x = {n: t.clone() for n, t in c.dev.items()}
        x[name][0, 70, 1, 3] = value
        out = gs.state_scan_forward(x["q"], x["k"], x["v"], x["a"], **c.kw())
        assert torch.equal(out[:, :70], clean[:, :70]), name
        assert torch.equal(out[:, :, 0], clean[:, :, 0]), name
        assert not torch.isfinite(out[0, 70, 1]).all(), name
        if name == "q":
            assert torch.equal(out[:, 71:], clean[:, 71:])
        if name == "v":  # only that column of the state
            keep = [i for i in range(40) if i != 3]
            assert torch.isfinite(out[0, :, 1, keep]).all()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_nonfinite_gradient_reaches_no_later_token(dtype):
    """d_out of token t enters the gradients of tokens up to t only; a NaN in q
    likewise through dk."""
    c = Case([150], H=2, Hk=2, Dk=32, Dv=40, dtype=dtype)
    clean = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw())
    do = c.dev["do"].clone()
    do[0, 70, 1, 3] = float("nan")
    g = gs.state_scan_backward(*c.args(), do, **c.kw())
    for j in (1, 2):
        assert torch.equal(g[j][:, 71:], clean[j][:, 71:])
        assert torch.equal(g[j][:, :, 0], clean[j][:, :, 0])
    assert torch.equal(g[0][:, 71:], clean[0][:, 71:])
    assert torch.equal(g[0][:, :70], clean[0][:, :70])
    k = c.dev["k"].clone()
    k[0, 70, 1, 3] = float("inf")
    g = gs.state_scan_backward(c.dev["q"], k, c.dev["v"], c.dev["a"], c.dev["do"], **c.kw())
    assert torch.equal(g[0][:, :70], clean[0][:, :70])  # dq of tokens before it
    assert torch.isfinite(g[1]).all()                   # dk does not read k


def test_no_tokens():
    c = Case([0, 0], packed=True, state=True)
    out, fin = gs.state_scan_forward(*c.args(), **c.kw(), final_state=True)
    assert out.shape == (0, 4, 32) and torch.equal(fin, c.s0.to(DEV))
    g = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw(), d_final_state=c.dsT.to(DEV))
    assert torch.equal(g[4], c.dsT.to(DEV)) and g[0].numel() == 0
    q = torch.empty(2, 0, 4, 32, device=DEV)
    a = torch.empty(2, 0, 4, device=DEV)
    out, fin = gs.state_scan_forward(q, q, q, a, final_state=True)
    assert out.shape == q.shape and torch.all(fin == 0)


def test_wrong_offsets_stay_in_range():
    """Offsets that decrease or pass the end: nothing is specified of the result
    but that the call returns and touches only its own memory."""
    c = Case([40, 30, 50], packed=True, H=2, Hk=2)
    guard = torch.full((120 * 2 * 32 + 4096,), 7.0, device=DEV)
    out = guard[2048:2048 + 120 * 2 * 32].view(120, 2, 32)
    for off in ([0, 500, 20, 120], [-5, 40, 1 << 30, 3], [120, 120, 120, 120], [7, 3, 2, 1]):
        off = torch.tensor(off, dtype=torch.int32, device=DEV)
        gs.state_scan_forward(*c.args(), seq_offsets=off, out=out, final_state=True)
        gs.state_scan_backward(*c.args(), c.dev["do"], seq_offsets=off)
        torch.cuda.synchronize()
        assert torch.all(guard[:2048] == 7) and torch.all(guard[-2048:] == 7)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_parts_of_a_sequence_continue_each_other(dtype):
    c = Case([300], H=2, Hk=1, Dk=64, Dv=64, dtype=dtype)
    kw = c.kw()
    kw.pop("initial_state")
    whole, fin = gs.state_scan_forward(*c.args(), **kw, final_state=True)
    s = torch.zeros(1, 2, 64, 64, device=DEV)
    parts = []
    for b, e in ((0, 100), (100, 101), (101, 300)):
        o, s2 = gs.state_scan_forward(*(x[:, b:e] for x in c.args()), **kw, initial_state=s,
                                      final_state=s)  # in place
        assert s2 is s
        parts.append(o)
    close(torch.cat(parts, 1), whole.double().cpu().numpy(), dtype, "out")
    close(s, fin.double().cpu().numpy(), F32, "final state")


def test_far_rows_of_a_large_tensor():
    """Rows that begin past 2^32 elements: a batch stride that large."""
    wide = torch.zeros(2 ** 32 + 70 * 64, dtype=BF, device=DEV)
    q = wide.as_strided((2, 70, 1, 64), (2 ** 32, 64, 64, 1))
    small = torch.randn(2, 70, 1, 64, device=DEV).to(BF)
    q.copy_(small)
    a = torch.randn(2, 70, 1, device=DEV)
    got = gs.state_scan_forward(q, q, q, a, final_state=True)
    ref = gs.state_scan_forward(small, small, small, a, final_state=True)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    got = gs.state_scan_backward(q, q, q, a, q)
    ref = gs.state_scan_backward(small, small, small, a, small)
    for x, y in zip(got[:4], ref[:4]):
        assert torch.equal(x, y)


def test_reproducible_and_other_stream():
    c = Case([700, 90], packed=True, H=4, Hk=2, Dk=64, Dv=64, dtype=BF, state=True)
    kw, dsT = c.kw(), c.dsT.to(DEV)
    torch.cuda.synchronize()
    a = gs.state_scan_forward(*c.args(), **kw, final_state=True)
    ga = gs.state_scan_backward(*c.args(), c.dev["do"], **kw, d_final_state=dsT)
    s = torch.cuda.Stream()
    b = gs.state_scan_forward(*c.args(), **kw, final_state=True, stream=s)
    gb = gs.state_scan_backward(*c.args(), c.dev["do"], **kw, d_final_state=dsT, stream=s)
    torch.cuda.synchronize()
    for x, y in zip(a + ga, b + gb):
        assert torch.equal(x, y)


def test_caller_workspace_and_outputs():
    c = Case([200], H=2, Hk=2)
    n = gs.state_scan_backward_workspace_bytes(*c.args())
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    g = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw(), workspace=ws)
    h = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw())
    for x, y in zip(g[:4], h[:4]):
        assert torch.equal(x, y)
    out = torch.empty_like(c.dev["v"])
    assert gs.state_scan_forward(*c.args(), **c.kw(), out=out) is out
    with pytest.raises(ValueError):
        gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw(), workspace=ws[:n - 1])


# ------------------------------------------------------------------- step

STEP = {
    "one": dict(N=1, pool=1, H=4, Hk=4, Dk=64, Dv=64, dtype=BF),
    "one, f32": dict(N=1, pool=3, H=1, Hk=1, Dk=8, Dv=8, dtype=F32),
    "odd": dict(N=7, pool=11, H=6, Hk=2, Dk=72, Dv=40, dtype=F32),
    "odd, bf16": dict(N=7, pool=11, H=6, Hk=2, Dk=72, Dv=88, dtype=BF),
    "widest": dict(N=5, pool=5, H=2, Hk=1, Dk=128, Dv=128, dtype=BF),
    "narrow values": dict(N=3, pool=4, H=2, Hk=1, Dk=128, Dv=8, dtype=F32),
}


@pytest.mark.parametrize("form", ["sigmoid", "log"])
@pytest.mark.parametrize("name", STEP)
def test_step(name, form):
    print(f"case state scan step: {name} {form}", flush=True)
    p = dict(STEP[name])
    dtype, N, pool, H, Hk, Dk, Dv = (p[x] for x in ("dtype", "N", "pool", "H", "Hk", "Dk", "Dv"))
    r = torch.Generator().manual_seed(3)
    q, k = torch.randn(N, Hk, Dk, generator=r).to(dtype), torch.randn(N, Hk, Dk, generator=r).to(dtype)
    v, a = torch.randn(N, H, Dv, generator=r).to(dtype), torch.randn(N, H, generator=r)
    a = (a if form == "sigmoid" else -a.abs()).to(dtype)
    state = torch.randn(pool, H, Dk, Dv, generator=r)
    slots = torch.randperm(pool, generator=r)[:N].to(torch.int32)
    if N > 2:
        slots[1], slots[2] = -1, pool  # padding
    dev = state.to(DEV)
    out = gs.state_scan_step(q.to(DEV), k.to(DEV), v.to(DEV), a.to(DEV), dev, slots=slots.to(DEV),
                             scale=0.3, gate_form=form, gate_shift=0.25)
    ref, want = state.double().numpy().copy(), np.zeros((N, H, Dv))
    for n, s in enumerate(slots.tolist()):
        if 0 <= s < pool:
            x = [t[n:n + 1].double().numpy() for t in (q, k, v, a)]
            o, S = sr.scan(*x, 0.3, form, 0.25, ref[s])
            want[n], ref[s] = o[0], S[-1]
    close(out, want, dtype, "out")
    close(dev, ref, F32, "pool")
    used = {s for s in slots.tolist() if 0 <= s < pool}
    for s in range(pool):
        if s not in used:
            assert torch.equal(dev[s].cpu(), state[s])


def test_steps_continue_a_scan():
    """A prompt through the scan, then tokens one by one, against one scan."""
    c = Case([90], H=4, Hk=2, Dk=64, Dv=64, dtype=BF)
    kw = dict(scale=c.scale, gate_shift=c.shift)
    whole, fin = gs.state_scan_forward(*c.args(), **kw, final_state=True)
    _, state = gs.state_scan_forward(*(x[:, :70] for x in c.args()), **kw, final_state=True)
    outs = [gs.state_scan_step(*(x[:, t] for x in c.args()), state, **kw) for t in range(70, 90)]
    close(torch.stack(outs, 1), whole[:, 70:].double().cpu().numpy(), BF, "out")
    close(state, fin.double().cpu().numpy(), F32, "state")


def test_step_without_requests_and_other_stream():
    state = torch.randn(3, 2, 16, 16, device=DEV)
    keep = state.clone()
    e = torch.empty(0, 2, 16, device=DEV)
    assert gs.state_scan_step(e, e, e, torch.empty(0, 2, device=DEV), state).shape == (0, 2, 16)
    assert torch.equal(state, keep)
    x, a = torch.randn(3, 2, 16, device=DEV), torch.randn(3, 2, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o1 = gs.state_scan_step(x, x, x, a, state, stream=s)
    o2 = gs.state_scan_step(x, x, x, a, keep)
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(state, keep)


# --------------------------------------------------------------- autograd

@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_autograd(dtype):
    c = Case([130, 0, 20], packed=True, H=4, Hk=2, dtype=dtype, state=True)
    leaves = [x.clone().requires_grad_() for x in c.args()]
    s0 = c.s0.to(DEV).requires_grad_()
    out, fin = gs.state_scan(*leaves, initial_state=s0, scale=c.scale, gate_shift=c.shift,
                             seq_offsets=c.off)
    ((out.float() * c.dev["do"].float()).sum() + (fin * c.dsT.to(DEV)).sum()).backward()
    g = gs.state_scan_backward(*c.args(), c.dev["do"], **c.kw(), d_final_state=c.dsT.to(DEV))
    for x, y in zip(leaves + [s0], g):
        assert torch.equal(x.grad, y)
    # expanded upstream gradient, no gradient of the final state, shared k broadcast over heads
    one = c.dev["k"][:, :1].clone().requires_grad_()
    out, _ = gs.state_scan(c.dev["q"], one.expand(-1, 2, -1), c.dev["v"], c.dev["a"], scale=c.scale,
                           gate_shift=c.shift, seq_offsets=c.off)
    out.sum().backward()
    kw = c.kw()
    kw["initial_state"] = None
    g = gs.state_scan_backward(c.dev["q"], one.detach().expand(-1, 2, -1), c.dev["v"], c.dev["a"],
                               torch.ones_like(c.dev["v"]), **kw)
    assert torch.equal(one.grad, g[1].sum(1, keepdim=True))
    # only the final state is used
    v = c.dev["v"].clone().requires_grad_()
    _, fin = gs.state_scan(c.dev["q"], c.dev["k"], v, c.dev["a"], seq_offsets=c.off)
    fin.sum().backward()
    assert torch.isfinite(v.grad).all() and v.grad.abs().sum() > 0


def test_graph_replays_match_eager():
    """Forward, backward and a step captured with caller workspaces, replayed on
    new inputs with eager work in between, bitwise against eager calls."""
    c = Case([500, 77], packed=True, H=4, Hk=2, Dk=64, Dv=64, dtype=BF, state=True)
    kw, dsT = c.kw(), c.dsT.to(DEV)
    nb = gs.state_scan_backward_workspace_bytes(*c.args(), seq_offsets=c.off)
    nf = gs.state_scan_forward_workspace_bytes(*c.args(), seq_offsets=c.off)
    wb = torch.empty(nb, dtype=torch.uint8, device=DEV)
    wf = torch.empty(nf, dtype=torch.uint8, device=DEV) if nf else None
    pool = torch.randn(577, 4, 64, 64, device=DEV)
    keep = pool.clone()

    def work():
        a = gs.state_scan_forward(*c.args(), **kw, final_state=True, workspace=wf)
        b = gs.state_scan_backward(*c.args(), c.dev["do"], **kw, d_final_state=dsT, workspace=wb)
        return a + b + (gs.state_scan_step(*c.args(), pool),)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = work()
    for rep in range(4):
        for n in ("q", "k", "v", "do"):
            c.dev[n].copy_(torch.randn(c.dev[n].shape, device=DEV))
        pool.copy_(keep)
        torch.randn(1 << 18, device=DEV).mul_(2)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs] + [pool.clone()]
        pool.copy_(keep)
        ref = list(work()) + [pool]
        torch.cuda.synchronize()
        for x, y in zip(got, ref):
            assert torch.equal(x, y), f"replay {rep}"
