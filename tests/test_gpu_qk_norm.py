"""The query/key norm with rotation (gscan_qk_norm_rope_*, through the package)
against the formulas in 64 bits.

Tolerances, relative 2-norms.  float32: the angle, reduced in fp64, is rounded
to float32 within [-pi, pi] (absolute pi * 2^-24), sine and cosine are good to
about two units, the norm adds the roundings of a sum of up to 256 squares (a
tree: 8 levels), a square root, a division and three products: 16 * 2^-24.
Weight gradients sum thousands of terms in float32 per lane and fp64 across
workgroups: 32 * 2^-24 of the root-sum-square they come from, which the test
takes as the result's norm (terms are independent).  bfloat16: that and one
rounding of the result, 2^-8."""
import numpy as np
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests import state_ref as sr

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 16 * 2.0 ** -24, BF: 2.0 ** -8 + 16 * 2.0 ** -24}


def close(got, ref, tol, what):
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    if ref.size == 0:
        return
    n = np.linalg.norm(ref)
    err = np.linalg.norm(got - ref)
    print(f"  {what}: rel {err / max(n, 1e-300):.2e}", flush=True)
    assert err <= tol * n, what
    assert np.max(np.abs(got - ref)) <= 8 * tol * np.max(np.abs(ref)), what


CASES = {
    "one token": dict(n=1, Hq=4, Hk=1, D=64, rot=64),
    "one token, far": dict(n=1, Hq=16, Hk=4, D=128, rot=128, start=2 ** 30 + 12345),
    "past 2^31": dict(n=3, Hq=2, Hk=1, D=32, rot=32, start=2 ** 33 + 1),
    "smallest": dict(n=5, Hq=1, Hk=1, D=8, rot=8),
    "no rotation": dict(n=9, Hq=2, Hk=2, D=48, rot=0),
    "part of the head": dict(n=70, Hq=3, Hk=2, D=80, rot=48),
    "halves of twelve": dict(n=33, Hq=2, Hk=1, D=40, rot=24),
    "halves of twenty": dict(n=33, Hq=2, Hk=1, D=256, rot=40),
    "widest": dict(n=19, Hq=5, Hk=3, D=256, rot=256),
    "many heads": dict(n=6, Hq=70, Hk=9, D=64, rot=32),
    "no keys": dict(n=12, Hq=4, Hk=0, D=64, rot=64),
    "many tokens": dict(n=3001, Hq=2, Hk=1, D=64, rot=64),
    "magnitude": dict(n=20, Hq=2, Hk=1, D=64, rot=32, magnitude=1.25),
}


def make(n, Hq, Hk, D, rot, dtype, start=0, magnitude=1.0, pos64=True, seed=2):
    r = torch.Generator().manual_seed(seed)
    both = torch.randn(n, (Hq + Hk) * D + 16, generator=r).to(dtype)
    dev = both.to(DEV)

    def split(x):  # slices of one projection
        k = x[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
        return x[:, :Hq * D].unflatten(1, (Hq, D)), k

    pos = start + torch.arange(n) * 3
    freq = (10000.0 ** (-torch.arange(0, rot, 2) / rot)).float() if rot else None
    return dict(host=split(both), dev=split(dev), pos=pos, freq=freq, magnitude=magnitude,
                w=[1 + 0.3 * torch.randn(D, generator=r) for _ in range(2)],
                dy=[None if x is None else torch.randn(x.shape, generator=r).to(dtype)
                    for x in split(both)], pos64=pos64)


def call_args(m):
    freq = None if m["freq"] is None else m["freq"].to(DEV)
    pos = m["pos"].to(DEV) if m["pos64"] else m["pos"].to(torch.int32).to(DEV)
    wk = None if m["dev"][1] is None else m["w"][1].to(DEV)
    return (*m["dev"], m["w"][0].to(DEV), wk, pos, freq)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("name", CASES)
def test_forward_and_backward(name, layout, dtype):
    print(f"case norm and rotation: {name} {layout} {dtype}", flush=True)
    p = dict(CASES[name])
    m = make(dtype=dtype, pos64=p.get("start", 0) > 0 or layout == "half", **p)
    args = call_args(m)
    kw = dict(eps=1e-5, layout=layout, magnitude=m["magnitude"])
    out = gs.qk_norm_rope_forward(*args, **kw)
    dy = [None if x is None else x.to(DEV) for x in m["dy"]]
    g = gs.qk_norm_rope_backward(*args, *dy, **kw)
    torch.cuda.synchronize()
    freq = np.zeros(0) if m["freq"] is None else m["freq"].numpy()
    for i in range(2):
        if m["host"][i] is None:
            assert out[i] is None and g[i] is None and g[2 + i] is None
            continue
        x, w = m["host"][i].double().numpy(), m["w"][i].double().numpy()
        close(out[i], sr.norm_rope(x, w, m["pos"].numpy(), freq, 1e-5, layout, m["magnitude"]),
              TOL[dtype], f"y{i}")
        dx, dw = sr.norm_rope_grad(x, w, m["pos"].numpy(), freq, m["dy"][i].double().numpy(), 1e-5, layout,
                                   m["magnitude"])
        close(g[i], dx, TOL[dtype], f"dx{i}")
        close(g[2 + i], dw, 32 * 2.0 ** -24, f"dw{i}")


def test_rows_of_zeros_and_no_weights():
    x = torch.zeros(4, 2, 64, device=DEV)
    x[1] = 2.0
    pos, freq = torch.arange(4, device=DEV), torch.ones(16, device=DEV)
    q, k = gs.qk_norm_rope_forward(x, x, None, None, pos, freq, eps=1e-6)
    assert torch.all(q[0] == 0) and torch.equal(q, k)
    assert torch.allclose(q[1, :, 32:], torch.ones(2, 32, device=DEV), rtol=1e-6)
    dq, dk, a, b = gs.qk_norm_rope_backward(x, x, None, None, pos, freq, x, x)
    assert a is None and b is None and torch.isfinite(dq).all()


def test_nonfinite_row_stays_alone():
    x = torch.randn(9, 3, 48, device=DEV)
    pos, freq = torch.arange(9, device=DEV), torch.ones(24, device=DEV)
    clean = gs.qk_norm_rope_forward(x, None, None, None, pos, freq)[0]
    x[4, 1, 7] = float("nan")
    out = gs.qk_norm_rope_forward(x, None, None, None, pos, freq)[0]
    assert torch.isnan(out[4, 1]).all()
    out[4, 1] = clean[4, 1]
    assert torch.equal(out, clean)


def test_no_tokens():
    x = torch.empty(0, 2, 64, device=DEV)
    pos, freq, w = torch.empty(0, dtype=torch.int64, device=DEV), torch.ones(32, device=DEV), \
        torch.ones(64, device=DEV)
    q, k = gs.qk_norm_rope_forward(x, x, w, w, pos, freq)
    assert q.shape == x.shape
    g = gs.qk_norm_rope_backward(x, x, w, w, pos, freq, x, x)
    assert torch.all(g[2] == 0) and torch.all(g[3] == 0)


def test_relative_position():
    """q . k after rotation depends on the distance alone (any start)."""
    r = torch.Generator(device=DEV).manual_seed(1)
    q, k = torch.randn(1, 1, 64, generator=r, device=DEV), torch.randn(1, 1, 64, generator=r, device=DEV)
    freq, _ = gs.rotary_frequencies(64, device=DEV)
    dots = []
    for s in (0, 7, 100000, 2 ** 30):
        a = gs.qk_norm_rope_forward(q, None, None, None, torch.tensor([s + 13], device=DEV), freq)[0]
        b = gs.qk_norm_rope_forward(k, None, None, None, torch.tensor([s], device=DEV), freq)[0]
        dots.append(float((a.double() * b.double()).sum()))
    # 64 products of size ~1, each with a few roundings
    assert max(dots) - min(dots) <= 64 * 16 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_autograd(dtype):
    m = make(50, 3, 2, 64, 32, dtype)
    args = call_args(m)
    leaves = [x.clone().contiguous().requires_grad_() for x in args[:4]]
    q, k = gs.qk_norm_rope(*leaves, *args[4:], layout="interleaved", magnitude=1.1)
    dy = [x.to(DEV) for x in m["dy"]]
    ((q.float() * dy[0].float()).sum() + (k.float() * dy[1].float()).sum()).backward()
    g = gs.qk_norm_rope_backward(*args, *dy, layout="interleaved", magnitude=1.1)
    for x, y in zip(leaves, g):
        assert torch.equal(x.grad, y)
    # only the keys are used
    leaves = [x.detach().clone().requires_grad_() for x in leaves]
    _, k = gs.qk_norm_rope(*leaves, *args[4:])
    k.sum().backward()
    assert torch.all(leaves[0].grad == 0) and leaves[1].grad.abs().sum() > 0


def test_other_stream_and_graph():
    m = make(300, 4, 2, 64, 64, BF)
    args = call_args(m)
    dy = [x.to(DEV) for x in m["dy"]]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)

    def work(stream=None):
        return gs.qk_norm_rope_forward(*args, stream=stream) + \
            gs.qk_norm_rope_backward(*args, *dy, workspace=ws, stream=stream)

    a = work()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = work(s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = work()
    for _ in range(3):
        args[0].copy_(torch.randn(args[0].shape, device=DEV))
        torch.randn(1 << 16, device=DEV).add_(1)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        assert all(torch.equal(x, y) for x, y in zip(got, work()))
