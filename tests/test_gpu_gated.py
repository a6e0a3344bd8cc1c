"""The gated projection (gscan_gated_projection_*, through the package) against its
64-bit form.

Tolerances (lm_ref).  The activation adds a few roundings of its argument's size (up to
8 here): 32 u.  bf16: one rounding of the output; in the backward the gradients of both
products are rounded before the products that take them: twice.  dx adds two products."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests import lm_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
NAMES = ["silu", "gelu", "gelu_tanh"]


def inside(t, fill=float("nan")):
    """t on the GPU in the middle of a larger tensor of NaN: nothing around it may be read."""
    big = torch.full((t.shape[0] + 3, t.shape[1] + 24), fill, dtype=t.dtype, device=DEV)
    big[1:1 + t.shape[0], 8:8 + t.shape[1]] = t.to(DEV)
    return big[1:1 + t.shape[0], 8:8 + t.shape[1]]


def make(n, D, F, dtype, seed=1):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(n, D, generator=gen).to(dtype)
    wg, wu = ((torch.randn(F, D, generator=gen) * 2 * D ** -0.5).to(dtype) for _ in range(2))
    return x, wg, wu, torch.randn(n, F, generator=gen).to(dtype)


CASES = {  # tokens, width, inner
    "smallest": (1, 8, 8),
    "one token": (1, 512, 1368),
    "few tokens": (16, 72, 40),
    "one more": (17, 136, 24),
    "last of the few": (32, 264, 520),
    "first tiles": (33, 64, 64),
    "k ends inside a step": (65, 200, 72),
    "a tile and one": (129, 128, 136),
    "tiles divided along k": (64, 4096, 64),
    "tokens divided": (3000, 64, 48),
    "odd": (515, 328, 680),
    "several rounds": (2100, 96, 4104),
    "large tiles": (4100, 136, 2056),
}


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_forward_and_backward(name, dtype):
    n, D, F = CASES[name]
    act = NAMES[(n + D) % 3]
    print(f"case gated projection: {name} {act} {dtype}", flush=True)
    x, wg, wu, d = make(n, D, F, dtype)
    args = inside(x), inside(wg), inside(wu)
    tol = ref.product(D) + 32 * ref.U
    out = torch.full((n + 2, F), 7.0, dtype=dtype, device=DEV)
    y = gs.gated_projection_forward(*args, activation=act, out=out[1:-1])
    ref.close(y, ref.gate(x, wg, wu, act), 2 * tol + ref.rounding(dtype), "out")
    assert bool((out[[0, -1]] == 7).all())
    assert torch.equal(y, gs.gated_projection_forward(*args, activation=act))
    g = gs.gated_projection_backward(*args, inside(d), activation=act)
    want = ref.gate_grad(x, wg, wu, d, act)
    for got, w, K, what in zip(g, want, (2 * F, n, n), ("dx", "d_w_gate", "d_w_up")):
        ref.close(got, w, 2 * tol + ref.product(K) + 2 * ref.rounding(dtype), what)
    again = gs.gated_projection_backward(*args, inside(d), activation=act)
    assert all(torch.equal(a, b) for a, b in zip(g, again))


@pytest.mark.parametrize("act", NAMES)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_halves_of_one_matrix_and_batches(dtype, act):
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(3, 5, 48, generator=gen).to(dtype)
    w = (torch.randn(2 * 40, 48, generator=gen) * 0.3).to(dtype)
    wd = w.to(DEV)
    y = gs.gated_projection_forward(x.to(DEV), wd[:40], wd[40:], activation=act)
    assert y.shape == (3, 5, 40)
    tol = 2 * (ref.product(48) + 32 * ref.U) + ref.rounding(dtype)
    ref.close(y.flatten(0, 1), ref.gate(x.flatten(0, 1), w[:40], w[40:], act), tol, "out")


@pytest.mark.parametrize("act", NAMES)
def test_far_arguments(act):
    """Products far from zero: the activation is linear or zero there, never NaN."""
    x = torch.eye(8, device=DEV)[:1].repeat(40, 1)
    far = torch.tensor([1e4, -1e4, 1e18, -1e18, 90.0, -90.0, 0.0, -0.0], device=DEV)
    wg = torch.zeros(8, 8, device=DEV)
    wg[:, 0] = far
    wu = torch.ones(8, 8, device=DEV)
    for rows in (x, x[:1]):  # tiles, and few tokens
        y = gs.gated_projection_forward(rows, wg, wu, activation=act)
        want = torch.where(far > 1, far, torch.zeros_like(far))
        assert torch.allclose(y, want.expand_as(y), rtol=1e-6, atol=1e-30)
        dx, dg, du = gs.gated_projection_backward(rows, wg, wu, torch.ones_like(y), activation=act)
        assert all(bool(torch.isfinite(t).all()) for t in (dx, dg, du))


@pytest.mark.parametrize("n", [5, 70, 400])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_nonfinite_token_stays_alone(n, dtype):
    x, wg, wu, d = (t.to(DEV) for t in make(n, 72, 80, dtype))
    clean = gs.gated_projection_forward(x, wg, wu)
    dx = gs.gated_projection_backward(x, wg, wu, d)[0]
    x[n // 2, 3] = float("nan")
    y, g = gs.gated_projection_forward(x, wg, wu), gs.gated_projection_backward(x, wg, wu, d)
    keep = torch.arange(n, device=DEV) != n // 2
    assert bool(torch.isnan(y[n // 2]).all()) and torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(g[0][n // 2]).all()) and torch.equal(g[0][keep], dx[keep])
    assert bool(torch.isnan(g[1][:, 3]).all())  # as in the formulas: da of that token is NaN


def test_nothing_and_parts():
    x, wg, wu, d = (t.to(DEV) for t in make(50, 64, 72, BF))
    empty = x[:0]
    assert gs.gated_projection_forward(empty, wg, wu).shape == (0, 72)
    g = gs.gated_projection_backward(empty, wg, wu, d[:0])
    assert g[0].shape == (0, 64) and bool((g[1] == 0).all()) and bool((g[2] == 0).all())
    full = gs.gated_projection_backward(x, wg, wu, d)
    a = gs.gated_projection_backward(x, wg, wu, d, wanted=(True, False))
    b = gs.gated_projection_backward(x, wg, wu, d, wanted=(False, True))
    assert a[1] is None and a[2] is None and b[0] is None
    assert torch.equal(a[0], full[0]) and torch.equal(b[1], full[1]) and torch.equal(b[2], full[2])


def test_rows_past_32_bits():
    n, D = 300000, 8192  # 4.9 GB
    x = torch.zeros(n, D, dtype=BF, device=DEV)
    x[-1, 5], x[-2, 8191], x[0, 0] = 2.0, 3.0, 1.0
    wg, wu = torch.zeros(8, D, dtype=BF, device=DEV), torch.ones(8, D, dtype=BF, device=DEV)
    wg[:, [0, 5, 8191]] = 1.0
    y = gs.gated_projection_forward(x, wg, wu)
    s = torch.sigmoid(torch.tensor([1.0, 2.0, 3.0], dtype=torch.float64))
    for row, v, g in ((0, 1.0, s[0]), (-1, 2.0, s[1]), (-2, 3.0, s[2])):
        assert abs(float(y[row, 7]) - v * v * float(g)) <= 2.0 ** -8 * v * v
    assert float(y[1:-2].abs().max()) == 0.0
    d = torch.ones(n, 8, dtype=BF, device=DEV)
    dg = gs.gated_projection_backward(x, wg, wu, d, wanted=(False, True))[1]
    assert dg.shape == (8, D) and float(dg[0, 1:5].abs().max()) == 0.0
    slope = float(s[1] * (1 + 2.0 * (1 - s[1])))
    assert abs(float(dg[3, 5]) - 2.0 * slope * 2.0) <= 2.0 ** -6 * 4 * slope  # x * b * act'


def test_far_rows():
    """The largest row stride."""
    big = torch.zeros(5 * 2 ** 21, dtype=F32, device=DEV).view(5, 2 ** 21)
    x, wg, wu, d = make(5, 16, 24, F32)
    big[:, :16] = x.to(DEV)
    y = gs.gated_projection_forward(big[:, :16], wg.to(DEV), wu.to(DEV))
    ref.close(y, ref.gate(x, wg, wu, "silu"), 2 * (ref.product(16) + 32 * ref.U), "out")
    g = gs.gated_projection_backward(big[:, :16], wg.to(DEV), wu.to(DEV), d.to(DEV))
    for got, w in zip(g, ref.gate_grad(x, wg, wu, d, "silu")):
        ref.close(got, w, 4 * (ref.product(48) + 32 * ref.U), "gradient")


def test_same_row_for_all_tokens():
    """A row stride of zero."""
    x, wg, wu, d = make(70, 40, 32, F32)
    rows = x[:1].to(DEV).expand(70, 40)
    y = gs.gated_projection_forward(rows, wg.to(DEV), wu.to(DEV))
    assert torch.equal(y, y[:1].expand_as(y))
    g = gs.gated_projection_backward(rows, wg.to(DEV), wu.to(DEV), d.to(DEV))
    want = ref.gate_grad(x[:1].expand(70, 40), wg, wu, d, "silu")
    for got, w in zip(g, want):
        ref.close(got, w, 4 * (ref.product(80) + 32 * ref.U), "gradient")


def test_directional_difference():
    """The gradient along a direction against the forward's own difference.  Step 2^-5 of a
    direction of unit elements: the cubic term is 2^-10 / 6 of third derivatives of a few
    times the sum's root-mean-square size, the forward's roundings 2^-24 * 2^5 of it."""
    x, wg, wu, d = (t.to(DEV) for t in make(40, 64, 96, F32))
    gen = torch.Generator().manual_seed(9)
    g = gs.gated_projection_backward(x, wg, wu, d, activation="gelu")
    for i, t in enumerate((x, wg, wu)):
        v = torch.randn(t.shape, generator=gen).to(DEV) * (1.0 if i == 0 else 64 ** -0.5)

        def f(sign):
            args = [x, wg, wu]
            args[i] = t + sign * 2.0 ** -5 * v
            return float((gs.gated_projection_forward(*args, activation="gelu").double() * d.double()).sum())

        slope = (f(1) - f(-1)) / 2.0 ** -4
        size = float(g[i].double().norm()) * float(v.double().norm()) / t.numel() ** 0.5
        assert abs(slope - float((g[i].double() * v.double()).sum())) <= 2.0 ** -6 * size


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_autograd(dtype):
    gen = torch.Generator().manual_seed(3)
    base = torch.randn(20, 69, generator=gen).to(dtype).to(DEV)
    _, wg, wu, d = (t.to(DEV) for t in make(20, 64, 48, dtype))
    for x in (base[:, :64].contiguous(), base[:, 5:69]):  # the second on no multiple of 16 bytes
        leaves = [t.detach().clone().requires_grad_() for t in (x, wg, wu)]
        gs.gated_projection(*leaves, activation="gelu").backward(d)
        g = gs.gated_projection_backward(x.contiguous().clone(), wg, wu, d, activation="gelu")
        assert all(torch.equal(a.grad, b) for a, b in zip(leaves, g))
    frozen = gs.gated_projection(leaves[0], wg, leaves[2].detach().requires_grad_())
    frozen.sum().backward()  # an upstream gradient without strides
    assert wg.grad is None


def test_other_stream_and_graph():
    x, wg, wu, d = (t.to(DEV) for t in make(300, 264, 136, BF))
    ws = torch.empty(gs.gated_projection_backward_workspace_bytes(x, wg, wu), dtype=torch.uint8, device=DEV)
    wf = torch.empty(max(1, gs.gated_projection_forward_workspace_bytes(x, wg, wu)), dtype=torch.uint8, device=DEV)

    def work(stream=None):
        return (gs.gated_projection_forward(x, wg, wu, workspace=wf, stream=stream),
                gs.gated_projection_forward(x[:3], wg, wu, stream=stream),
                *gs.gated_projection_backward(x, wg, wu, d, workspace=ws, stream=stream))

    a = work()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = work(s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for _ in range(3):
        x.copy_(torch.randn(x.shape, device=DEV))
        torch.randn(1 << 16, device=DEV).add_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        assert all(torch.equal(p, q) for p, q in zip(got, work()))


def test_two_streams_at_once():
    x, wg, wu, d = (t.to(DEV) for t in make(700, 512, 264, F32))
    want = gs.gated_projection_backward(x, wg, wu, d)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for s, into in zip(streams, got):
            with torch.cuda.stream(s):
                into.append(gs.gated_projection_backward(x, wg, wu, d))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for into in got for g in into for p, q in zip(g, want))


def test_refusals():
    x, wg, wu, d = (t.to(DEV) for t in make(4, 16, 24, F32))
    for args in ((x, wg, wu[:8]), (x, wg.T, wu.T), (x, wg.to(BF), wu.to(BF)), (x.half(), wg.half(), wu.half()),
                 (x, wg, wu.cpu()), (x[:, :8], wg, wu)):
        with pytest.raises((TypeError, ValueError)):
            gs.gated_projection_forward(*args)
    with pytest.raises(ValueError):
        gs.gated_projection_forward(x, wg, wu, activation="relu")
    with pytest.raises(ValueError):
        gs.gated_projection_backward(x, wg, wu, d[:2])
    with pytest.raises(ValueError):
        gs.gated_projection_backward(x, wg, wu, None)
    with pytest.raises(gs.GScanError):
        gs.gated_projection_forward(torch.zeros(4, 12, device=DEV), torch.zeros(8, 12, device=DEV),
                                    torch.zeros(8, 12, device=DEV))
    with pytest.raises((ValueError, gs.GScanError)):
        gs.gated_projection_backward(x, wg, wu, d, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
