"""The vocabulary's cross entropy (gscan_linear_cross_entropy_*, through the package)
against its 64-bit form.

Tolerances (lm_ref).  Log-sums and losses are differences of logits and of the logarithm
of a sum of up to V exponentials: absolute, of the largest logit's size z: a product's
roundings, a dozen of z and of the logarithm, and of the sum its chains (64 of a lane, then
a tree).  The gradient of a logit has the exponential's argument's error (|z| + |lse|
roundings); bf16: it is rounded, and the output again."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests import lm_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def inside(t, fill=float("nan")):
    big = torch.full((t.shape[0] + 3, t.shape[1] + 24), fill, dtype=t.dtype, device=DEV)
    big[1:1 + t.shape[0], 8:8 + t.shape[1]] = t.to(DEV)
    return big[1:1 + t.shape[0], 8:8 + t.shape[1]]


def make(n, D, V, dtype, ignored=0.0, seed=1, size=2.0):
    gen = torch.Generator().manual_seed(seed)
    h = torch.randn(n, D, generator=gen).to(dtype)
    w = (torch.randn(V, D, generator=gen) * size * D ** -0.5).to(dtype)
    target = torch.randint(0, V, (n,), generator=gen)
    target[torch.rand(n, generator=gen) < ignored] = -100
    return h, w, target, torch.rand(n, generator=gen) + 0.5


def loss_tolerance(h, w, target, scale):
    z = float(ref.logits(h, w, scale).abs().max()) if len(h) else 0.0
    return (z + 1) * (ref.product(h.shape[1]) + 12 * ref.U) + 80 * ref.U, z


CASES = {  # tokens, width, vocabulary, ignored, reduction, scale
    "smallest": (1, 8, 1, 0, "none", 1.0),
    "one token": (1, 256, 3001, 0, "mean", 1.0),
    "few tokens": (16, 72, 130, 0.3, "none", 0.5),
    "one more": (17, 136, 1000, 0, "sum", 1.0),
    "last of the few": (32, 64, 8193, 0.5, "mean", 1.0),
    "first tiles": (33, 64, 257, 0.2, "none", 1.0),
    "vocabulary of five": (200, 40, 5, 0.1, "sum", -1.0),
    "most do not count": (300, 128, 777, 0.97, "mean", 1.0),
    "none counts": (70, 64, 100, 1.1, "mean", 1.0),
    "odd": (515, 200, 1003, 0.125, "mean", 0.7),
    "tiles divided along k": (130, 2048, 136, 0, "none", 1.0),
    "large tiles": (2100, 64, 6011, 0.05, "mean", 1.0),
    "tiles divided as many do not count": (1141, 1248, 1134, 0.6, "none", 1.0),
}


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_forward_and_backward(name, dtype):
    n, D, V, ignored, reduction, scale = CASES[name]
    print(f"case cross entropy: {name} {dtype}", flush=True)
    h, w, target, up = make(n, D, V, dtype, ignored)
    if V > 3:
        target[target == 2] = V + 5  # not counted either
    dead = (target < 0) | (target >= V)
    h[dead] = float("nan")  # what rows that do not count hold reaches nothing
    clean = torch.where(dead[:, None], torch.zeros((), dtype=dtype), h)
    hd, wd = inside(h), inside(w)
    td = target.to(DEV) if n % 2 else target.to(torch.int32).to(DEV)
    kw = dict(scale=scale, reduction=reduction)
    loss, lse = gs.linear_cross_entropy_forward(hd, wd, td, **kw)
    want, want_lse = ref.loss(clean, w, target, scale, reduction)
    tol, z = loss_tolerance(clean, w, target, scale)
    assert loss.dtype == lse.dtype == F32 and loss.shape == want.shape and lse.shape == (n,)
    many = (~dead).sum() if reduction == "sum" else 1
    assert float((loss.double().cpu() - want).abs().max()) <= tol * many
    assert float((lse.double().cpu() - want_lse).abs().max()) <= tol
    assert bool((lse.cpu()[dead] == 0).all())

    d = up if reduction == "none" else torch.tensor(1.3)
    lse[dead.to(DEV)] = float("nan")  # not read
    dh, dw = gs.linear_cross_entropy_backward(hd, wd, td, lse, d.to(DEV), **kw)
    want = ref.loss_grad(clean, w, target, d, scale, reduction)
    exponent = 2 * (2 * z + 2) * (ref.product(D) + 4 * ref.U)
    for got, r, K, what in zip((dh, dw), want, (V, n), ("dh", "dw")):
        if float(r.norm()) < 1e-6 * (1 + z):  # one class, or none counts: differences of equal numbers
            assert float(got.double().abs().max()) <= 4 * tol * float(d.max()) * (1 + float(w.double().abs().max()))
            continue
        ref.close(got, r, exponent + ref.product(K) + 2 * ref.rounding(dtype), what)
    assert bool((dh.cpu()[dead] == 0).all())
    again = gs.linear_cross_entropy_backward(hd, wd, td, lse, d.to(DEV), **kw)
    assert torch.equal(dh, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_pieces_of_the_vocabulary(dtype):
    """So many tokens that the gradient of the logits is formed in several pieces."""
    n, D, V = (70000 if dtype == F32 else 140000), 8, 5003
    h, w, target, _ = make(n, D, V, dtype, 0.3)
    hd, wd, td = h.to(DEV), w.to(DEV), target.to(DEV)
    loss, lse = gs.linear_cross_entropy_forward(hd, wd, td)
    d = torch.ones((), device=DEV)
    dh, dw = gs.linear_cross_entropy_backward(hd, wd, td, lse, d)
    ok = td >= 0
    count, total = int(ok.sum()), 0.0
    want_h, want_w = torch.zeros(n, D, dtype=torch.float64, device=DEV), torch.zeros(V, D, dtype=torch.float64, device=DEV)
    for rows in torch.nonzero(ok)[:, 0].split(8192):
        logp = torch.log_softmax(hd[rows].double() @ wd.double().T, -1)
        total += float(-logp[torch.arange(len(rows), device=DEV), td[rows]].sum())
        p = logp.exp()
        p[torch.arange(len(rows), device=DEV), td[rows]] -= 1
        want_h[rows] = p @ wd.double() / count
        want_w += p.T @ hd[rows].double() / count
    assert abs(float(loss) - total / count) <= 1e-5
    tol = 40 * (ref.product(D) + 4 * ref.U) + 2 * ref.rounding(dtype)
    ref.close(dh, want_h, tol + ref.product(V), "dh")
    ref.close(dw, want_w, tol + ref.product(n), "dw")
    assert bool((dh[~ok] == 0).all())


@pytest.mark.parametrize("n", [7, 90])
def test_nonfinite_logits_stay_alone(n):
    h, w, target, up = (t.to(DEV) for t in make(n, 48, 200, F32))
    clean, lse0 = gs.linear_cross_entropy_forward(h, w, target, reduction="none")
    dh0, _ = gs.linear_cross_entropy_backward(h, w, target, lse0, up, reduction="none")
    bad, keep = n // 2, torch.arange(n, device=DEV) != n // 2
    for value in (float("nan"), float("inf")):
        h2 = h.clone()
        h2[bad, 5] = value
        loss, lse = gs.linear_cross_entropy_forward(h2, w, target, reduction="none")
        assert bool(torch.isnan(loss[bad])) and torch.equal(loss[keep], clean[keep])
        dh, _ = gs.linear_cross_entropy_backward(h2, w, target, lse, up, reduction="none")
        assert bool(torch.isnan(dh[bad]).any()) and torch.equal(dh[keep], dh0[keep])


@pytest.mark.parametrize("n", [3, 60])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_extreme_logits(n, dtype):
    """A class that no token can have (its logits are minus infinity), and logits in the
    thousands."""
    h, w, target, _ = make(n, 32, 150, dtype, size=300.0)
    h, target = h.abs() + 0.5, torch.where(target == 7, torch.zeros_like(target), target)
    want, want_lse = ref.loss(h, torch.cat([w[:7], w[8:]]), torch.where(target > 7, target - 1, target), 1.0, "none")
    w[7] = float("-inf")
    loss, lse = gs.linear_cross_entropy_forward(h.to(DEV), w.to(DEV), target.to(DEV), reduction="none")
    size = float(want_lse.abs().max()) + float(want.abs().max())
    tol = size * (ref.product(32) + 12 * ref.U)
    assert float((loss.double().cpu() - want).abs().max()) <= tol
    assert float((lse.double().cpu() - want_lse).abs().max()) <= tol


def test_a_certain_token_has_no_loss():
    """One class far above all others: loss and gradient are zero, not noise."""
    h = torch.ones(40, 8, device=DEV)
    w = torch.zeros(50, 8, device=DEV)
    w[3] = 100.0
    t = torch.full((40,), 3, device=DEV)
    for rows in (40, 5):
        loss, lse = gs.linear_cross_entropy_forward(h[:rows], w, t[:rows], reduction="none")
        assert bool((loss == 0).all()) and bool((lse == 800).all())
        dh, dw = gs.linear_cross_entropy_backward(h[:rows], w, t[:rows], lse, torch.ones(rows, device=DEV),
                                                  reduction="none")
        assert bool((dh == 0).all()) and bool((dw == 0).all())


def test_nothing():
    h, w = torch.empty(0, 16, device=DEV), torch.ones(9, 16, device=DEV)
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    for reduction in ("none", "sum", "mean"):
        loss, lse = gs.linear_cross_entropy_forward(h, w, t, reduction=reduction)
        assert lse.shape == (0,) and float(loss.sum()) == 0.0
        d = torch.ones(loss.shape, device=DEV)
        dh, dw = gs.linear_cross_entropy_backward(h, w, t, lse, d, reduction=reduction)
        assert dh.shape == (0, 16) and bool((dw == 0).all())


def test_weights_past_32_bits():
    V, D = 300001, 8192  # 4.9 GB
    w = torch.zeros(V, D, dtype=BF, device=DEV)
    w[-1, 3] = 4.0
    h = torch.zeros(40, D, dtype=BF, device=DEV)
    h[:, 3] = 2.0
    t = torch.full((40,), V - 1, device=DEV)
    want = torch.log(torch.tensor(float(V - 1), dtype=torch.float64) + torch.exp(torch.tensor(8.0, dtype=torch.float64)))
    for rows in (40, 2):
        loss, lse = gs.linear_cross_entropy_forward(h[:rows], w, t[:rows], reduction="none")
        assert float((lse.double().cpu() - want).abs().max()) <= 200 * ref.U * 13
        assert float((loss.double().cpu() - (want - 8)).abs().max()) <= 200 * ref.U * 13
    dh, dw = gs.linear_cross_entropy_backward(h, w, t, lse.repeat(20), torch.ones((), device=DEV), reduction="sum")
    p = float(torch.exp(8 - want))
    assert abs(float(dw[-1, 3]) - 40 * 2 * (p - 1)) <= 2.0 ** -7 * 80
    assert abs(float(dh[0, 3]) - 4 * (p - 1)) <= 2.0 ** -7 * 4


def test_more_tokens_than_a_launch_has_groups():
    n, D, V = 2 ** 24 + 1000, 8, 5  # 16 tokens a workgroup, or one
    gen = torch.Generator(device=DEV).manual_seed(3)
    h = torch.randn(n, D, generator=gen, device=DEV)
    w = torch.randn(V, D, generator=gen, device=DEV)
    target = torch.randint(-1, V, (n,), generator=gen, device=DEV)
    ok = target >= 0
    z = h.double() @ w.double().T
    lse = torch.where(ok, torch.logsumexp(z, -1), 0.0)
    picked = torch.gather(z, 1, target.clamp(min=0)[:, None])[:, 0]
    loss, got = gs.linear_cross_entropy_forward(h, w, target, reduction="none")
    top = float(z.abs().max())
    tol = (top + 1) * (ref.product(D) + 12 * ref.U) + 80 * ref.U
    assert float((got.double() - lse).abs().max()) <= tol
    assert float((loss.double() - torch.where(ok, lse - picked, 0.0)).abs().max()) <= tol
    dh, dw = gs.linear_cross_entropy_backward(h, w, target, got, torch.ones(n, device=DEV), reduction="none")
    g = torch.softmax(z, -1)
    g[torch.arange(n, device=DEV), target.clamp(min=0)] -= 1.0
    g[~ok] = 0.0
    assert bool((dh[~ok] == 0).all())
    # a gradient of a logit: its exponential's argument is off by tol; then products of V and n terms
    ref.close(dh, g @ w.double(), 2 * tol + ref.product(V), "dh")
    ref.close(dw, g.T @ h.double(), 2 * tol + ref.product(n), "dW")


def test_directional_difference():
    """Step 2^-5 along directions that move logits by about one standard deviation: the
    cubic term is 2^-10 / 6 of the third derivative, of the size of the loss."""
    h, w, target, _ = (t.to(DEV) for t in make(60, 64, 300, F32, 0.1))
    loss, lse = gs.linear_cross_entropy_forward(h, w, target)
    g = gs.linear_cross_entropy_backward(h, w, target, lse, torch.ones((), device=DEV))
    gen = torch.Generator().manual_seed(9)
    for i in range(2):
        v = torch.randn((h, w)[i].shape, generator=gen).to(DEV) * (0.5 if i == 0 else 64 ** -0.5)

        def f(sign):
            a = (h + sign * 2.0 ** -5 * v, w) if i == 0 else (h, w + sign * 2.0 ** -5 * v)
            return float(gs.linear_cross_entropy_forward(*a, target)[0].double())

        # a mean of 54 losses of about six, each good to 2^-20
        assert abs((f(1) - f(-1)) / 2.0 ** -4 - float((g[i].double() * v.double()).sum())) <= 2.0 ** -9


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_autograd(dtype, reduction):
    gen = torch.Generator().manual_seed(3)
    base = torch.randn(4, 10, 69, generator=gen).to(dtype).to(DEV)
    _, w, target, _ = (t.to(DEV) for t in make(40, 64, 333, dtype, 0.2))
    for h in (base[..., :64].contiguous(), base[..., 5:69]):  # the second on no multiple of 16 bytes
        leaves = [h.detach().clone().requires_grad_(), w.clone().requires_grad_()]
        loss = gs.linear_cross_entropy(*leaves, target.view(4, 10), reduction=reduction)
        (loss * 2.0).sum().backward()  # without strides for "none"
        flat = h.reshape(40, 64).contiguous()
        _, lse = gs.linear_cross_entropy_forward(flat, w, target, reduction=reduction)
        d = torch.full((40,) if reduction == "none" else (), 2.0, device=DEV)
        g = gs.linear_cross_entropy_backward(flat, w, target, lse, d, reduction=reduction)
        assert torch.equal(leaves[0].grad.view(40, 64), g[0]) and torch.equal(leaves[1].grad, g[1])
    part = w.clone().requires_grad_()
    gs.linear_cross_entropy(flat, part, target).backward()
    dh, dw = gs.linear_cross_entropy_backward(flat, w, target, lse, torch.ones((), device=DEV), wanted=(False, True))
    assert dh is None and torch.equal(part.grad, dw)


def test_a_batch_without_its_first_targets():
    h, w, target, _ = (t.to(DEV) for t in make(36, 24, 50, F32, 0.1))
    target = target.view(4, 9)
    leaf = h.view(4, 9, 24)[:, :-1].clone().requires_grad_()
    loss = gs.linear_cross_entropy(leaf, w, target[:, 1:])
    dense = target[:, 1:].contiguous()
    want, lse = gs.linear_cross_entropy_forward(leaf.detach(), w, dense)
    assert torch.equal(loss.detach(), want)
    loss.backward()
    dh, _ = gs.linear_cross_entropy_backward(leaf.detach(), w, dense, lse, torch.ones((), device=DEV),
                                             wanted=(True, False))
    assert torch.equal(leaf.grad, dh)
    with pytest.raises(ValueError):
        gs.linear_cross_entropy_forward(leaf.detach(), w, target[:, 1:])


def test_other_stream_and_graph():
    h, w, target, _ = (t.to(DEV) for t in make(300, 136, 1003, BF, 0.2))
    d = torch.ones((), device=DEV)
    wf = torch.empty(gs.linear_cross_entropy_forward_workspace_bytes(h, w, target), dtype=torch.uint8, device=DEV)
    wb = torch.empty(gs.linear_cross_entropy_backward_workspace_bytes(h, w, target), dtype=torch.uint8, device=DEV)

    def work(stream=None):
        loss, lse = gs.linear_cross_entropy_forward(h, w, target, workspace=wf, stream=stream)
        few = gs.linear_cross_entropy_forward(h[:9], w, target[:9], stream=stream)
        return (loss, lse, *few, *gs.linear_cross_entropy_backward(h, w, target, lse, d, workspace=wb, stream=stream))

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
    for i in range(4):
        h.copy_(torch.randn(h.shape, device=DEV))
        # other tokens count, at last none: what the device finds decides, not what was captured
        target.copy_(torch.randint(-500 * i, 1003 if i < 3 else 0, (300,), device=DEV))
        torch.randn(1 << 16, device=DEV).add_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        assert all(torch.equal(p, q) for p, q in zip(got, work()))


def test_refusals():
    h, w, target, up = (t.to(DEV) for t in make(4, 16, 24, F32))
    for args in ((h, w[:, :8], target), (h, w.to(BF), target), (h.half(), w.half(), target), (h, w, target[:2]),
                 (h, w, target.float()), (h, w.cpu(), target), (h.T, w, target)):
        with pytest.raises((TypeError, ValueError)):
            gs.linear_cross_entropy_forward(*args)
    with pytest.raises(ValueError):
        gs.linear_cross_entropy_forward(h, w, target, reduction="average")
    _, lse = gs.linear_cross_entropy_forward(h, w, target)
    for bad in (dict(d_loss=up), dict(d_loss=up[0].double()), dict(lse=lse[:2]), dict(d_loss=1.0)):
        with pytest.raises(ValueError):
            gs.linear_cross_entropy_backward(h, w, target, **dict(dict(lse=lse, d_loss=up[0].clone()), **bad))
    with pytest.raises((ValueError, gs.GScanError)):
        gs.linear_cross_entropy_forward(h, w, target, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
