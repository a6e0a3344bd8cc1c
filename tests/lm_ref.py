"""Plain 64-bit forms of the token embedding, the gated projection and the
vocabulary's cross entropy (torch, elementary operations), and the tolerances of
their tests.

Rounding, u = 2^-24.  A product of the library sums its k in chains of at most 256
(fp32) or K / 16 matrix instructions (bf16: each exact to fp32), joined by a chain
of K / 256.  Roundings of a chain of n are independent: their sum is sqrt(n) / 2 of
the terms' size at a typical element, and the 2-norm over an output holds the typical
element; four times that is asked of the norm (`product`).  One rounding to bf16 is at
most half a step: eps / 2 = 2^-8 relative, of every element and so of the norm.
"""
import math

import torch

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def product(K):
    """Of the 2-norm of a product's result with K terms in fp32 accumulation."""
    return (2 * math.sqrt(256) + 2 * math.sqrt(K / 256 + 1) + 8) * U


def rounding(dtype):
    return torch.finfo(dtype).eps / 2 if dtype == BF else 0.0


def embed(table, tokens, scale):
    ok = (tokens >= 0) & (tokens < len(table))
    rows = table.double()[tokens.clamp(0, len(table) - 1).long()] * scale
    return torch.where(ok[..., None], rows, torch.zeros((), dtype=torch.float64))


def embed_grad(d_out, tokens, vocabulary, scale):
    d, t = d_out.double().reshape(-1, d_out.shape[-1]), tokens.reshape(-1).long()
    ok = (t >= 0) & (t < vocabulary)
    g = torch.zeros(vocabulary, d.shape[1], dtype=torch.float64)
    for i in torch.nonzero(ok)[:, 0].tolist():
        g[t[i]] += d[i]
    return g * scale


def act(a, name):
    """(act(a), its derivative)"""
    if name == "silu":
        g = 1 / (1 + torch.exp(-a))
        return a * g, g + a * g * (1 - g)
    if name == "gelu":
        p = (1 + torch.erf(a / math.sqrt(2))) / 2
        return a * p, p + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (a + 0.044715 * a ** 3))
    return a * (1 + t) / 2, (1 + t) / 2 + a / 2 * (1 - t * t) * c * (1 + 3 * 0.044715 * a * a)


def gate(x, wg, wu, name):
    x, wg, wu = x.double(), wg.double(), wu.double()
    return act(x @ wg.T, name)[0] * (x @ wu.T)


def gate_grad(x, wg, wu, d_out, name):
    x, wg, wu, d = x.double(), wg.double(), wu.double(), d_out.double()
    a, b = x @ wg.T, x @ wu.T
    f, slope = act(a, name)
    da, db = d * b * slope, d * f
    return da @ wg + db @ wu, da.T @ x, db.T @ x


def logits(h, w, scale):
    return h.double() @ w.double().T * scale


def loss(h, w, target, scale, reduction):
    """(loss, lse) of the tokens that count; the others' rows of h are not looked at."""
    ok = (target >= 0) & (target < len(w))
    z = logits(h[ok], w, scale)
    m = z.amax(-1, keepdim=True)
    lse = (m + torch.log(torch.exp(z - m).sum(-1, keepdim=True)))[:, 0]
    each, all_lse = torch.zeros(len(h), dtype=torch.float64), torch.zeros(len(h), dtype=torch.float64)
    each[ok] = lse - z[torch.arange(len(z)), target[ok].long()]
    all_lse[ok] = lse
    if reduction != "none":
        each = each.sum() / (max(1, int(ok.sum())) if reduction == "mean" else 1)
    return each, all_lse


def loss_grad(h, w, target, d_loss, scale, reduction):
    ok = (target >= 0) & (target < len(w))
    z = logits(h[ok], w, scale)
    p = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
    p[torch.arange(len(z)), target[ok].long()] -= 1
    d = d_loss.double()
    if reduction == "none":
        p = p * d[ok][:, None]
    else:
        p = p * d / (max(1, int(ok.sum())) if reduction == "mean" else 1)
    dh = torch.zeros(h.shape, dtype=torch.float64)
    dh[ok] = scale * (p @ w.double())
    return dh, scale * (p.T @ h[ok].double())


def close(got, ref, tol, what):
    """The 2-norm of the difference, and no element further than eight times as far as
    the largest allows."""
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), what
    if not ref.numel():
        return
    norm, err = float(ref.norm()), float((got - ref).norm())
    print(f"  {what}: {err / max(norm, 1e-300):.2e} of {tol:.2e}", flush=True)
    assert err <= tol * norm, what
    assert float((got - ref).abs().max()) <= 8 * tol * float(ref.abs().max()), what
