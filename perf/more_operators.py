"""Measured cases of a language model's two ends and its feed-forward block:
the token embedding, the gated projection, and the cross entropy over a
vocabulary, each with its gradients.  Inputs, plain forms in elementary torch
operations, the definitions in 64 bits, and the work each pass cannot do
without.

A case is a dict with a "kind":
  embed   embed_forward: rows of a table, scaled
  dembed  embed_backward: the table's gradient
  gate    gated_projection_forward: act(x Wg^T) * (x Wu^T)
  dgate   gated_projection_backward: gradients of x and both weights
  loss    linear_cross_entropy_forward: losses and log-sums of h W^T, of the
          tokens that count (zero for the others)
  dloss   linear_cross_entropy_backward: gradients of h and W
"""
import math

import torch

own = False

EPOCH = 1024  # rows at a time of the definitions in 64 bits


# ------------------------------------------------------------------- cases

def _embed(kind, name, table, dtype, tokens, vocabulary, width, scale):
    c = {"kind": kind, "table": table, "dtype": dtype, "tokens": tokens, "vocabulary": vocabulary,
         "width": width, "scale": scale}
    return dict(c, name=name) if name else c


def _gate(kind, name, dtype, tokens, width, inner, activation):
    c = {"kind": kind, "dtype": dtype, "tokens": tokens, "width": width, "inner": inner,
         "activation": activation}
    return dict(c, name=name) if name else c


def _loss(kind, name, dtype, tokens, width, vocabulary, ignored, reduction):
    c = {"kind": kind, "dtype": dtype, "tokens": tokens, "width": width, "vocabulary": vocabulary,
         "ignored": ignored, "reduction": reduction}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the last token of one request, looked up for the next step
        _embed("embed", "embed_one_bf16", "bf16", "bf16", 1, 32000, 2048, 1.0),
        # a training batch: a float32 table read into bfloat16 activations, scaled by the root of the width
        _embed("embed", "embed_batch_f32", "f32", "bf16", 16384, 32000, 1024, 32.0),
        # gradients of a small model's table
        _embed("dembed", "dembed_small_f32", "f32", "f32", 777, 1003, 200, 1.0),
        # ... and of a training batch: a few tokens make up much of it, most of the table gets nothing
        _embed("dembed", "dembed_batch_bf16", "f32", "bf16", 16384, 32000, 2048, 1.0),
        # one request generates one token: the weights are all there is to read
        _gate("gate", "gate_one_bf16", "bf16", 1, 2048, 5504, "silu"),
        # the forward of a training step
        _gate("gate", "gate_batch_bf16", "bf16", 8192, 2048, 5504, "silu"),
        # gradients of a small float32 model
        _gate("dgate", "dgate_small_f32", "f32", 515, 512, 1368, "gelu_tanh"),
        # gradients of packed sequences, whose number of tokens is what it is
        _gate("dgate", "dgate_batch_bf16", "bf16", 4109, 2048, 5504, "silu"),
        # a few continuations of a request scored
        _loss("loss", "loss_few_bf16", "bf16", 19, 2048, 32000, 0.0, "none"),
        # the loss of a training step
        _loss("loss", "loss_batch_bf16", "bf16", 8192, 2048, 32000, 0.0, "mean"),
        # gradients of a small float32 model
        _loss("dloss", "dloss_small_f32", "f32", 300, 256, 1003, 0.0, "mean"),
        # gradients of packed sequences, an eighth of whose tokens (prompts, padding) does not count
        _loss("dloss", "dloss_packed_bf16", "bf16", 6007, 1024, 50021, 0.125, "mean"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + (n % 1024 == 0)  # hardly ever a round size


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / (50 if case["dtype"] == "bf16" else 10))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        case = _any(rng)
        if _cost(case) <= top:
            return case


def _any(rng):
    kind = rng.choice(["embed", "dembed", "gate", "gate", "dgate", "loss", "loss", "dloss"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    width = 8 * _log_int(rng, 8, 256)
    if kind in ("embed", "dembed"):
        return _embed(kind, None, rng.choice(["bf16", "f32"]), dtype, _log_int(rng, 1, 32768),
                      _log_int(rng, 50, 50021), width, rng.choice([1.0, 1.0, width ** 0.5]))
    if kind in ("gate", "dgate"):
        return _gate(kind, None, dtype, _log_int(rng, 1, 8192), width, 8 * _log_int(rng, 8, 688),
                     rng.choice(["silu", "silu", "gelu", "gelu_tanh"]))
    return _loss(kind, None, dtype, _log_int(rng, 1, 8192), width, _log_int(rng, 50, 50021),
                 rng.choice([0.0, 0.125, 0.5]), rng.choice(["none", "sum", "mean"]))


# ------------------------------------------------------------------ inputs

def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _zipf(n, vocabulary, gen, dev):
    """Tokens whose frequencies fall with their rank, the ranks in no order."""
    u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocabulary + 1.0)).long() - 1).clamp(0, vocabulary - 1)
    return torch.randperm(vocabulary, generator=gen, device=dev)[rank]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ty = _type(case["dtype"])
    n, D = case["tokens"], case["width"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": case}
    if case["kind"] in ("embed", "dembed"):
        s["tokens"] = _zipf(n, case["vocabulary"], gen, dev)
        if case["kind"] == "embed":
            s["table"] = normal(case["vocabulary"], D).mul_(D ** -0.5).to(_type(case["table"]))
        else:
            s["dy"] = normal(n, D).to(ty)
    elif case["kind"] in ("gate", "dgate"):
        s["x"] = normal(n, D).to(ty)
        s["wg"] = normal(case["inner"], D).mul_(D ** -0.5).to(ty)
        s["wu"] = normal(case["inner"], D).mul_(D ** -0.5).to(ty)
        if case["kind"] == "dgate":
            s["dy"] = normal(n, case["inner"]).to(ty)
    else:
        V = case["vocabulary"]
        s["h"] = normal(n, D).to(ty)
        s["w"] = normal(V, D).mul_(2.0 * D ** -0.5).to(ty)
        target = _zipf(n, V, gen, dev)
        dead = torch.rand(n, generator=gen, device=dev) < case["ignored"]
        s["target"] = target.masked_fill(dead, -100)
        if case["kind"] == "dloss":
            # what the forward has left, and the gradient of its result
            s["lse"] = torch.cat([_plain_lse(h.float() @ s["w"].float().T) for h in s["h"].split(4096)])
            up = torch.rand((n,) if case["reduction"] == "none" else (), generator=gen, device=dev)
            s["up"] = up + 0.5
    return s


# -------------------------------------------------------------- plain forms

def _plain_lse(z):
    m = z.amax(-1, keepdim=True)
    return (m + torch.log(torch.sum(torch.exp(z - m), -1, keepdim=True)))[:, 0]


def _plain_act(a, activation):
    """(act(a), its derivative)"""
    if activation == "silu":
        g = 1 / (1 + torch.exp(-a))
        return a * g, g * (1 + a * (1 - g))
    if activation == "gelu":
        p = 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
        return a * p, p + a * torch.exp(-0.5 * a * a) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (a + 0.044715 * a * a * a))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * c * (1 + 3 * 0.044715 * a * a)


def _plain_reduce(loss, live, reduction):
    if reduction == "none":
        return loss
    total = torch.sum(loss.double())
    return (total / live.sum().clamp(min=1) if reduction == "mean" else total).float()


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import gated_linear_recurrence_history_amd as gs
        if kind == "embed":
            return gs.embed_forward(s["table"], s["tokens"], scale=case["scale"], dtype=_type(case["dtype"]))
        if kind == "dembed":
            return gs.embed_backward(s["dy"], s["tokens"], case["vocabulary"], scale=case["scale"],
                                     dtype=_type(case["table"]))
        if kind == "gate":
            return gs.gated_projection_forward(s["x"], s["wg"], s["wu"], activation=case["activation"])
        if kind == "dgate":
            return gs.gated_projection_backward(s["x"], s["wg"], s["wu"], s["dy"],
                                                activation=case["activation"])
        if kind == "loss":
            return gs.linear_cross_entropy_forward(s["h"], s["w"], s["target"], reduction=case["reduction"])
        return gs.linear_cross_entropy_backward(s["h"], s["w"], s["target"], s["lse"], s["up"],
                                                reduction=case["reduction"])

    ty = _type(case["dtype"])
    if kind == "embed":
        return (s["table"][s["tokens"]].float() * case["scale"]).to(ty)
    if kind == "dembed":
        total = torch.zeros(case["vocabulary"], case["width"], device=s["dy"].device)
        total.index_add_(0, s["tokens"], s["dy"].float())
        return (total * case["scale"]).to(_type(case["table"]))
    if kind in ("gate", "dgate"):
        x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
        a, b = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
        f, slope = _plain_act(a, case["activation"])
        if kind == "gate":
            return (f * b).to(ty)
        dy = s["dy"].float()
        da, db = dy * b * slope, dy * f
        dx = torch.matmul(da, wg) + torch.matmul(db, wu)
        return dx.to(ty), torch.matmul(da.T, x).to(ty), torch.matmul(db.T, x).to(ty)
    h, w = s["h"].float(), s["w"].float()
    live = s["target"] >= 0
    at = s["target"].clamp(min=0)[:, None]
    z = torch.matmul(h, w.T)
    if kind == "loss":
        lse = _plain_lse(z)
        loss = torch.where(live, lse - torch.gather(z, 1, at)[:, 0], torch.zeros_like(lse))
        return _plain_reduce(loss, live, case["reduction"]), torch.where(live, lse, torch.zeros_like(lse))
    up = s["up"] / live.sum().clamp(min=1) if case["reduction"] == "mean" else s["up"]
    up = torch.where(live, up.expand(len(h)), torch.zeros_like(s["lse"]))[:, None]
    g = torch.exp(z - s["lse"][:, None])
    g = g.scatter_add(1, at, torch.full_like(up, -1.0)) * up
    return torch.matmul(g, w).to(ty), torch.matmul(g.T, h).to(ty)


# ---------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "embed":
        return torch.index_select(s["table"].double(), 0, s["tokens"]) * case["scale"]
    if kind == "dembed":
        # sorted by token: running sums and their differences
        order = torch.argsort(s["tokens"], stable=True)
        ends = torch.cumsum(torch.bincount(s["tokens"], minlength=case["vocabulary"]), 0)
        total = torch.cumsum(s["dy"].double()[order], 0)
        total = torch.cat([torch.zeros_like(total[:1]), total])
        return (total[ends] - total[torch.cat([torch.zeros_like(ends[:1]), ends[:-1]])]) * case["scale"]
    if kind in ("gate", "dgate"):
        x, wg, wu = (s[n].double().requires_grad_(kind == "dgate") for n in ("x", "wg", "wu"))
        act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
               "gelu_tanh": lambda a: torch.nn.functional.gelu(a, approximate="tanh")}[case["activation"]]
        if kind == "gate":
            return act(x @ wg.T) * (x @ wu.T)
        total = [torch.zeros_like(wg), torch.zeros_like(wu)]
        dx = []
        for i in range(0, len(x), EPOCH):
            rows = x[i:i + EPOCH].detach().requires_grad_()
            y = act(rows @ wg.T) * (rows @ wu.T)
            g = torch.autograd.grad(y, (rows, wg, wu), s["dy"][i:i + EPOCH].double())
            dx.append(g[0])
            total = [t + u for t, u in zip(total, g[1:])]
        return torch.cat(dx), total[0].detach(), total[1].detach()
    h, w, target = s["h"].double(), s["w"].double(), s["target"]
    count = max(1, int((target != -100).sum()))
    losses, lses, dh, dw = [], [], [], torch.zeros_like(w)
    for i in range(0, len(h), EPOCH):
        rows, t = h[i:i + EPOCH], target[i:i + EPOCH]
        logp = torch.log_softmax(rows @ w.T, -1)
        if kind == "loss":
            losses.append(torch.nn.functional.nll_loss(logp, t, ignore_index=-100, reduction="none"))
            lses.append(torch.logsumexp(rows @ w.T, -1).masked_fill(t == -100, 0.0))
            continue
        p = logp.exp()
        known = torch.nonzero(t != -100)[:, 0]
        p[known, t[known]] -= 1.0
        p[t == -100] = 0.0
        up = s["up"].double()
        if case["reduction"] == "none":
            p *= up[i:i + EPOCH, None]
        else:
            p *= up / count if case["reduction"] == "mean" else up
        dh.append(p @ w)
        dw += p.T @ rows
    if kind == "dloss":
        return torch.cat(dh), dw
    loss = torch.cat(losses)
    if case["reduction"] != "none":
        loss = loss.sum() / (count if case["reduction"] == "mean" else 1)
    return loss, torch.cat(lses)


# -------------------------------------------------------------------- work

def work(case):
    def size(name):
        return 2 if case[name] == "bf16" else 4

    e, n, D = size("dtype"), case["tokens"], case["width"]
    kind = case["kind"]
    if kind in ("embed", "dembed"):
        V, t = case["vocabulary"], size("table")
        if kind == "embed":  # no row of the table is read twice, every output written
            return {"bytes": 8 * n + n * D * e + min(n, V) * D * t, "flops": n * D}
        # upstream gradients read, the table's gradient written
        return {"bytes": 8 * n + n * D * e + V * D * t, "flops": n * D}
    if kind in ("gate", "dgate"):
        F = case["inner"]
        if kind == "gate":  # two products
            return {"bytes": e * (n * D + 2 * F * D + n * F), "flops": 4 * n * D * F}
        # x, weights, upstream gradient read, three gradients written; two products replayed, four more
        return {"bytes": e * (2 * n * D + 4 * F * D + n * F), "flops": 12 * n * D * F}
    V, live = case["vocabulary"], int(n * (1 - case["ignored"]))  # the tokens that count
    if kind == "loss":
        return {"bytes": e * (live * D + V * D) + 16 * n, "flops": 2 * live * D * V}
    # the logits again, and a product for each gradient
    return {"bytes": e * (live * D + n * D + 2 * V * D) + 16 * n, "flops": 6 * live * D * V}
