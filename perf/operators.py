"""Measured cases of the matrix-state scan, its single-token step, and the
query/key norm with rotation: inputs, plain forms in elementary torch
operations, the definitions in 64 bits, and the work each pass cannot do
without.

A case is a dict with a "kind":
  scan   state_scan_forward: outputs per token and the final states
  grad   state_scan_backward: gradients of every input
  step   state_scan_step: one token per request over a pool of states
  norm   qk_norm_rope_forward
  dnorm  qk_norm_rope_backward
"""
import math

import torch

own = False

CHUNK = 64  # tokens per chunk of the plain scan


# ------------------------------------------------------------------- cases

def _scan(kind, name, dtype, lens, H, Hk, Dk, Dv, packed, state, gate="sigmoid"):
    c = {"kind": kind, "dtype": dtype, "lens": ",".join(map(str, lens)), "H": H, "Hk": Hk,
         "Dk": Dk, "Dv": Dv, "packed": packed, "state": state, "gate": gate}
    return dict(c, name=name) if name else c


def _step(name, dtype, N, pool, H, Hk, Dk, Dv):
    c = {"kind": "step", "dtype": dtype, "N": N, "pool": pool, "H": H, "Hk": Hk, "Dk": Dk, "Dv": Dv}
    return dict(c, name=name) if name else c


def _norm(kind, name, dtype, tokens, Hq, Hk, D, rot, layout, far):
    c = {"kind": kind, "dtype": dtype, "tokens": tokens, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot,
         "layout": layout, "far": far}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short prompt of one request: latency counts
        _scan("scan", "scan_prompt_bf16", "bf16", [77], 8, 8, 64, 64, False, False),
        # the forward of a training step: a batch of equal sequences, one head width twice the other
        _scan("scan", "scan_batch_bf16", "bf16", [2048] * 8, 16, 16, 64, 128, False, False),
        # one long document, few heads, keys shared by groups of heads: the length has to be split
        _scan("scan", "scan_long_bf16", "bf16", [32771], 16, 4, 128, 64, False, True),
        # requests of mixed length packed together, an empty and a one-token one among them, widths
        # that are no power of two, states continued from an earlier part
        _scan("scan", "scan_packed_f32", "f32", [613, 1, 0, 1024, 45, 380, 64, 129, 700, 2, 991, 257],
              12, 4, 96, 80, True, True),
        # gradients of a small layer
        _scan("grad", "grad_small_f32", "f32", [129] * 2, 4, 4, 32, 48, False, False),
        # gradients of the training step above
        _scan("grad", "grad_batch_bf16", "bf16", [2048] * 8, 16, 16, 64, 128, False, False),
        # gradients over packed sequences with shared keys, a carried state and log decays
        _scan("grad", "grad_packed_bf16", "bf16", [4096, 1500, 37, 2600, 1, 0, 1999, 5000], 16, 4, 128, 64,
              True, True, "log"),
        # one request generates one token
        _step("step_one_bf16", "bf16", 1, 4, 16, 16, 64, 64),
        # a full serving batch, its states scattered over the pool
        _step("step_many_bf16", "bf16", 250, 320, 32, 8, 128, 64),
        # the norm and rotation of one generated token, far into a long context
        _norm("norm", "norm_one_bf16", "bf16", 1, 16, 4, 128, 128, "half", True),
        # ... and of a training batch, a part of the head rotated
        _norm("norm", "norm_batch_bf16", "bf16", 16384, 32, 8, 128, 64, "interleaved", False),
        # its gradients, float32, an odd width
        _norm("dnorm", "dnorm_batch_f32", "f32", 8191, 16, 16, 80, 48, "half", False),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + (n % 1024 == 0)  # hardly ever a round size


def _lens(rng, top):
    total = _log_int(rng, 33, top)
    n = min(total, _log_int(rng, 1, 24))
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        case = _any(rng)
        if _cost(case) <= top:
            return case


def _any(rng):
    kind = rng.choice(["scan", "scan", "grad", "grad", "step", "norm", "dnorm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("scan", "grad"):
        Hk = rng.choice([1, 2, 4, 5, 8])
        H = Hk * rng.choice([1, 1, 2, 3])
        Dk, Dv = rng.choice([16, 32, 48, 64, 96, 128]), rng.choice([16, 40, 64, 80, 128])
        packed = rng.random() < 0.5
        top = (24000 if kind == "scan" else 12000) * 16 // max(16, H)
        if packed:
            lens = _lens(rng, top)
        else:
            T = _log_int(rng, 17, top)
            lens = [T] * rng.randrange(1, max(2, min(8, top // T) + 1))
        return _scan(kind, None, dtype, lens, H, Hk, Dk, Dv, packed, rng.random() < 0.5,
                     rng.choice(["sigmoid", "sigmoid", "log"]))
    if kind == "step":
        Hk = rng.choice([1, 2, 4, 8])
        N = _log_int(rng, 1, 200)
        return _step(None, dtype, N, N + rng.randrange(0, 40), Hk * rng.choice([1, 2, 4]), Hk,
                     rng.choice([32, 64, 96, 128]), rng.choice([32, 64, 80, 128]))
    D = rng.choice([32, 64, 80, 96, 128, 256])
    rot = rng.choice([D, D, D // 2])
    Hk = rng.choice([1, 2, 4, 8])
    return _norm(kind, None, dtype, _log_int(rng, 1, 8192), Hk * rng.choice([1, 2, 4]), Hk, D,
                 rot, rng.choice(["half", "interleaved"]), rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _lengths(case):
    return [int(x) for x in case["lens"].split(",")]


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _rows(lens, dev):
    """(Tp, row of each packed token among the sequences padded to Tp tokens, whole chunks)."""
    n = torch.tensor(lens, device=dev)
    start = torch.cumsum(n, 0) - n
    Tp = max(1, -(-max(lens) // CHUNK)) * CHUNK
    seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), n)
    return Tp, seq * Tp + torch.arange(sum(lens), device=dev) - start[seq]


def _unit(x):
    """Rows of mean square 1, as the norm of queries and keys leaves them."""
    return x * torch.rsqrt(torch.mean(x * x, -1, keepdim=True) + 1e-6)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ty = _type(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": case}
    if case["kind"] in ("scan", "grad"):
        lens = _lengths(case)
        N, total = len(lens), sum(lens)
        H, Hk, Dk, Dv = case["H"], case["Hk"], case["Dk"], case["Dv"]
        s["scale"] = Dk ** -0.5
        q, k = _unit(normal(total, Hk, Dk)).to(ty), _unit(normal(total, Hk, Dk)).to(ty)
        v = normal(total, H, Dv).to(ty)
        # heads that forget within a few tokens beside heads that remember over a thousand
        a = normal(total, H) + torch.linspace(0.5, 7.0, H, device=dev)
        if case["gate"] == "log":
            a = -torch.log1p(torch.exp(-a))
        a = a.to(ty)
        s["N"] = N
        s["Tp"], s["rows"] = _rows(lens, dev)
        if case["packed"]:
            off = [0]
            for n in lens:
                off.append(off[-1] + n)
            s["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev)
            lead = (total,)
        else:
            s["offsets"] = None
            lead = (N, lens[0])
        s["q"], s["k"] = q.view(*lead, Hk, Dk), k.view(*lead, Hk, Dk)
        s["v"], s["a"] = v.view(*lead, H, Dv), a.view(*lead, H)
        s["S0"] = normal(N, H, Dk, Dv) if case["state"] else None
        if case["kind"] == "grad":
            s["do"] = normal(total, H, Dv).to(ty).view(*lead, H, Dv)
            s["dS"] = normal(N, H, Dk, Dv) if case["state"] else None
    elif case["kind"] == "step":
        N, H, Hk, Dk, Dv = case["N"], case["H"], case["Hk"], case["Dk"], case["Dv"]
        s["scale"] = Dk ** -0.5
        s["q"], s["k"] = _unit(normal(N, Hk, Dk)).to(ty), _unit(normal(N, Hk, Dk)).to(ty)
        s["v"] = normal(N, H, Dv).to(ty)
        s["a"] = (normal(N, H) + torch.linspace(0.5, 7.0, H, device=dev)).to(ty)
        s["pool"] = normal(case["pool"], H, Dk, Dv)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device=dev)[:N].to(torch.int32)
    else:
        n, D, rot = case["tokens"], case["D"], case["rot"]
        # queries and keys are slices of one projection's output
        both = normal(n, case["Hq"] + case["Hk"], D).to(ty)
        s["q"], s["k"] = both[:, :case["Hq"]], both[:, case["Hq"]:]
        s["wq"], s["wk"] = 1 + 0.2 * normal(D), 1 + 0.2 * normal(D)
        s["freq"] = torch.exp(torch.arange(0, rot, 2, device=dev) * (-math.log(10000.0) / rot))
        s["pos"] = torch.arange(n, device=dev) + (1000003 if case["far"] else 0)
        if case["kind"] == "dnorm":
            s["dq"], s["dk"] = normal(n, case["Hq"], D).to(ty), normal(n, case["Hk"], D).to(ty)
    return s


# -------------------------------------------------------------- plain forms

def _log_gate(a, form):
    return -torch.log1p(torch.exp(-a)) if form == "sigmoid" else a


def _plain_scan(q, k, v, a, S0, N, Tp, rows, scale, form):
    """Outputs [tokens, H, Dv] and final states in 32 bits: chunks of tokens as
    products, the chunks' states joined by one product with their decays (sums of
    log gates and their differences in 64 bits)."""
    nc, H, Hk, Dk, Dv = Tp // CHUNK, v.shape[-2], q.shape[-2], q.shape[-1], v.shape[-1]

    def chunks(x, reps):
        x = x.new_zeros(N * Tp, *x.shape[1:]).index_copy(0, rows, x)
        x = x.reshape(N, nc, CHUNK, *x.shape[1:]).transpose(2, 3)         # [N, nc, heads, C, ...]
        return x.repeat_interleave(reps, 2) if reps > 1 else x

    qc, kc, vc = chunks(q, H // Hk), chunks(k, H // Hk), chunks(v, 1)
    L = torch.cumsum(chunks(_log_gate(a.double(), form), 1), -1)          # [N, nc, H, C]
    later = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).triu(1)
    D = torch.exp((L[..., :, None] - L[..., None, :]).masked_fill(later, -math.inf)).float()
    inner = torch.matmul(torch.matmul(qc, kc.transpose(-1, -2)) * D, vc)
    end = L[..., -1:]
    U = torch.matmul((kc * torch.exp(end - L).float()[..., None]).transpose(-1, -2), vc)
    first = torch.zeros_like(U[:, :1]) if S0 is None else S0[:, None]
    U = torch.cat([first, U], 1).transpose(1, 2).reshape(N, H, nc + 1, Dk * Dv)
    E = torch.cat([torch.zeros_like(end[:, :1]), torch.cumsum(end, 1)], 1)[..., 0].transpose(1, 2)
    later = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=q.device).triu(1)
    M = torch.exp((E[..., :, None] - E[..., None, :]).masked_fill(later, -math.inf)).float()
    S = torch.matmul(M, U).reshape(N, H, nc + 1, Dk, Dv)
    outer = torch.matmul(qc * torch.exp(L).float()[..., None], S[:, :, :-1].transpose(1, 2))
    o = (scale * (inner + outer)).transpose(2, 3).reshape(N * Tp, H, Dv)
    return o[rows], S[:, :, -1]


def _flat(x, case):
    return x if case["packed"] else x.reshape(-1, *x.shape[2:])


def _plain_rotate(y, pos, freq, layout):
    rot = 2 * freq.shape[0]
    angle = pos.double()[:, None] * freq.double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if layout == "half":
        x1, x2 = y[..., :rot // 2], y[..., rot // 2:rot]
        return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, y[..., rot:]], -1)
    x1, x2 = y[..., 0:rot:2], y[..., 1:rot:2]
    turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    return torch.cat([turned.reshape(*y.shape[:-1], rot), y[..., rot:]], -1)


def _plain_norm(x, w, s):
    x = x.float()
    y = x * torch.rsqrt(torch.mean(x * x, -1, keepdim=True) + 1e-6) * w
    return _plain_rotate(y, s["pos"], s["freq"], s["case"]["layout"])


def _plain_norm_grad(x, w, dy, s):
    x = x.float()
    g = _plain_rotate(dy.float(), -s["pos"], s["freq"], s["case"]["layout"])
    r = torch.rsqrt(torch.mean(x * x, -1, keepdim=True) + 1e-6)
    gw = g * w
    dx = r * gw - x * (r * r * r) * torch.mean(gw * x, -1, keepdim=True)
    return dx, torch.sum(g * x * r, (0, 1))


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import gated_linear_recurrence_history_amd as gs
        if kind == "scan":
            return gs.state_scan_forward(s["q"], s["k"], s["v"], s["a"], scale=s["scale"],
                                         gate_form=case["gate"], seq_offsets=s["offsets"],
                                         initial_state=s["S0"], final_state=True)
        if kind == "grad":
            d = gs.state_scan_backward(s["q"], s["k"], s["v"], s["a"], s["do"], scale=s["scale"],
                                       gate_form=case["gate"], seq_offsets=s["offsets"],
                                       initial_state=s["S0"], d_final_state=s["dS"])
            return d if s["S0"] is not None else d[:4]
        if kind == "step":
            return gs.state_scan_step(s["q"], s["k"], s["v"], s["a"], s["pool"], slots=s["slots"],
                                      scale=s["scale"]), s["pool"]
        if kind == "norm":
            return gs.qk_norm_rope_forward(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"],
                                           eps=1e-6, layout=case["layout"])
        return gs.qk_norm_rope_backward(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], s["dq"],
                                        s["dk"], eps=1e-6, layout=case["layout"])

    ty = _type(case)
    if kind == "scan":
        o, S = _plain_scan(_flat(s["q"], case).float(), _flat(s["k"], case).float(),
                           _flat(s["v"], case).float(), _flat(s["a"], case), s["S0"], s["N"], s["Tp"],
                           s["rows"], s["scale"], case["gate"])
        return o.reshape(s["v"].shape).to(ty), S
    if kind == "grad":
        leaves = [_flat(s[n], case).float().requires_grad_() for n in ("q", "k", "v", "a")]
        ends = [] if s["S0"] is None else [s["S0"].clone().requires_grad_()]
        o, S = _plain_scan(*leaves, ends[0] if ends else None, s["N"], s["Tp"], s["rows"], s["scale"],
                           case["gate"])
        tops, ups = [o], [_flat(s["do"], case).float()]
        if ends:
            tops, ups = tops + [S], ups + [s["dS"]]
        g = torch.autograd.grad(tops, leaves + ends, ups)
        return tuple(x.reshape(s[n].shape).to(ty) for x, n in zip(g, ("q", "k", "v", "a"))) + tuple(g[4:])
    if kind == "step":
        reps = case["H"] // case["Hk"]
        q, k = (s[n].float().repeat_interleave(reps, 1) for n in ("q", "k"))
        i = s["slots"].long()
        S = s["pool"][i] * torch.sigmoid(s["a"].float())[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
        s["pool"][i] = S
        return (s["scale"] * torch.sum(S * q[..., None], -2)).to(ty), s["pool"]
    if kind == "norm":
        return _plain_norm(s["q"], s["wq"], s).to(ty), _plain_norm(s["k"], s["wk"], s).to(ty)
    dq, dwq = _plain_norm_grad(s["q"], s["wq"], s["dq"], s)
    dk, dwk = _plain_norm_grad(s["k"], s["wk"], s["dk"], s)
    return dq.to(ty), dk.to(ty), dwq, dwk


# ---------------------------------------------------- definitions in 64 bits

def _exact_scan(s, case):
    """The recurrence token by token; with "do" the gradients, from the running
    state forwards and its gradient backwards."""
    lens = _lengths(case)
    N, total, reps, form = len(lens), sum(lens), case["H"] // case["Hk"], case["gate"]
    H, Dk, Dv = case["H"], case["Dk"], case["Dv"]
    dev = s["q"].device
    T = max(lens)

    def steps(x, reps=1):  # [T, N, H, ...]
        x = x.double().reshape(total, *x.shape[1 if case["packed"] else 2:])
        ends = torch.split(x, lens)
        x = torch.stack([torch.cat([y, y.new_zeros(T - len(y), *y.shape[1:])]) for y in ends], 1)
        return x.repeat_interleave(reps, 2) if reps > 1 else x

    def tokens(x):
        return torch.cat([x[:n, i] for i, n in enumerate(lens)])

    q, k, v, a = steps(s["q"], reps), steps(s["k"], reps), steps(s["v"]), steps(s["a"])
    g = torch.sigmoid(a) if form == "sigmoid" else torch.exp(a)
    live = torch.arange(T, device=dev)[:, None] < torch.tensor(lens, device=dev)
    g = torch.where(live[..., None], g, torch.ones_like(g))  # past its end a sequence rests
    S = torch.zeros(N, H, Dk, Dv, dtype=torch.float64, device=dev) if s["S0"] is None else s["S0"].double()
    o = torch.zeros_like(v)
    do = steps(s["do"]) if "do" in s else None
    dq = torch.zeros_like(q)
    for t in range(T):
        S = S * g[t][..., None, None] + k[t][..., None] * v[t][..., None, :]
        o[t] = s["scale"] * torch.matmul(q[t][..., None, :], S)[..., 0, :]
        if do is not None:
            dq[t] = s["scale"] * torch.matmul(S, do[t][..., None])[..., 0]
    if do is None:
        return tokens(o).reshape(s["v"].shape), S
    dS = torch.zeros_like(S) if s["dS"] is None else s["dS"].double()
    F = torch.sum(S * dS, (-1, -2))  # <S_t, dS_t>, before what the output adds
    dk, dv, da = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(a)
    for t in range(T - 1, -1, -1):
        dS = dS + s["scale"] * q[t][..., None] * do[t][..., None, :]
        dk[t] = torch.matmul(dS, v[t][..., None])[..., 0]
        dv[t] = torch.matmul(k[t][..., None, :], dS)[..., 0, :]
        F = F + torch.sum(q[t] * dq[t], -1) - torch.sum(k[t] * dk[t], -1)
        da[t] = F
        dS = dS * g[t][..., None, None]
    if form == "sigmoid":
        da = da * (1 - g)

    def group(x):
        return x.reshape(*x.shape[:2], case["Hk"], reps, Dk).sum(3)

    out = [tokens(x).reshape(s[n].shape) for x, n in ((group(dq), "q"), (group(dk), "k"), (dv, "v"), (da, "a"))]
    return tuple(out) + (() if s["S0"] is None else (dS,))


def _exact_turn(x, s, sign):
    """Each rotated pair as a complex number times e^{i angle}."""
    rot = 2 * s["freq"].shape[0]
    angle = sign * s["pos"].double()[:, None] * s["freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    y = x.clone()
    if s["case"]["layout"] == "half":
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("scan", "grad"):
        return _exact_scan(s, case)
    if kind == "step":
        reps = case["H"] // case["Hk"]
        pool, o = s["pool"].double(), []
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        for n in range(case["N"]):
            kn, qn = k[n].repeat_interleave(reps, 0), q[n].repeat_interleave(reps, 0)
            g = 1 / (1 + torch.exp(-s["a"][n].double()))
            i = int(s["slots"][n])
            pool[i] = g[:, None, None] * pool[i] + torch.einsum("hd,he->hde", kn, v[n])
            o.append(s["scale"] * torch.einsum("hd,hde->he", qn, pool[i]))
        return torch.stack(o), pool
    out, dw = [], []
    for x, w, dy in (("q", "wq", "dq"), ("k", "wk", "dk")):
        x, w = s[x].double(), s[w].double()
        rms = torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
        if kind == "norm":
            out.append(_exact_turn(x / rms * w, s, 1))
        else:
            g = _exact_turn(s[dy].double(), s, -1)
            n = x / rms
            out.append((g * w - n * (g * w * n).mean(-1, keepdim=True)) / rms)
            dw.append((g * n).sum(0).sum(0))
    return tuple(out + dw)


# -------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if kind in ("scan", "grad"):
        lens = _lengths(case)
        n, H, Hk, Dk, Dv = sum(lens), case["H"], case["Hk"], case["Dk"], case["Dv"]
        states = len(lens) * H * Dk * Dv * 4
        if kind == "scan":
            # q, k, v, gates read and outputs written; final states written, initial ones read
            return {"bytes": n * e * (2 * Hk * Dk + 2 * H * Dv + H) + states * (2 if case["state"] else 1),
                    "flops": 4 * n * H * Dk * Dv}  # the update and the read-out
        # the same and the upstream gradient read, four gradients written; with states: S0, dS_T, dS0
        return {"bytes": n * e * (4 * Hk * Dk + 3 * H * Dv + 2 * H) + states * (3 if case["state"] else 0),
                "flops": 10 * n * H * Dk * Dv}  # both running states, dq, dk, dv
    if kind == "step":
        n, H, Hk, Dk, Dv = case["N"], case["H"], case["Hk"], case["Dk"], case["Dv"]
        return {"bytes": 2 * n * H * Dk * Dv * 4 + n * e * (2 * Hk * Dk + 2 * H * Dv + H),
                "flops": 5 * n * H * Dk * Dv}
    rows, D = case["tokens"] * (case["Hq"] + case["Hk"]), case["D"]
    if kind == "norm":
        return {"bytes": 2 * rows * D * e, "flops": 7 * rows * D}
    return {"bytes": 3 * rows * D * e, "flops": 14 * rows * D}
