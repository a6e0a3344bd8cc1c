"""Plain 64-bit forms of the matrix-state scan and the query/key norm with
rotation, token by token and row by row (numpy, host), for the tests of the
kernels.  Nothing here is shared with the package."""
import numpy as np


def gates(a, form, shift):
    x = np.asarray(a, np.float64) + shift
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x)) if form == "sigmoid" else np.exp(x)


def scan(q, k, v, a, scale=1.0, form="sigmoid", shift=0.0, s0=None):
    """One sequence: q, k [T, Hk, Dk], v [T, H, Dv], a [T, H] -> out [T, H, Dv],
    states [T + 1, H, Dk, Dv] (the first is the initial one)."""
    T, H, Dv = v.shape
    Hk, Dk = q.shape[1:]
    g = gates(a, form, shift)
    q, k = np.repeat(q, H // Hk, 1), np.repeat(k, H // Hk, 1)
    S = np.zeros((T + 1, H, Dk, Dv))
    if s0 is not None:
        S[0] = s0
    o = np.zeros((T, H, Dv))
    for t in range(T):
        S[t + 1] = g[t][:, None, None] * S[t] + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * np.matmul(q[t][:, None, :], S[t + 1])[:, 0]
    return o, S


def scan_grad(q, k, v, a, do, scale=1.0, form="sigmoid", shift=0.0, s0=None, dsT=None):
    """Gradients of one sequence by the reverse recurrence: dq, dk, dv, da, ds0."""
    T, H, Dv = v.shape
    Hk, Dk = q.shape[1:]
    r = H // Hk
    _, S = scan(q, k, v, a, scale, form, shift, s0)
    g = gates(a, form, shift)
    qh, kh = np.repeat(q, r, 1), np.repeat(k, r, 1)
    dS = np.zeros((H, Dk, Dv)) if dsT is None else dsT.astype(np.float64).copy()
    dq, dk, dv, da = np.zeros(qh.shape), np.zeros(kh.shape), np.zeros(v.shape), np.zeros(a.shape)
    for t in range(T - 1, -1, -1):
        dS = dS + scale * qh[t][:, :, None] * do[t][:, None, :]
        dq[t] = scale * np.matmul(S[t + 1], do[t][:, :, None])[:, :, 0]
        dk[t] = np.matmul(dS, v[t][:, :, None])[:, :, 0]
        dv[t] = np.matmul(kh[t][:, None, :], dS)[:, 0]
        dg = np.sum(S[t] * dS, (1, 2))
        # dg/da: g (1 - g) or g
        da[t] = dg * g[t] * (gates(-(np.asarray(a[t], np.float64) + shift), "sigmoid", 0.0)
                             if form == "sigmoid" else 1.0)
        dS = g[t][:, None, None] * dS
    shared = (T, Hk, r, Dk)
    return dq.reshape(shared).sum(2), dk.reshape(shared).sum(2), dv, da, dS


def turn(y, pos, freq, layout, magnitude=1.0):
    """Rows [tokens, heads, D], each pair as a complex number times m e^{i angle}."""
    rot = 2 * len(freq)
    z = magnitude * np.exp(1j * np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64))[:, None]
    out = np.array(y, np.float64)
    if layout == "half":
        w = (out[..., :rot // 2] + 1j * out[..., rot // 2:rot]) * z
        out[..., :rot // 2], out[..., rot // 2:rot] = w.real, w.imag
    else:
        w = (out[..., 0:rot:2] + 1j * out[..., 1:rot:2]) * z
        out[..., 0:rot:2], out[..., 1:rot:2] = w.real, w.imag
    return out


def norm_rope(x, w, pos, freq, eps, layout, magnitude=1.0):
    x = np.asarray(x, np.float64)
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w
    return turn(y, pos, freq, layout, magnitude)


def norm_rope_grad(x, w, pos, freq, dy, eps, layout, magnitude=1.0):
    """(dx, dw): the rotation's transpose turns back by the same angle."""
    x = np.asarray(x, np.float64)
    g = turn(np.asarray(dy, np.float64), -np.asarray(pos, np.float64), freq, layout, magnitude)
    s = np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n = x / s
    gw = g * w
    return (gw - n * np.mean(gw * n, -1, keepdims=True)) / s, np.sum(g * n, (0, 1))
