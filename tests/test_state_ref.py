"""The 64-bit host forms the kernels are tested against, checked by themselves:
closed forms, and every gradient against central differences."""
import numpy as np
import pytest

from tests import state_ref as sr


def _inputs(T, H, Hk, Dk, Dv, seed=3):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, Hk, Dk)), r.standard_normal((T, Hk, Dk)),
            r.standard_normal((T, H, Dv)), r.standard_normal((T, H)),
            r.standard_normal((H, Dk, Dv)))


def test_open_gate_is_a_running_sum():
    q, k, v, _, s0 = _inputs(5, 2, 1, 3, 4)
    o, S = sr.scan(q, k, v, np.zeros((5, 2)), 0.5, "log", 0.0, s0)
    want = s0 + np.einsum("ti,thj->hij", k[:, 0], v)
    assert np.allclose(S[-1], want, rtol=1e-13)
    assert np.allclose(o[-1], 0.5 * np.einsum("i,hij->hj", q[-1, 0], want), rtol=1e-12)


def test_closed_gate_keeps_one_token():
    q, k, v, _, s0 = _inputs(4, 2, 2, 3, 4)
    o, S = sr.scan(q, k, v, np.full((4, 2), -np.inf), 1.0, "log", 0.0, s0)
    assert np.array_equal(S[-1], k[-1][:, :, None] * v[-1][:, None, :])


@pytest.mark.parametrize("form", ["sigmoid", "log"])
def test_scan_gradients_against_differences(form):
    T, H, Hk, Dk, Dv, scale, shift = 4, 4, 2, 3, 2, 0.7, 0.3
    q, k, v, a, s0 = _inputs(T, H, Hk, Dk, Dv)
    a = a if form == "sigmoid" else -np.abs(a) - 0.5
    r = np.random.default_rng(8)
    do, dsT = r.standard_normal(v.shape), r.standard_normal(s0.shape)

    def loss(q, k, v, a, s0):
        o, S = sr.scan(q, k, v, a, scale, form, shift, s0)
        return np.sum(o * do) + np.sum(S[-1] * dsT)

    got = sr.scan_grad(q, k, v, a, do, scale, form, shift, s0, dsT)
    x = [q, k, v, a, s0]
    for n, g in enumerate(got):
        for i in np.ndindex(g.shape):
            e = 1e-5
            lo, hi = [y.copy() for y in x], [y.copy() for y in x]
            lo[n][i] -= e
            hi[n][i] += e
            d = (loss(*hi) - loss(*lo)) / (2 * e)
            assert abs(d - g[i]) <= 1e-8 * (1 + abs(g[i])) * 10, (n, i)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_gradients_against_differences(layout):
    r = np.random.default_rng(4)
    x, dy, w = r.standard_normal((3, 2, 8)), r.standard_normal((3, 2, 8)), r.standard_normal(8)
    pos, freq, eps, m = np.array([0, 5, 1000]), np.array([1.0, 0.3]), 1e-3, 1.3

    def loss(x, w):
        return np.sum(sr.norm_rope(x, w, pos, freq, eps, layout, m) * dy)

    dx, dw = sr.norm_rope_grad(x, w, pos, freq, dy, eps, layout, m)
    for n, g in enumerate((dx, dw)):
        for i in np.ndindex(g.shape):
            e = 1e-5
            lo, hi = [x.copy(), w.copy()], [x.copy(), w.copy()]
            lo[n][i] -= e
            hi[n][i] += e
            d = (loss(*hi) - loss(*lo)) / (2 * e)
            assert abs(d - g[i]) <= 1e-7 * (1 + abs(g[i])), (n, i)


def test_rotation_keeps_length_and_position_zero():
    r = np.random.default_rng(4)
    y = r.standard_normal((2, 3, 16))
    for layout in ("half", "interleaved"):
        z = sr.turn(y, np.array([0, 77]), np.array([1.0, 0.1, 0.01]), layout)
        assert np.allclose(z[0], y[0], rtol=1e-15)
        assert np.allclose((z ** 2).sum(-1), (y ** 2).sum(-1), rtol=1e-12)
        assert np.array_equal(z[..., 6:], y[..., 6:])
