"""Operands whose rows lie on no multiple of 16 bytes: the differentiable calls
and the step copy them, and give the same bits as for dense ones; the example's
layer has such rows when its heads are no multiple of 8."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests.test_gpu_mixing_example import example  # noqa: F401  (a fixture)
from tests.test_gpu_state_scan import BF, DEV, F32

pytestmark = pytest.mark.gpu


def rows(x, pad):
    """The same values as a slice of rows `pad` elements longer."""
    wide = torch.zeros(*x.shape[:-2], x.shape[-2] * x.shape[-1] + pad, dtype=x.dtype, device=DEV)
    part = wide[..., :x.shape[-2] * x.shape[-1]].unflatten(-1, x.shape[-2:])
    part.copy_(x)
    return part


@pytest.mark.parametrize("dtype,pad", [(BF, 4), (BF, 1), (F32, 2)])
def test_same_bits_as_dense(dtype, pad):
    r = torch.Generator(device=DEV).manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=r, device=DEV).to(dtype)  # noqa: E731
    T, H, Hk, Dk, Dv = 70, 4, 2, 32, 40
    q, k, v, a, do = n(T, Hk, Dk), n(T, Hk, Dk), n(T, H, Dv), n(T, H), n(T, H, Dv)
    off = torch.tensor([0, 33, T], dtype=torch.int32, device=DEV)
    w, freq, pos = torch.ones(Dk, device=DEV), torch.ones(16, device=DEV), torch.arange(T, device=DEV)

    def run(ops):
        x = [t.detach().requires_grad_() for t in ops]
        qn, kn = gs.qk_norm_rope(x[0], x[1], w, w, pos, freq)
        out, fin = gs.state_scan(qn, kn, x[2], x[3], seq_offsets=off)
        out2, _ = gs.state_scan(x[0], x[1], x[2], x[3], seq_offsets=off)
        g = torch.autograd.grad([out, out2], x, [do, do])
        pool = torch.ones(T, H, Dk, Dv, device=DEV)
        return (out, out2, fin, *g, gs.state_scan_step(*ops, pool), pool)

    want = run([q, k, v, a])
    got = run([rows(q, pad), rows(k, pad), rows(v, pad), a])
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    # the step's copies are made on its stream
    pool = torch.ones(T, H, Dk, Dv, device=DEV)
    ops = [rows(q, pad), rows(k, pad), rows(v, pad), a]
    torch.cuda.synchronize()
    out = gs.state_scan_step(*ops, pool, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(out, want[-2]) and torch.equal(pool, want[-1])


def test_the_calls_under_state_scan_refuse():
    x = rows(torch.ones(9, 2, 32, dtype=BF, device=DEV), 4)
    a = torch.zeros(9, 2, device=DEV)
    off = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    with pytest.raises(gs.GScanError, match="16 bytes"):
        gs.state_scan_forward(x, x, x, a, seq_offsets=off)
    with pytest.raises(gs.GScanError, match="16 bytes"):
        gs.qk_norm_rope_forward(x, None, None, None, None, None)


@pytest.mark.parametrize("heads,key_heads", [(4, 2), (12, 4), (3, 1)])
def test_example_layer_of_any_heads_in_bfloat16(example, heads, key_heads):  # noqa: F811
    torch.manual_seed(7)
    layer = example.MixingLayer(128, heads=heads, key_heads=key_heads, key_width=32, value_width=40)
    off, pos = example.pack([37, 1, 30])
    x = torch.randn(68, 128, device=DEV)
    with torch.autocast("cuda", torch.bfloat16):
        y, state = layer(x, pos, off)
        y.float().square().sum().backward()
        assert all(bool(p.grad.abs().sum() > 0) for p in layer.parameters())
        pool = state.detach().clone()
        slots = torch.arange(3, dtype=torch.int32, device=DEV)
        z = layer.step(x[:3], torch.tensor([37, 1, 30], device=DEV), pool, slots)
    assert bool(torch.isfinite(z).all()) and not torch.equal(pool, state)
