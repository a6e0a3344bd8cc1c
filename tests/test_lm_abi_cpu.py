"""Refusals of the embedding, the gated projection and the cross entropy, and the
arithmetic of their workspaces (no GPU: every call here fails its checks before
anything is enqueued)."""
import ctypes
import os

import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from gated_linear_recurrence_history_amd import binding, cross_entropy, embedding, gated

OK, INVALID, UNSUPPORTED, MISALIGNED, WS_SMALL = 0, 1, 2, 3, 4
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from gated_linear_recurrence_history_amd import _build
        _build.build_hip()
    return binding.lib()


def embed_desc(tokens=7, vocabulary=100, width=64, stride=64, table_dtype=0, dtype=1, token_int64=1, scale=1.0):
    return embedding._Desc(tokens, vocabulary, width, stride, table_dtype, dtype, token_int64, scale)


def gate_desc(tokens=7, width=64, inner=48, x_stride=64, gate_stride=64, up_stride=64, d_out_stride=48, dtype=1,
              activation=0):
    return gated._Desc(tokens, width, inner, x_stride, gate_stride, up_stride, d_out_stride, dtype,
                       activation)


def loss_desc(tokens=7, width=64, vocabulary=101, h_stride=64, weight_stride=64, dtype=1, reduction=2,
              target_int64=1, scale=1.0):
    return cross_entropy._Desc(tokens, width, vocabulary, h_stride, weight_stride, dtype, reduction, target_int64,
                               scale)


SIZES = [(dict(tokens=-1), INVALID), (dict(width=0), INVALID), (dict(width=12), UNSUPPORTED),
         (dict(width=65544), UNSUPPORTED), (dict(tokens=2 ** 31), UNSUPPORTED), (dict(dtype=2), INVALID)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(vocabulary=0), INVALID), (dict(vocabulary=2 ** 31), UNSUPPORTED), (dict(table_dtype=-1), INVALID),
    (dict(vocabulary=2 ** 30, width=2048), UNSUPPORTED), (dict(stride=-8), INVALID),
    (dict(stride=66), MISALIGNED)])
def test_embed_sizes(lib, kw, code):
    d = embed_desc(**kw)
    assert lib.gscan_embed_forward(ctypes.byref(d), FAKE, FAKE, FAKE, None) == code
    assert lib.gscan_last_error() != b""
    if code != MISALIGNED:
        assert lib.gscan_embed_workspace_bytes(ctypes.byref(d)) == 0


@pytest.mark.parametrize("table,tokens,out,code", [
    (None, FAKE, FAKE, INVALID), (FAKE, None, FAKE, INVALID), (FAKE, FAKE, None, INVALID),
    (FAKE + 8, FAKE, FAKE, MISALIGNED), (FAKE, FAKE + 4, FAKE, MISALIGNED), (FAKE, FAKE, FAKE + 2, MISALIGNED)])
def test_embed_pointers(lib, table, tokens, out, code):
    d = embed_desc()
    assert lib.gscan_embed_forward(ctypes.byref(d), table, tokens, out, None) == code
    assert lib.gscan_embed_backward(ctypes.byref(d), table, tokens, out, None, 0, None) == code


def test_embed_workspace(lib):
    for n, v, w in [(1, 10, 8), (777, 1003, 200), (2048, 2 ** 20 - 1, 512), (64, 32000, 4096)]:  # added up at once
        assert lib.gscan_embed_workspace_bytes(ctypes.byref(embed_desc(tokens=n, vocabulary=v, width=w))) == 0
    for n, v, w in [(1, 2 ** 20, 8), (777, 1003, 520), (16384, 32000, 2048), (16385, 32000, 64), (2049, 2 ** 18, 8),
                    (65537, 300, 24), (2 ** 20, 50000, 128)]:
        d = embed_desc(tokens=n, vocabulary=v, width=w)
        need = lib.gscan_embed_workspace_bytes(ctypes.byref(d))
        # keys and positions, and two partial sums a chunk of at least eight tokens
        assert 8 * n <= need <= 16 * n + (n // 4 + 8) * w * 4 + 4096 + n
        assert lib.gscan_embed_backward(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, need - 1, None) == WS_SMALL
        assert lib.gscan_embed_backward(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE + 16, need, None) == MISALIGNED
    assert lib.gscan_embed_workspace_bytes(ctypes.byref(embed_desc(tokens=0))) == 0


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(inner=0), INVALID), (dict(inner=20), UNSUPPORTED), (dict(inner=65544), UNSUPPORTED),
    (dict(activation=3), INVALID), (dict(x_stride=-8), UNSUPPORTED), (dict(gate_stride=2 ** 21 + 8), UNSUPPORTED),
    (dict(up_stride=68), MISALIGNED), (dict(tokens=2 ** 28, width=65536), UNSUPPORTED)])
def test_gate_sizes(lib, kw, code):
    d = gate_desc(**kw)
    r = ctypes.byref(d)
    assert lib.gscan_gated_projection_forward(r, FAKE, FAKE, FAKE, FAKE, None, 0, None) == code
    assert lib.gscan_gated_projection_backward(r, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, None) == code
    assert lib.gscan_gated_projection_forward_workspace_bytes(r) == 0
    assert lib.gscan_gated_projection_backward_workspace_bytes(r) == 0


def test_gate_pointers(lib):
    r = ctypes.byref(gate_desc())
    good = [FAKE] * 7  # x, w_gate, w_up, d_out, dx, d_w_gate, d_w_up
    for i in (0, 1, 2, 3, 5, 6):
        args = list(good)
        args[i] = None  # one of the weights' gradients without the other, too
        assert lib.gscan_gated_projection_backward(r, *args, None, 0, None) == INVALID
    for i in range(7):
        args = list(good)
        args[i] = FAKE + 8
        assert lib.gscan_gated_projection_backward(r, *args, None, 0, None) == MISALIGNED
    bad = gate_desc(d_out_stride=2 ** 21 + 8)
    assert lib.gscan_gated_projection_backward(ctypes.byref(bad), *good, None, 0, None) == UNSUPPORTED
    assert lib.gscan_gated_projection_forward(r, FAKE, FAKE, FAKE, None, None, 0, None) == INVALID
    assert lib.gscan_gated_projection_forward(r, FAKE, FAKE, FAKE, FAKE + 4, None, 0, None) == MISALIGNED
    need = lib.gscan_gated_projection_backward_workspace_bytes(r)
    assert need >= 7 * 2 * 48 * 2
    assert lib.gscan_gated_projection_backward(r, *good, FAKE, need - 1, None) == WS_SMALL
    assert lib.gscan_gated_projection_backward(r, *good, FAKE + 64, need, None) == MISALIGNED


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(vocabulary=0), INVALID), (dict(vocabulary=2 ** 31), UNSUPPORTED), (dict(reduction=3), INVALID),
    (dict(h_stride=2 ** 21 + 8), UNSUPPORTED), (dict(weight_stride=-8), UNSUPPORTED),
    (dict(h_stride=65), MISALIGNED), (dict(tokens=2 ** 27, vocabulary=2 ** 20), UNSUPPORTED)])
def test_loss_sizes(lib, kw, code):
    r = ctypes.byref(loss_desc(**kw))
    assert lib.gscan_linear_cross_entropy_forward(r, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, None) == code
    assert lib.gscan_linear_cross_entropy_backward(r, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, None) == code
    assert lib.gscan_linear_cross_entropy_forward_workspace_bytes(r) == 0
    assert lib.gscan_linear_cross_entropy_backward_workspace_bytes(r) == 0


def test_loss_pointers(lib):
    r = ctypes.byref(loss_desc())
    for i in range(5):  # h, weight, target, loss / lse, lse / d_loss
        args = [FAKE] * 5
        args[i] = None
        assert lib.gscan_linear_cross_entropy_forward(r, *args, None, 0, None) == INVALID
        assert lib.gscan_linear_cross_entropy_backward(r, *args, FAKE, FAKE, None, 0, None) == INVALID
    for i, off in ((0, 8), (1, 8), (2, 4), (3, 2), (4, 2), (5, 8), (6, 8)):
        args = [FAKE] * 7
        args[i] += off
        assert lib.gscan_linear_cross_entropy_backward(r, *args, None, 0, None) == MISALIGNED
    need = lib.gscan_linear_cross_entropy_backward_workspace_bytes(r)
    assert lib.gscan_linear_cross_entropy_backward(r, *[FAKE] * 7, FAKE, need - 1, None) == WS_SMALL
    assert lib.gscan_linear_cross_entropy_backward(r, *[FAKE] * 7, FAKE + 32, need, None) == MISALIGNED


def test_loss_workspace_does_not_grow_with_the_vocabulary(lib):
    def need(f, **kw):
        return f(ctypes.byref(loss_desc(tokens=65536, width=1024, **kw)))

    b = lib.gscan_linear_cross_entropy_backward_workspace_bytes
    # gradients of the logits of a piece, sums of the tokens' gradients, a copy of their rows, parts of tiles
    assert need(b, vocabulary=2 ** 18) <= (512 + 256 + 128 + 256) * 2 ** 20
    assert need(b, vocabulary=2 ** 20) == need(b, vocabulary=2 ** 18)
    # the forward leaves a pair a tile of 128 of the vocabulary, at most
    f = lib.gscan_linear_cross_entropy_forward_workspace_bytes
    assert need(f, vocabulary=2 ** 18) <= 65536 * (2 ** 18 // 128) * 8 + (128 + 256 + 64) * 2 ** 20


def test_python_refusals():
    x, t = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        gs.embed_forward(x, t)
    with pytest.raises(TypeError):
        gs.embed_backward(x, t, 10)
    with pytest.raises(TypeError):
        gs.embed(None, t)
    with pytest.raises(TypeError):
        gs.gated_projection_forward(x, x, x)
    with pytest.raises(TypeError):
        gs.gated_projection_backward(x, x, x, x)
    with pytest.raises(TypeError):
        gs.linear_cross_entropy_forward(x, x, t)
    with pytest.raises(TypeError):
        gs.linear_cross_entropy_backward(x, x, t, t, t)
