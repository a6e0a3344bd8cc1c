"""Gated projection, the first half of a feed-forward block (include/gscan.h,
gscan_gated_projection_forward):

    out = act(x w_gate^T) * (x w_up^T)

in one kernel that keeps both products in registers.  `gated_projection` is
differentiable; `gated_projection_forward` / `_backward` are the calls under
it.  Argument marshalling only.

x [..., width], w_gate, w_up [inner, width] (as torch.nn.Linear keeps them; both
may be halves of one matrix), one type, float32 or bfloat16; width and inner
are multiples of 8 up to 65536.  Rows may lie any multiple of 16 bytes up to
2^21 elements apart.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .embedding import _device_of, _row_stride, _type_code
from .matrix_state import _check_dense, _On, _on_device, _ptr, _readable, _workspace

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


class _Desc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("width", ctypes.c_int64), ("inner", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
                ("up_stride", ctypes.c_int64), ("d_out_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("activation", ctypes.c_int)]


def _describe(x, w_gate, w_up, activation):
    dev = _device_of(x, "x")
    _on_device(dev, w_gate=w_gate, w_up=w_up)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    if w_gate.dtype != x.dtype or w_up.dtype != x.dtype:
        raise TypeError(f"x and the weights must share a type; got {x.dtype}, {w_gate.dtype}, {w_up.dtype}")
    if x.dim() < 1 or w_gate.dim() != 2 or w_up.shape != w_gate.shape or w_gate.shape[1] != x.shape[-1]:
        raise ValueError("x must be [..., width], the weights [inner, width]; got "
                         f"{tuple(x.shape)}, {tuple(w_gate.shape)}, {tuple(w_up.shape)}")
    tokens = x.numel() // x.shape[-1] if x.shape[-1] else 0
    return _Desc(tokens, x.shape[-1], w_gate.shape[0], _row_stride(x, "x"), _row_stride(w_gate, "w_gate"),
                 _row_stride(w_up, "w_up"), 0, _type_code(x.dtype, "x"), ACTIVATIONS[activation])


def gated_projection_forward_workspace_bytes(x, w_gate, w_up) -> int:
    """Workspace of gated_projection_forward for these operands (0: none needed)."""
    d = _describe(x, w_gate, w_up, "silu")
    return int(binding.lib().gscan_gated_projection_forward_workspace_bytes(ctypes.byref(d)))


def gated_projection_backward_workspace_bytes(x, w_gate, w_up) -> int:
    """Workspace of gated_projection_backward for these operands."""
    d = _describe(x, w_gate, w_up, "silu")
    return int(binding.lib().gscan_gated_projection_backward_workspace_bytes(ctypes.byref(d)))


def gated_projection_forward(x, w_gate, w_up, activation: str = "silu", out=None, workspace=None,
                             stream=None):
    """act(x w_gate^T) * (x w_up^T), [..., inner] in the type of x.  `activation`:
    "silu", "gelu" or "gelu_tanh".

    `workspace` may be a uint8 device tensor of at least
    gated_projection_forward_workspace_bytes() bytes; otherwise one is taken from
    torch's caching allocator where needed.
    """
    d = _describe(x, w_gate, w_up, activation)
    dev, shape, L = x.device, (*x.shape[:-1], w_gate.shape[0]), binding.lib()
    need = int(L.gscan_gated_projection_forward_workspace_bytes(ctypes.byref(d)))
    if out is not None:
        _check_dense(out, shape, x.dtype, dev, "out")
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=dev)
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(L.gscan_gated_projection_forward(
            ctypes.byref(d), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), out.data_ptr(), wp, wn, s))
    return out


def gated_projection_backward(x, w_gate, w_up, d_out, activation: str = "silu", wanted=(True, True),
                              workspace=None, stream=None):
    """(dx, d_w_gate, d_w_up) in the operands' type.  `wanted`: whether the
    gradient of x, and those of the weights, are formed (None where not).

    `workspace` may be a uint8 device tensor of at least
    gated_projection_backward_workspace_bytes() bytes; otherwise one is taken
    from torch's caching allocator.
    """
    d = _describe(x, w_gate, w_up, activation)
    dev, L = x.device, binding.lib()
    _on_device(dev, d_out=d_out)
    if d_out.dtype != x.dtype or d_out.shape != (*x.shape[:-1], w_gate.shape[0]):
        raise ValueError(f"d_out must be {x.dtype} {(*x.shape[:-1], w_gate.shape[0])}; got {d_out.dtype} "
                         f"{tuple(d_out.shape)}")
    d.d_out_stride = _row_stride(d_out, "d_out")
    need = int(L.gscan_gated_projection_backward_workspace_bytes(ctypes.byref(d)))
    with _On(dev, stream) as s:
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if wanted[0] else None
        dg, du = (torch.empty(w_gate.shape, dtype=x.dtype, device=dev) if wanted[1] else None for _ in range(2))
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(L.gscan_gated_projection_backward(
            ctypes.byref(d), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), d_out.data_ptr(), _ptr(dx),
            _ptr(dg), _ptr(du), wp, wn, s))
    return dx, dg, du


def _rows(t):
    """t as the library reads it: copied where its rows lie on no multiple of 16
    bytes or at no single stride."""
    return _readable(t, t) if t.dim() == 2 else _readable(t.contiguous(), t)


class GatedProjectionFunction(torch.autograd.Function):
    """act(x w_gate^T) * (x w_up^T); the backward forms both products again from
    the saved operands."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation):
        x, w_gate, w_up = _rows(x), _rows(w_gate), _rows(w_up)
        ctx.save_for_backward(x, w_gate, w_up)
        ctx.activation = activation
        return gated_projection_forward(x, w_gate, w_up, activation)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        x, w_gate, w_up = ctx.saved_tensors
        need = ctx.needs_input_grad
        g = gated_projection_backward(x, w_gate, w_up, _rows(d_out.to(x.dtype)), ctx.activation,
                                      (need[0], need[1] or need[2]))
        return tuple(t if n else None for t, n in zip(g, need)) + (None,)


def gated_projection(x, w_gate, w_up, activation: str = "silu"):
    """Differentiable act(x w_gate^T) * (x w_up^T); see gated_projection_forward.
    Operands that the library cannot read as they are, are copied."""
    return GatedProjectionFunction.apply(x, w_gate, w_up, activation)
