"""Gated projection, the first half of a feed-forward block (include/gscan.h,
gscan_gated_projection_forward):

    out = act(x w_gate^T) * (x w_up^T)

in one kernel that keeps both products in registers.  `gated_projection` is
differentiable; `gated_projection_forward` / `_backward` are the calls under
it.  Argument marshalling only.

x [..., width], w_gate, w_up [inner, width] (as torch.nn.Linear keeps them; both
may be halves of one matrix), one type, float32 or bfloat16; width and inner
are multiples of 8 up to 65536.  Rows may lie any multiple of 16 bytes up to
2^21 elements apart; `gated_projection` copies operands and upstream gradients
whose rows are further apart.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .embedding import _device_of, _product_rows, _row_stride, _type_code
from .matrix_state import _check_dense, _layout, _On, _on_device, _ptr, _workspace

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


class _Desc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("width", ctypes.c_int64), ("inner", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
                ("up_stride", ctypes.c_int64), ("d_out_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("activation", ctypes.c_int)]


@functools.lru_cache(maxsize=256)
def _template(x, w_gate, w_up, dtypes, activation, d_out):
    """The descriptor of a call, as bytes; operands are (shape, stride), d_out None
    in the forward."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    if dtypes[1] != dtypes[0] or dtypes[2] != dtypes[0]:
        raise TypeError(f"x and the weights must share a type; got {dtypes[0]}, {dtypes[1]}, {dtypes[2]}")
    xs, gs, us = x[0], w_gate[0], w_up[0]
    if len(xs) < 1 or len(gs) != 2 or us != gs or gs[1] != xs[-1]:
        raise ValueError("x must be [..., width], the weights [inner, width]; got "
                         f"{tuple(xs)}, {tuple(gs)}, {tuple(us)}")
    d = _Desc(xs[:-1].numel(), xs[-1], gs[0], _row_stride(*x, "x"), _row_stride(*w_gate, "w_gate"),
              _row_stride(*w_up, "w_up"), 0, _type_code(dtypes[0], "x"), ACTIVATIONS[activation])
    if d_out is not None:
        if dtypes[3] != dtypes[0] or d_out[0] != (*xs[:-1], gs[0]):
            raise ValueError(f"d_out must be {dtypes[0]} {(*xs[:-1], gs[0])}; got {dtypes[3]} {tuple(d_out[0])}")
        d.d_out_stride = _row_stride(*d_out, "d_out")
    return bytes(d)


@functools.lru_cache(maxsize=256)
def _need(desc, backward):
    L = binding.lib()
    return int((L.gscan_gated_projection_backward_workspace_bytes if backward else
                L.gscan_gated_projection_forward_workspace_bytes)(desc))


def _describe(x, w_gate, w_up, activation, d_out=None):
    dev = _device_of(x, "x")
    _on_device(dev, w_gate=w_gate, w_up=w_up)
    if d_out is None:
        return _template(_layout(x), _layout(w_gate), _layout(w_up), (x.dtype, w_gate.dtype, w_up.dtype),
                         activation, None)
    _on_device(dev, d_out=d_out)
    return _template(_layout(x), _layout(w_gate), _layout(w_up),
                     (x.dtype, w_gate.dtype, w_up.dtype, d_out.dtype), activation, _layout(d_out))


def gated_projection_forward_workspace_bytes(x, w_gate, w_up) -> int:
    """Workspace of gated_projection_forward for these operands (0: none needed)."""
    return _need(_describe(x, w_gate, w_up, "silu"), False)


def gated_projection_backward_workspace_bytes(x, w_gate, w_up) -> int:
    """Workspace of gated_projection_backward for these operands."""
    return _need(_describe(x, w_gate, w_up, "silu"), True)


def gated_projection_forward(x, w_gate, w_up, activation: str = "silu", out=None, workspace=None,
                             stream=None):
    """act(x w_gate^T) * (x w_up^T), [..., inner] in the type of x.  `activation`:
    "silu", "gelu" or "gelu_tanh".

    `workspace` may be a uint8 device tensor of at least
    gated_projection_forward_workspace_bytes() bytes; otherwise one is taken from
    torch's caching allocator where needed.
    """
    d = _describe(x, w_gate, w_up, activation)
    dev, shape, need = x.device, (*x.shape[:-1], w_gate.shape[0]), _need(d, False)
    if out is not None:
        _check_dense(out, shape, x.dtype, dev, "out")
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=dev)
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(binding.lib().gscan_gated_projection_forward(
            d, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), out.data_ptr(), wp, wn, s))
    return out


def gated_projection_backward(x, w_gate, w_up, d_out, activation: str = "silu", wanted=(True, True),
                              workspace=None, stream=None):
    """(dx, d_w_gate, d_w_up) in the operands' type.  `wanted`: whether the
    gradient of x, and those of the weights, are formed (None where not).

    `workspace` may be a uint8 device tensor of at least
    gated_projection_backward_workspace_bytes() bytes; otherwise one is taken
    from torch's caching allocator.
    """
    if d_out is None:
        raise ValueError("d_out must be a tensor")
    d = _describe(x, w_gate, w_up, activation, d_out)
    dev, need = x.device, _need(d, True)
    with _On(dev, stream) as s:
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if wanted[0] else None
        dg, du = (torch.empty(w_gate.shape, dtype=x.dtype, device=dev) if wanted[1] else None for _ in range(2))
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(binding.lib().gscan_gated_projection_backward(
            d, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), d_out.data_ptr(), _ptr(dx), _ptr(dg),
            _ptr(du), wp, wn, s))
    return dx, dg, du


class GatedProjectionFunction(torch.autograd.Function):
    """act(x w_gate^T) * (x w_up^T); the backward forms both products again from
    the saved operands."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation):
        x, w_gate, w_up = _product_rows(x), _product_rows(w_gate), _product_rows(w_up)
        out = gated_projection_forward(x, w_gate, w_up, activation)
        ctx.save_for_backward(x, w_gate, w_up)
        ctx.activation = activation
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        x, w_gate, w_up = ctx.saved_tensors
        need = ctx.needs_input_grad
        g = gated_projection_backward(x, w_gate, w_up, _product_rows(d_out.to(x.dtype)), ctx.activation,
                                      (need[0], need[1] or need[2]))
        return tuple(t if n else None for t, n in zip(g, need)) + (None,)


def gated_projection(x, w_gate, w_up, activation: str = "silu"):
    """Differentiable act(x w_gate^T) * (x w_up^T); see gated_projection_forward.
    Operands that the library cannot read as they are, are copied."""
    return GatedProjectionFunction.apply(x, w_gate, w_up, activation)
