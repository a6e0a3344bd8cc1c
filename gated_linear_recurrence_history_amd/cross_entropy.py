"""Cross entropy over a vocabulary from the last hidden states and the output
weights, without the logits in memory (include/gscan.h,
gscan_linear_cross_entropy_forward):

    lse[n] = log sum_v exp(scale * <h_n, weight_v>)
    loss[n] = lse[n] - scale * <h_n, weight_target[n]>

`linear_cross_entropy` is differentiable; `linear_cross_entropy_forward` /
`_backward` are the calls under it.  Argument marshalling only.

h [..., width] and weight [vocabulary, width] (as torch.nn.Linear keeps it)
share a type, float32 or bfloat16; the width is a multiple of 8 up to 65536,
the vocabulary any size.  Rows may lie any multiple of 16 bytes up to 2^21
elements apart; `linear_cross_entropy` copies h or weights whose rows are further
apart.  target [...]: int32 or int64, contiguous; a token
whose target is outside the vocabulary (-100, say) does not count: its loss and
lse are zero, and what its row of h holds reaches nothing.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .embedding import _check_tokens, _dense, _device_of, _product_rows, _row_stride, _type_code
from .matrix_state import _check_dense, _layout, _On, _on_device, _ptr, _workspace

REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}


class _Desc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("width", ctypes.c_int64), ("vocabulary", ctypes.c_int64),
                ("h_stride", ctypes.c_int64), ("weight_stride", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("reduction", ctypes.c_int), ("target_int64", ctypes.c_int), ("scale", ctypes.c_float)]


@functools.lru_cache(maxsize=256)
def _template(h, weight, target, dtypes, scale, reduction):
    """The descriptor of a call, as bytes; h and weight are (shape, stride)."""
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}, got {reduction!r}")
    if dtypes[1] != dtypes[0]:
        raise TypeError(f"h and weight must share a type; got {dtypes[0]}, {dtypes[1]}")
    hs, ws = h[0], weight[0]
    if len(hs) < 1 or len(ws) != 2 or ws[1] != hs[-1] or target != hs[:-1]:
        raise ValueError("h must be [..., width], weight [vocabulary, width], target [...]; got "
                         f"{tuple(hs)}, {tuple(ws)}, {tuple(target)}")
    return bytes(_Desc(target.numel(), hs[-1], ws[0], _row_stride(*h, "h"), _row_stride(*weight, "weight"),
                       _type_code(dtypes[0], "h"), REDUCTIONS[reduction], dtypes[2] == torch.int64, scale))


@functools.lru_cache(maxsize=256)
def _need(desc, backward):
    L = binding.lib()
    return int((L.gscan_linear_cross_entropy_backward_workspace_bytes if backward else
                L.gscan_linear_cross_entropy_forward_workspace_bytes)(desc))


def _describe(h, weight, target, scale, reduction):
    dev = _device_of(h, "h")
    _on_device(dev, weight=weight)
    _check_tokens(target, dev, "target")
    return _template(_layout(h), _layout(weight), target.shape, (h.dtype, weight.dtype, target.dtype),
                     float(scale), reduction)


def linear_cross_entropy_forward_workspace_bytes(h, weight, target) -> int:
    """Workspace of linear_cross_entropy_forward for these operands."""
    return _need(_describe(h, weight, target, 1.0, "none"), False)


def linear_cross_entropy_backward_workspace_bytes(h, weight, target) -> int:
    """Workspace of linear_cross_entropy_backward for these operands."""
    return _need(_describe(h, weight, target, 1.0, "none"), True)


def linear_cross_entropy_forward(h, weight, target, scale: float = 1.0, reduction: str = "mean",
                                 workspace=None, stream=None):
    """(loss, lse), float32: loss of target's shape (reduction "none") or a scalar
    (over the tokens that count; a mean over none is zero), lse of target's shape,
    which the backward takes.

    `workspace` may be a uint8 device tensor of at least
    linear_cross_entropy_forward_workspace_bytes() bytes; otherwise one is taken
    from torch's caching allocator.
    """
    d = _describe(h, weight, target, scale, reduction)
    dev, need = h.device, _need(d, False)
    with _On(dev, stream) as s:
        lse = torch.empty(target.shape, dtype=torch.float32, device=dev)
        loss = torch.empty(target.shape if reduction == "none" else (), dtype=torch.float32, device=dev)
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(binding.lib().gscan_linear_cross_entropy_forward(
            d, h.data_ptr(), weight.data_ptr(), target.data_ptr(), loss.data_ptr(),
            lse.data_ptr(), wp, wn, s))
    return loss, lse


def linear_cross_entropy_backward(h, weight, target, lse, d_loss, scale: float = 1.0,
                                  reduction: str = "mean", wanted=(True, True), workspace=None, stream=None):
    """(dh, d_weight) in the operands' type, for d_loss (float32, of the loss's
    shape) and the lse of the forward.  `wanted`: whether each is formed (None
    where not).

    `workspace` may be a uint8 device tensor of at least
    linear_cross_entropy_backward_workspace_bytes() bytes; otherwise one is taken
    from torch's caching allocator.
    """
    d = _describe(h, weight, target, scale, reduction)
    dev, need = h.device, _need(d, True)
    _check_dense(lse, target.shape, torch.float32, dev, "lse")
    _check_dense(d_loss, target.shape if reduction == "none" else torch.Size(), torch.float32, dev, "d_loss")
    with _On(dev, stream) as s:
        dh = torch.empty(h.shape, dtype=h.dtype, device=dev) if wanted[0] else None
        dw = torch.empty(weight.shape, dtype=h.dtype, device=dev) if wanted[1] else None
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(binding.lib().gscan_linear_cross_entropy_backward(
            d, h.data_ptr(), weight.data_ptr(), target.data_ptr(), lse.data_ptr(),
            d_loss.data_ptr(), _ptr(dh), _ptr(dw), wp, wn, s))
    return dh, dw


class LinearCrossEntropyFunction(torch.autograd.Function):
    """The loss; the backward forms the logits again, a piece of the vocabulary at
    a time, from the saved operands and log-sums."""

    @staticmethod
    def forward(ctx, h, weight, target, scale, reduction):
        h, weight, target = _product_rows(h), _product_rows(weight), _dense(target)
        loss, lse = linear_cross_entropy_forward(h, weight, target, scale, reduction)
        ctx.save_for_backward(h, weight, target, lse)
        ctx.args = (float(scale), reduction)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, d_loss):
        need = ctx.needs_input_grad
        g = linear_cross_entropy_backward(*ctx.saved_tensors, d_loss.to(torch.float32).contiguous(), *ctx.args,
                                          (need[0], need[1]))
        return tuple(g) + (None,) * 3


def linear_cross_entropy(h, weight, target, scale: float = 1.0, reduction: str = "mean"):
    """Differentiable loss; see linear_cross_entropy_forward.  Operands that the
    library cannot read as they are, are copied."""
    return LinearCrossEntropyFunction.apply(h, weight, target, scale, reduction)
