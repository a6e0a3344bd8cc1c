"""Token embedding (include/gscan.h, gscan_embed_forward):

    out[n] = scale * table[tokens[n]]

and the gradient of the table, summed by sorted tokens in a fixed order.
`embed` is differentiable; `embed_forward` / `embed_backward` are the calls
under it.  Argument marshalling only.

tokens: int32 or int64, contiguous, any shape.  One outside the table is
padding: a row of zeros, no gradient (the values are not looked at on the
host).  table: float32 or bfloat16 [vocabulary, width], the width contiguous
and a multiple of 8 up to 65536; the output may have either type, so that a
float32 table gives bfloat16 activations without a copy of its own.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .matrix_state import (_CODES, _On, _check_dense, _layout, _on_device, _outer_strides, _ptr, _readable,
                           _reads_rows, _workspace)


class _Desc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("vocabulary", ctypes.c_int64), ("width", ctypes.c_int64),
                ("stride", ctypes.c_int64), ("table_dtype", ctypes.c_int), ("dtype", ctypes.c_int),
                ("token_int64", ctypes.c_int), ("scale", ctypes.c_float)]


def _row_stride(t, name):
    """The one stride between the rows of a tensor [..., width]."""
    if not _reads_rows(*_layout(t)):
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if t.dim() == 2:
        return _outer_strides(*_layout(t))[0]
    if not t.is_contiguous():
        raise ValueError(f"{name} of more than two dimensions must be contiguous")
    return t.shape[-1]


def _check_tokens(tokens, dev, name="tokens"):
    _on_device(dev, **{name: tokens})
    if tokens.dtype not in (torch.int32, torch.int64) or not tokens.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 or int64 tensor; got {tokens.dtype} "
                         f"{tuple(tokens.shape)}")


def _type_code(dtype, name):
    if dtype not in _CODES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    return _CODES[dtype]


def _device_of(t, name):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a torch tensor on a GPU device")
    return t.device


def embed_forward(table, tokens, scale: float = 1.0, dtype=None, out=None, stream=None):
    """scale * table[tokens], of shape [*tokens.shape, width] and type `dtype`
    (float32 or bfloat16; the table's own by default)."""
    dev = _device_of(table, "table")
    if table.dim() != 2:
        raise ValueError(f"table must be [vocabulary, width], got {tuple(table.shape)}")
    _check_tokens(tokens, dev)
    dtype = table.dtype if dtype is None else dtype
    shape = (*tokens.shape, table.shape[1])
    d = _Desc(tokens.numel(), *table.shape, _row_stride(table, "table"), _type_code(table.dtype, "table"),
              _type_code(dtype, "dtype"), tokens.dtype == torch.int64, float(scale))
    if out is not None:
        _check_dense(out, shape, dtype, dev, "out")
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
        binding._check(binding.lib().gscan_embed_forward(
            ctypes.byref(d), table.data_ptr(), tokens.data_ptr(), out.data_ptr(), s))
    return out


def _describe_backward(d_out, tokens, vocabulary, scale, dtype):
    dev = _device_of(d_out, "d_out")
    _check_tokens(tokens, dev)
    if d_out.dim() < 1 or d_out.shape[:-1] != tokens.shape:
        raise ValueError(f"d_out must be [*tokens.shape, width]; got {tuple(d_out.shape)} beside "
                         f"{tuple(tokens.shape)}")
    return _Desc(tokens.numel(), int(vocabulary), d_out.shape[-1], _row_stride(d_out, "d_out"),
                 _type_code(dtype, "dtype"), _type_code(d_out.dtype, "d_out"), tokens.dtype == torch.int64,
                 float(scale))


def embed_backward_workspace_bytes(d_out, tokens, vocabulary) -> int:
    """Workspace of embed_backward for these operands."""
    d = _describe_backward(d_out, tokens, vocabulary, 1.0, d_out.dtype)
    return int(binding.lib().gscan_embed_workspace_bytes(ctypes.byref(d)))


def embed_backward(d_out, tokens, vocabulary: int, scale: float = 1.0, dtype=None, out=None,
                   workspace=None, stream=None):
    """The table's gradient [vocabulary, width] for d_out [*tokens.shape, width],
    in `dtype` (d_out's by default); rows of tokens that do not occur are zero.

    `workspace` may be a uint8 device tensor of at least
    embed_backward_workspace_bytes() bytes; otherwise one is taken from torch's
    caching allocator.
    """
    dtype = d_out.dtype if dtype is None and isinstance(d_out, torch.Tensor) else dtype
    d = _describe_backward(d_out, tokens, vocabulary, scale, dtype)
    dev, L = d_out.device, binding.lib()
    shape = (d.vocabulary, d.width)
    if out is not None:
        _check_dense(out, shape, dtype, dev, "out")
    need = int(L.gscan_embed_workspace_bytes(ctypes.byref(d)))
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty(shape if d.vocabulary > 0 else (0, 0), dtype=dtype, device=dev)
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(L.gscan_embed_backward(ctypes.byref(d), _ptr(d_out), tokens.data_ptr(),
                                              out.data_ptr(), wp, wn, s))
    return out


class EmbedFunction(torch.autograd.Function):
    """Rows of a table by token, with the table's gradient in its own type."""

    @staticmethod
    def forward(ctx, table, tokens, scale, dtype):
        ctx.save_for_backward(tokens)
        ctx.args = (table.shape, table.dtype, float(scale))
        return embed_forward(_readable(table, table), tokens, scale, dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        if not ctx.needs_input_grad[0]:
            return (None,) * 4
        (tokens,), (shape, dtype, scale) = ctx.saved_tensors, ctx.args
        if d_out.dim() != 2:
            d_out = d_out.contiguous()
        return embed_backward(_readable(d_out, d_out), tokens, shape[0], scale, dtype), None, None, None


def embed(table, tokens, scale: float = 1.0, dtype=None):
    """Differentiable scale * table[tokens]; see embed_forward.  A table whose
    rows are not 16-byte aligned is copied."""
    return EmbedFunction.apply(table, tokens, scale, dtype)
