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
import functools

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .matrix_state import (_CODES, _On, _check_dense, _layout, _on_device, _outer_strides, _readable,
                           _reads_rows, _workspace)


class _Desc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("vocabulary", ctypes.c_int64), ("width", ctypes.c_int64),
                ("stride", ctypes.c_int64), ("table_dtype", ctypes.c_int), ("dtype", ctypes.c_int),
                ("token_int64", ctypes.c_int), ("scale", ctypes.c_float)]


def _row_stride(shape, stride, name):
    """The one stride between the rows of a tensor [..., width]."""
    if not _reads_rows(shape, stride):
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if len(shape) == 2:
        return _outer_strides(shape, stride)[0]
    dense = 1
    for n, x in zip(reversed(shape), reversed(stride)):
        if n > 1 and x != dense and 0 not in shape:
            raise ValueError(f"{name} of more than two dimensions must be contiguous")
        dense *= n
    return shape[-1]


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


# Elements between rows, at most: of a table and its output's gradient, of the matrix products.
_FURTHEST, _PRODUCTS_FURTHEST = 1 << 31, 1 << 21


def _rows(t, furthest=_FURTHEST):
    """t as the library reads it: copied where its rows lie on no multiple of 16
    bytes, at no single stride or too far apart (the last token of each long sequence, or
    a gradient that comes as such a slice); what is no tensor, or has no dimension, is
    left to the checks."""
    if not isinstance(t, torch.Tensor) or t.dim() == 0:
        return t
    t = _readable(t if t.dim() == 2 else t.contiguous(), t)
    if t.dim() == 2 and _outer_strides(*_layout(t))[0] > furthest:
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _product_rows(t):
    return _rows(t, _PRODUCTS_FURTHEST)


def _dense(t):
    """Tokens or targets one after the other (a batch without its first or last token
    is not); what is no tensor is left to the checks."""
    return t.contiguous() if isinstance(t, torch.Tensor) else t


@functools.lru_cache(maxsize=256)
def _template(rows, dtype, other, tokens, token_dtype, vocabulary, scale):
    """The descriptor of a call, as bytes; rows: (shape, stride) of the table
    (vocabulary None) or of the gradients of the output."""
    if vocabulary is None:
        if len(rows[0]) != 2:
            raise ValueError(f"table must be [vocabulary, width], got {tuple(rows[0])}")
        d = _Desc(tokens.numel(), *rows[0], _row_stride(*rows, "table"), _type_code(dtype, "table"),
                  _type_code(other, "dtype"))
    else:
        if len(rows[0]) < 1 or rows[0][:-1] != tokens:
            raise ValueError(f"d_out must be [*tokens.shape, width]; got {tuple(rows[0])} beside {tuple(tokens)}")
        d = _Desc(tokens.numel(), vocabulary, rows[0][-1], _row_stride(*rows, "d_out"),
                  _type_code(other, "dtype"), _type_code(dtype, "d_out"))
    d.token_int64, d.scale = token_dtype == torch.int64, scale
    return bytes(d)


@functools.lru_cache(maxsize=256)
def _need(desc):
    return int(binding.lib().gscan_embed_workspace_bytes(desc))


def embed_forward(table, tokens, scale: float = 1.0, dtype=None, out=None, stream=None):
    """scale * table[tokens], of shape [*tokens.shape, width] and type `dtype`
    (float32 or bfloat16; the table's own by default)."""
    dev = _device_of(table, "table")
    _check_tokens(tokens, dev)
    dtype = table.dtype if dtype is None else dtype
    d = _template(_layout(table), table.dtype, dtype, tokens.shape, tokens.dtype, None, float(scale))
    shape = (*tokens.shape, table.shape[1])
    if out is not None:
        _check_dense(out, shape, dtype, dev, "out")
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
        binding._check(binding.lib().gscan_embed_forward(d, table.data_ptr(), tokens.data_ptr(),
                                                         out.data_ptr(), s))
    return out


def _describe_backward(d_out, tokens, vocabulary, scale, dtype):
    dev = _device_of(d_out, "d_out")
    _check_tokens(tokens, dev)
    return _template(_layout(d_out), d_out.dtype, d_out.dtype if dtype is None else dtype, tokens.shape,
                     tokens.dtype, int(vocabulary), float(scale))


def embed_backward_workspace_bytes(d_out, tokens, vocabulary) -> int:
    """Workspace of embed_backward for these operands."""
    return _need(_describe_backward(d_out, tokens, vocabulary, 1.0, None))


def embed_backward(d_out, tokens, vocabulary: int, scale: float = 1.0, dtype=None, out=None,
                   workspace=None, stream=None):
    """The table's gradient [vocabulary, width] for d_out [*tokens.shape, width],
    in `dtype` (d_out's by default); rows of tokens that do not occur are zero.

    `workspace` may be a uint8 device tensor of at least
    embed_backward_workspace_bytes() bytes; otherwise one is taken from torch's
    caching allocator.
    """
    d = _describe_backward(d_out, tokens, vocabulary, scale, dtype)
    dev = d_out.device
    dtype = d_out.dtype if dtype is None else dtype
    shape, need = (int(vocabulary), d_out.shape[-1]), _need(d)
    if out is not None:
        _check_dense(out, shape, dtype, dev, "out")
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty(shape if shape[0] > 0 else (0, 0), dtype=dtype, device=dev)
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(binding.lib().gscan_embed_backward(d, d_out.data_ptr(), tokens.data_ptr(),
                                                          out.data_ptr(), wp, wn, s))
    return out


class EmbedFunction(torch.autograd.Function):
    """Rows of a table by token, with the table's gradient in its own type."""

    @staticmethod
    def forward(ctx, table, tokens, scale, dtype):
        tokens = _dense(tokens)
        out = embed_forward(_rows(table), tokens, scale, dtype)
        ctx.save_for_backward(tokens)
        ctx.args = (table.shape[0], float(scale), table.dtype)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        if not ctx.needs_input_grad[0]:
            return (None,) * 4
        return embed_backward(_rows(d_out), ctx.saved_tensors[0], *ctx.args), None, None, None


def embed(table, tokens, scale: float = 1.0, dtype=None):
    """Differentiable scale * table[tokens]; see embed_forward.  A table whose
    rows are not 16-byte aligned or more than 2^31 elements apart, and tokens that are
    not contiguous, are copied."""
    return EmbedFunction.apply(table, tokens, scale, dtype)
