"""RMS norm of every query and key head and the rotation by position, in one
pass (include/gscan.h, gscan_qk_norm_rope_forward):

    y = x / sqrt(mean(x^2) + eps) * weight,

then the first 2 * len(freq) elements of y turned in pairs by the angles
position * freq[i].  `qk_norm_rope` is differentiable; `rotary_frequencies`
gives freq for plain and lengthened contexts.  Argument marshalling only.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .matrix_state import (_CODES, _On, _check_dense, _empty, _layout, _on_device, _outer_strides, _ptr,
                           _readable, _readable_rows, _reads_rows, _workspace)

LAYOUTS = {"half": 0, "interleaved": 1}
_i64x2 = ctypes.c_int64 * 2


class _Desc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hk", ctypes.c_int64),
                ("D", ctypes.c_int64), ("rot", ctypes.c_int64), ("q_stride", _i64x2),
                ("k_stride", _i64x2), ("dy_q_stride", _i64x2), ("dy_k_stride", _i64x2),
                ("dtype", ctypes.c_int), ("layout", ctypes.c_int), ("pos_int64", ctypes.c_int),
                ("eps", ctypes.c_float), ("magnitude", ctypes.c_float)]


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None,
                       factor: float = 1.0, original_length: int = 4096, beta_fast: float = 32.0,
                       beta_slow: float = 1.0, device=None):
    """(freq, magnitude): freq float32 [rot / 2] and the factor of the rotated
    elements for qk_norm_rope.

    freq_i = base^(-2i / rot).  For contexts `factor` times the
    `original_length` a model was trained on:
      "linear"  every frequency divided by factor (position interpolation);
      "base"    base * factor^(rot / (rot - 2)): the fastest pair keeps its
                frequency, the slowest is divided by factor;
      "parts"   (YaRN, Peng et al. 2023) pairs that turn more than beta_fast
                times over the original length keep their frequency, those
                below beta_slow turns are divided by factor, a linear ramp
                over the pair index between, from whole pair indexes outwards
                (the lower at least 0, the upper at most rot - 1 and so beyond
                the last pair where that turns more than beta_slow times);
                magnitude 0.1 ln(factor) + 1.
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError(f"need base > 1 and factor >= 1, got {base}, {factor}")
    i = torch.arange(rot // 2, dtype=torch.float64)
    magnitude = 1.0
    if scaling == "base":
        if rot < 4:
            raise ValueError("scaling 'base' needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    freq = base ** (-2.0 * i / rot)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "parts":
        def pair(turns):  # the (real) index of the pair with this many turns
            return rot * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))
        low = max(math.floor(pair(beta_fast)), 0)
        high = min(math.ceil(pair(beta_slow)), rot - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freq = freq / factor * ramp + freq * (1.0 - ramp)
        magnitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(torch.float32).to(device), magnitude


def _stride2(t):
    return _i64x2(*_outer_strides(*t)[:2])


@functools.lru_cache(maxsize=256)
def _template(q, k, qdt, kdt, qdev, kdev, eps, layout, magnitude):
    """The descriptor of a call, as bytes, from what shapes, strides and types
    say; refuses what does not fit.  q, k are (shape, stride), k may be None."""
    if qdev.type != "cuda":
        raise TypeError("q and k must be torch tensors on a GPU device")
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
    if qdt not in _CODES:
        raise TypeError(f"q and k must be float32 or bfloat16, got {qdt}")
    d = _Desc()
    for name, t, dt, dev in (("q", q, qdt, qdev), ("k", k, kdt, kdev)):
        if t is None:
            continue
        if dev != qdev:
            raise ValueError(f"{name} must be a tensor on {qdev}")
        shape = tuple(t[0])
        if len(shape) != 3 or dt != qdt or shape[0] != q[0][0] or shape[2] != q[0][2]:
            raise ValueError(f"q and k must be [tokens, heads, D] of one type; got {name} {dt} {shape} "
                             f"beside {qdt} {tuple(q[0])}")
        if not _reads_rows(*t):
            raise ValueError(f"the last dimension of {name} must be contiguous")
        setattr(d, name + "_stride", _stride2(t))
    d.tokens, d.Hq, d.D = q[0]
    d.Hk = 0 if k is None else k[0][1]
    if k is not None and d.Hk < 1:
        raise ValueError("k has no heads; pass None")
    d.dtype, d.layout = _CODES[qdt], LAYOUTS[layout]
    d.eps, d.magnitude = eps, magnitude
    return bytes(d)


def _describe(q, k, weight_q, weight_k, positions, freq, eps, layout, magnitude):
    if not isinstance(q, torch.Tensor) or not (k is None or isinstance(k, torch.Tensor)):
        raise TypeError("q and k must be torch tensors on a GPU device")
    dev = q.device
    d = _Desc.from_buffer_copy(_template(
        _layout(q), None if k is None else _layout(k), q.dtype, None if k is None else k.dtype, dev,
        None if k is None else k.device, float(eps), layout, float(magnitude)))
    for name, w in (("weight_q", weight_q), ("weight_k", weight_k)):
        if w is not None:
            _check_dense(w, (d.D,), torch.float32, dev, name)
    if freq is not None:
        if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
            raise ValueError("freq must be a float32 tensor [rot / 2]")
        _check_dense(freq, freq.shape, torch.float32, dev, "freq")
        d.rot = 2 * freq.shape[0]
        if not isinstance(positions, torch.Tensor) or positions.device != dev:
            raise ValueError(f"positions must be a tensor on {dev}")
        if positions.dtype not in (torch.int32, torch.int64) or \
                positions.shape != (d.tokens,) or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 or int64 tensor [{d.tokens}]; "
                             f"got {positions.dtype} {tuple(positions.shape)}")
        d.pos_int64 = int(positions.dtype == torch.int64)
    return d


def qk_norm_rope_forward(q, k, weight_q, weight_k, positions, freq, eps: float = 1e-6,
                         layout: str = "half", magnitude: float = 1.0, out=None, stream=None):
    """(q', k') of q [tokens, Hq, D] and k [tokens, Hk, D] (strided slices of a
    projection are fine; k may be None, then k' is): every head normalised,
    weighted (float32 [D], or None) and rotated by positions (int32 or int64
    [tokens]) times freq (float32 [rot / 2], or None: no rotation).  D is a
    multiple of 8 up to 256, rot of 8 up to D.  `out`: a pair to write into.
    """
    d = _describe(q, k, weight_q, weight_k, positions, freq, eps, layout, magnitude)
    dev = q.device
    if out is not None:
        if not isinstance(out, (tuple, list)) or len(out) != 2:
            raise ValueError("out must hold two tensors")
        _check_dense(out[0], q.shape, q.dtype, dev, "out[0]")
        if k is not None:
            _check_dense(out[1], k.shape, k.dtype, dev, "out[1]")
    with _On(dev, stream) as s:
        if out is None:
            out = (_empty(q), None if k is None else _empty(k))
        binding._check(binding.lib().gscan_qk_norm_rope_forward(
            ctypes.byref(d), q.data_ptr(), _ptr(k), _ptr(weight_q), _ptr(weight_k),
            _ptr(positions) if d.rot else None, _ptr(freq), out[0].data_ptr(),
            None if k is None else out[1].data_ptr(), s))
    return tuple(out)


def qk_norm_rope_backward(q, k, weight_q, weight_k, positions, freq, dy_q, dy_k,
                          eps: float = 1e-6, layout: str = "half", magnitude: float = 1.0,
                          workspace=None, stream=None):
    """(dq, dk, d_weight_q, d_weight_k): gradients in the types of their tensors
    (the weights' are None where the weight is)."""
    d = _describe(q, k, weight_q, weight_k, positions, freq, eps, layout, magnitude)
    dev, L = q.device, binding.lib()
    for name, t, like in (("dy_q", dy_q, q), ("dy_k", dy_k, k)):
        if like is None:
            continue
        _on_device(dev, **{name: t})
        if t.dtype != like.dtype or t.shape != like.shape or not _reads_rows(*_layout(t)):
            raise ValueError(f"{name} must be {like.dtype} {tuple(like.shape)}, last dimension "
                             f"contiguous; got {t.dtype} {tuple(t.shape)}")
        setattr(d, name + "_stride", _stride2(_layout(t)))
    need = 0
    if weight_q is not None or weight_k is not None:
        need = int(L.gscan_qk_norm_rope_workspace_bytes(ctypes.byref(d)))
    with _On(dev, stream) as s:
        dq, dk, dwq, dwk = (None if t is None else _empty(t)
                            for t in (q, k, weight_q, weight_k))
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(L.gscan_qk_norm_rope_backward(
            ctypes.byref(d), q.data_ptr(), _ptr(k), _ptr(weight_q), _ptr(weight_k),
            _ptr(positions) if d.rot else None, _ptr(freq), dy_q.data_ptr(),
            None if k is None else dy_k.data_ptr(), dq.data_ptr(), _ptr(dk), _ptr(dwq), _ptr(dwk), wp,
            wn, s))
    return dq, dk, dwq, dwk


class QkNormRopeFunction(torch.autograd.Function):
    """(q', k') of qk_norm_rope_forward with the gradients of q, k and weights."""

    @staticmethod
    def forward(ctx, q, k, weight_q, weight_k, positions, freq, eps, layout, magnitude):
        ctx.set_materialize_grads(False)
        q, k = _readable_rows(q, k)
        ctx.save_for_backward(q, k, weight_q, weight_k, positions, freq)
        ctx.args = (float(eps), layout, float(magnitude))
        return qk_norm_rope_forward(q, k, weight_q, weight_k, positions, freq, *ctx.args)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy_q, dy_k=None):
        q, k, wq, wk, positions, freq = ctx.saved_tensors
        if dy_q is None and dy_k is None:
            return (None,) * 9

        def up(g, like):
            if like is None:
                return None
            if g is None:
                return torch.zeros_like(like, memory_format=torch.contiguous_format)
            return _readable(g, like)

        g = qk_norm_rope_backward(q, k, wq, wk, positions, freq, up(dy_q, q), up(dy_k, k), *ctx.args)
        return tuple(x if n else None for x, n in zip(g, ctx.needs_input_grad)) + (None,) * 5


def qk_norm_rope(q, k, weight_q, weight_k, positions, freq, eps: float = 1e-6,
                 layout: str = "half", magnitude: float = 1.0):
    """Differentiable (q', k'); see qk_norm_rope_forward.  q and k whose rows are
    not 16-byte aligned are copied."""
    return QkNormRopeFunction.apply(q, k, weight_q, weight_k, positions, freq, eps, layout, magnitude)
