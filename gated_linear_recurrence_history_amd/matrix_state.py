"""The matrix-state scan: a gated recurrence with a state per head, an output
per token and sequences of any length (include/gscan.h):

    g_t = sigmoid(gate_t + gate_shift)    (gate_form "sigmoid"), or
    g_t = exp(gate_t + gate_shift)        (gate_form "log")
    S_t = g_t S_{t-1} + k_t v_t^T,        out_t = scale * S_t^T q_t

`state_scan` is differentiable, `state_scan_forward` / `state_scan_backward`
are the calls under it, `state_scan_step` advances one token of each of many
requests over a pool of states.  Argument marshalling only: every step of the
computation runs in the library's kernels.

Shapes.  Dense: q, k [B, T, Hk, Dk], v [B, T, H, Dv], gate [B, T, H].  Packed
sequences: q, k [tokens, Hk, Dk], v [tokens, H, Dv], gate [tokens, H] and
seq_offsets, an int32 GPU tensor [sequences + 1] that starts at 0, does not
decrease and ends at the number of tokens (its values are not checked: that
would wait for the GPU; wrong ones give wrong outputs but no access out of
range).  Hk divides H: head h uses q and k of head h // (H // Hk).  Dk and Dv
are multiples of 8 up to 128.  q, k, v share a type, float32 or bfloat16; the
gate may have either; states are float32 [sequences, H, Dk, Dv].  The last
dimension is contiguous, the others may have any stride of 16 bytes'
multiple, such as a slice of a fused projection's output has (the gate: any
stride).  `state_scan` and `state_scan_step` copy q, k or v whose rows are not
16-byte aligned; the two calls under `state_scan` refuse them.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from . import binding

GATE_FORMS = {"sigmoid": 0, "log": 1}
_CODES = {torch.float32: binding.GSCAN_F32, torch.bfloat16: binding.GSCAN_BF16}
_i64x3 = ctypes.c_int64 * 3


class _Desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("Hk", ctypes.c_int64), ("Dk", ctypes.c_int64), ("Dv", ctypes.c_int64),
                ("seq_offsets", ctypes.c_void_p), ("q_stride", _i64x3), ("k_stride", _i64x3),
                ("v_stride", _i64x3), ("gate_stride", _i64x3), ("d_out_stride", _i64x3),
                ("dtype", ctypes.c_int), ("gate_dtype", ctypes.c_int),
                ("gate_form", ctypes.c_int), ("gate_shift", ctypes.c_float),
                ("scale", ctypes.c_float)]


def _on_device(dev, **tensors):
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor) or t.device != dev:
            raise ValueError(f"{name} must be a tensor on {dev}")


def _reads_rows(shape, stride):
    """Whether the last dimension is contiguous (or there is nothing to read)."""
    return shape[-1] <= 1 or stride[-1] == 1 or 0 in shape


def _outer_strides(shape, stride):
    """Strides of the dimensions; one without a second element has none."""
    return [0] * len(shape) if 0 in shape else [0 if n <= 1 else x for n, x in zip(shape, stride)]


def _strides(t, lead):
    """(batch, token, head) strides of an operand, given as (shape, stride)."""
    s = _outer_strides(*t)
    return _i64x3(s[0], s[1], s[2]) if lead == 2 else _i64x3(0, s[0], s[1])


def _layout(t):
    return t.shape, t.stride()


@functools.lru_cache(maxsize=256)
def _template(q, k, v, gate, dtypes, devices, scale, gate_form, gate_shift, sequences, single):
    """The descriptor of a call, as bytes, from what shapes, strides and types
    say; refuses what does not fit.  q, k, v, gate are (shape, stride)."""
    if devices[0].type != "cuda":
        raise TypeError("q, k, v and gate must be torch tensors on a GPU device")
    for name, dev in zip(("k", "v", "gate"), devices[1:]):
        if dev != devices[0]:
            raise ValueError(f"{name} must be a tensor on {devices[0]}")
    if dtypes[0] not in _CODES or dtypes[1] != dtypes[0] or dtypes[2] != dtypes[0]:
        raise TypeError(f"q, k, v must share a type, float32 or bfloat16; got {dtypes[0]}, {dtypes[1]}, "
                        f"{dtypes[2]}")
    if dtypes[3] not in _CODES:
        raise TypeError(f"gate must be float32 or bfloat16, got {dtypes[3]}")
    if gate_form not in GATE_FORMS:
        raise ValueError(f"gate_form must be one of {sorted(GATE_FORMS)}, got {gate_form!r}")
    qs, ks, vs, gs = (tuple(x[0]) for x in (q, k, v, gate))
    lead = 1 if single or sequences else 2
    if len(qs) != lead + 2 or len(vs) != lead + 2:
        want = ("[requests, heads, width]" if single else "[tokens, heads, width] (packed)"
                if lead == 1 else "[batch, tokens, heads, width]")
        raise ValueError(f"q, k, v must be {want}; got {qs}, {vs}")
    if ks != qs or vs[:lead] != qs[:lead] or gs != vs[:-1]:
        raise ValueError(f"shapes do not fit: q {qs}, k {ks}, v {vs}, gate {gs}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not _reads_rows(*t):
            raise ValueError(f"the last dimension of {name} must be contiguous")
    d = _Desc()
    if single:
        d.B, d.T = qs[0], 1
    elif lead == 2:
        d.B, d.T = qs[0], qs[1]
    else:
        d.B, d.T = sequences, qs[0]
    d.H, d.Hk, d.Dk, d.Dv = vs[-2], qs[-2], qs[-1], vs[-1]
    if single:  # requests are the batch dimension
        for name, t in (("q", q), ("k", k), ("v", v), ("gate", gate)):
            s = _outer_strides(*t)
            setattr(d, name + "_stride", _i64x3(s[0], 0, s[1]))
    else:
        d.q_stride, d.k_stride = _strides(q, lead), _strides(k, lead)
        d.v_stride, d.gate_stride = _strides(v, lead), _strides(gate, lead)
    d.dtype, d.gate_dtype = _CODES[dtypes[0]], _CODES[dtypes[3]]
    d.gate_form, d.gate_shift, d.scale = GATE_FORMS[gate_form], gate_shift, scale
    return bytes(d)


def _describe(q, k, v, gate, scale, gate_form, gate_shift, seq_offsets, single=False):
    """Checks shapes, types and devices; returns the descriptor.  `single`: one
    token per request ([N, heads, width])."""
    for t in (q, k, v, gate):
        if not isinstance(t, torch.Tensor):
            raise TypeError("q, k, v and gate must be torch tensors on a GPU device")
    n = 0
    if seq_offsets is not None:
        _on_device(q.device, seq_offsets=seq_offsets)
        if seq_offsets.dtype != torch.int32 or seq_offsets.dim() != 1 or \
                seq_offsets.numel() < 2 or not seq_offsets.is_contiguous():
            raise ValueError("seq_offsets must be a contiguous int32 tensor [sequences + 1]; got "
                             f"{seq_offsets.dtype} {tuple(seq_offsets.shape)}")
        n = seq_offsets.numel() - 1
    d = _Desc.from_buffer_copy(_template(
        _layout(q), _layout(k), _layout(v), _layout(gate), (q.dtype, k.dtype, v.dtype, gate.dtype),
        (q.device, k.device, v.device, gate.device), float(scale), gate_form, float(gate_shift), n,
        single))
    if n:
        d.seq_offsets = seq_offsets.data_ptr()
    return d


def _check_dense(t, shape, dtype, dev, name):
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}")
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}; "
                         f"got {t.dtype} {tuple(t.shape)}")


def _empty(like):
    """A dense tensor of the shape and type of `like`."""
    return torch.empty_like(like, memory_format=torch.contiguous_format)


def _workspace(workspace, need, dev):
    """(pointer, bytes, tensor to keep alive)"""
    if workspace is not None:
        binding._check_workspace(workspace, need, dev)
        return workspace.data_ptr(), workspace.numel(), workspace
    if need == 0:
        return None, 0, None
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    return ws.data_ptr(), need, ws


class _On:
    """The device and stream a call runs on, current while it allocates: what
    it takes from torch's allocator then belongs to that stream."""

    def __init__(self, dev, stream):
        self.ctx = None
        if stream is None and torch.cuda.current_device() == dev.index:
            self.handle = torch._C._cuda_getCurrentRawStream(dev.index)
        else:
            stream = torch.cuda.current_stream(dev) if stream is None else stream
            self.ctx, self.handle = torch.cuda.stream(stream), stream.cuda_stream

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.ctx is not None:
            return self.ctx.__exit__(*exc)
        return False


def _ptr(t):
    return None if t is None else t.data_ptr()


def state_scan_forward_workspace_bytes(q, k, v, gate, seq_offsets=None) -> int:
    """Workspace of state_scan_forward for these operands (0: none needed)."""
    d = _describe(q, k, v, gate, 1.0, "sigmoid", 0.0, seq_offsets)
    return int(binding.lib().gscan_state_scan_forward_workspace_bytes(ctypes.byref(d)))


def state_scan_backward_workspace_bytes(q, k, v, gate, seq_offsets=None) -> int:
    """Workspace of state_scan_backward for these operands."""
    d = _describe(q, k, v, gate, 1.0, "sigmoid", 0.0, seq_offsets)
    return int(binding.lib().gscan_state_scan_backward_workspace_bytes(ctypes.byref(d)))


def state_scan_forward(q, k, v, gate, scale: float = 1.0, gate_form: str = "sigmoid",
                       gate_shift: float = 0.0, seq_offsets=None, initial_state=None,
                       final_state=None, out=None, workspace=None, stream=None):
    """Outputs of every token, of the shape and type of v; with `final_state`
    True (or a float32 tensor [sequences, H, Dk, Dv] to write into, which may
    be initial_state itself) the pair (out, final state).

    `workspace` may be a uint8 device tensor of at least
    state_scan_forward_workspace_bytes() bytes; otherwise one is taken from
    torch's caching allocator where needed.
    """
    d = _describe(q, k, v, gate, scale, gate_form, gate_shift, seq_offsets)
    dev, L = q.device, binding.lib()
    states = (d.B, d.H, d.Dk, d.Dv)
    if initial_state is not None:
        _check_dense(initial_state, states, torch.float32, dev, "initial_state")
    if out is not None:
        _check_dense(out, v.shape, v.dtype, dev, "out")
    want = final_state is not None and final_state is not False
    if want and final_state is not True:
        _check_dense(final_state, states, torch.float32, dev, "final_state")
    need = int(L.gscan_state_scan_forward_workspace_bytes(ctypes.byref(d)))
    with _On(dev, stream) as s:
        if out is None:
            out = _empty(v)
        if final_state is True:
            final_state = v.new_empty(states, dtype=torch.float32)
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(L.gscan_state_scan_forward(
            ctypes.byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), gate.data_ptr(),
            _ptr(initial_state), out.data_ptr(), final_state.data_ptr() if want else None, wp, wn, s))
    return (out, final_state) if want else out


def state_scan_backward(q, k, v, gate, d_out, scale: float = 1.0, gate_form: str = "sigmoid",
                        gate_shift: float = 0.0, seq_offsets=None, initial_state=None,
                        d_final_state=None, workspace=None, stream=None):
    """(dq, dk, dv, dgate, d_initial_state) for L = sum(d_out * out) +
    sum(d_final_state * final state), in the types of their tensors (sums in
    float32); d_initial_state is None unless initial_state is given.

    `workspace` may be a uint8 device tensor of at least
    state_scan_backward_workspace_bytes() bytes; otherwise one is taken from
    torch's caching allocator.
    """
    d = _describe(q, k, v, gate, scale, gate_form, gate_shift, seq_offsets)
    dev, L = q.device, binding.lib()
    states = (d.B, d.H, d.Dk, d.Dv)
    _on_device(dev, d_out=d_out)
    if d_out.dtype != v.dtype or d_out.shape != v.shape:
        raise ValueError(f"d_out must be {v.dtype} {tuple(v.shape)}; got {d_out.dtype} "
                         f"{tuple(d_out.shape)}")
    if not _reads_rows(*_layout(d_out)):
        raise ValueError("the last dimension of d_out must be contiguous")
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None:
            _check_dense(t, states, torch.float32, dev, name)
    d.d_out_stride = _strides(_layout(d_out), d_out.dim() - 2)
    need = int(L.gscan_state_scan_backward_workspace_bytes(ctypes.byref(d)))
    with _On(dev, stream) as s:
        dq, dk, dv, dgate = (_empty(t) for t in (q, k, v, gate))
        ds0 = None
        if initial_state is not None:
            ds0 = v.new_empty(states, dtype=torch.float32)
        wp, wn, _keep = _workspace(workspace, need, dev)
        binding._check(L.gscan_state_scan_backward(
            ctypes.byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), gate.data_ptr(),
            _ptr(initial_state), d_out.data_ptr(), _ptr(d_final_state), dq.data_ptr(), dk.data_ptr(),
            dv.data_ptr(), dgate.data_ptr(), _ptr(ds0), wp, wn, s))
    return dq, dk, dv, dgate, ds0


def state_scan_step(q, k, v, gate, state, slots=None, scale: float = 1.0,
                    gate_form: str = "sigmoid", gate_shift: float = 0.0, out=None, stream=None):
    """One token for each request: q, k [N, Hk, Dk], v [N, H, Dv], gate [N, H];
    updates state[slots[n]] (float32 [pool, H, Dk, Dv]) in place and returns
    the outputs [N, H, Dv] in the type of v.  `slots`: int32 [N], none twice;
    one outside the pool is padding (nothing is updated, its output is zero).
    Without slots request n uses state n.  q, k, v whose rows are not 16-byte
    aligned are copied.
    """
    d = _describe(q, k, v, gate, scale, gate_form, gate_shift, None, single=True)
    dev = q.device
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a tensor [pool, H, Dk, Dv]")
    _check_dense(state, (state.shape[0], d.H, d.Dk, d.Dv), torch.float32, dev, "state")
    if slots is not None:
        _check_dense(slots, (d.B,), torch.int32, dev, "slots")
    if out is not None:
        _check_dense(out, v.shape, v.dtype, dev, "out")
    with _On(dev, stream) as s:
        if out is None:
            out = _empty(v)
        if d.B:
            status = binding.lib().gscan_state_scan_step(
                ctypes.byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), gate.data_ptr(),
                state.data_ptr(), state.shape[0], _ptr(slots), out.data_ptr(), s)
            if status == binding.GSCAN_ERR_MISALIGNED:  # nothing was enqueued
                rows = _readable_rows(q, k, v)
                if any(x is not y for x, y in zip(rows, (q, k, v))):
                    return state_scan_step(*rows, gate, state, slots, scale, gate_form, gate_shift, out,
                                           stream)
            binding._check(status)
    return out


def _readable(g, like):
    """An upstream gradient the library can read as it is, else a dense copy."""
    g = g.to(like.dtype)
    fits = _reads_rows(*_layout(g)) and g.data_ptr() % 16 == 0 and all(
        s * g.element_size() % 16 == 0 for s in _outer_strides(*_layout(g))[:-1])
    # (contiguous() would return a dense tensor that begins on no 16 bytes)
    return g if fits else g.clone(memory_format=torch.contiguous_format)


def _readable_rows(*operands):
    """The same of inputs; what is no tensor is left to the checks."""
    return [_readable(x, x) if isinstance(x, torch.Tensor) else x for x in operands]


class StateScanFunction(torch.autograd.Function):
    """(out, final state) of the matrix-state scan; the backward replays the
    forward from the saved inputs, so nothing else is kept in between."""

    @staticmethod
    def forward(ctx, q, k, v, gate, initial_state, scale, gate_form, gate_shift, seq_offsets):
        ctx.set_materialize_grads(False)
        q, k, v = _readable_rows(q, k, v)
        ctx.save_for_backward(q, k, v, gate, initial_state, seq_offsets)
        ctx.args = (float(scale), gate_form, float(gate_shift))
        return state_scan_forward(q, k, v, gate, *ctx.args, seq_offsets, initial_state, True)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_final):
        q, k, v, gate, s0, off = ctx.saved_tensors
        if d_out is None and d_final is None:
            return (None,) * 9
        d_out = torch.zeros_like(v, memory_format=torch.contiguous_format) if d_out is None \
            else _readable(d_out, v)
        if d_final is not None:
            d_final = d_final.to(torch.float32).contiguous()
        g = state_scan_backward(q, k, v, gate, d_out, *ctx.args, off, s0, d_final)
        return tuple(x if n else None for x, n in zip(g, ctx.needs_input_grad)) + (None,) * 4


def state_scan(q, k, v, gate, initial_state=None, scale: float = 1.0, gate_form: str = "sigmoid",
               gate_shift: float = 0.0, seq_offsets=None):
    """Differentiable scan: (out, final state); see state_scan_forward.  q, k, v
    that the library cannot read as they are, are copied."""
    return StateScanFunction.apply(q, k, v, gate, initial_state, scale, gate_form, gate_shift,
                                   seq_offsets)
