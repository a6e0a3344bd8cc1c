"""Refusals of the matrix-state scan, its step and the query/key norm, at the C
ABI and in the binding, without a GPU: every call here fails its checks before
anything is enqueued (or has nothing to do).  Pointers are never dereferenced
on these paths.  Also the rotary frequencies, which the host computes."""
import ctypes
import math
import os

import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from gated_linear_recurrence_history_amd import binding, matrix_state as ms, qk_norm as qn

OK, INVALID, UNSUPPORTED, MISALIGNED, WS_SMALL = 0, 1, 2, 3, 4
P = 0x10000  # an aligned "device pointer"
BF, F32 = binding.GSCAN_BF16, binding.GSCAN_F32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from gated_linear_recurrence_history_amd import _build
        _build.build_hip()
    return binding.lib()


def scan_desc(**kw):
    """A valid dense descriptor with `kw` changed."""
    c = dict(B=2, T=100, H=8, Hk=4, Dk=64, Dv=48, dtype=BF, gate_dtype=F32, gate_form=0,
             gate_shift=0.0, scale=1.0, seq_offsets=None)
    c.update({k: v for k, v in kw.items() if k in c})
    d = ms._Desc(**c)
    for name, heads, width in (("q", c["Hk"], c["Dk"]), ("k", c["Hk"], c["Dk"]), ("v", c["H"], c["Dv"]),
                               ("gate", c["H"], 1), ("d_out", c["H"], c["Dv"])):
        row = heads * width
        setattr(d, name + "_stride", (ctypes.c_int64 * 3)(row * c["T"], row, width))
    for k, v in kw.items():
        if k.endswith("_stride"):
            setattr(d, k, (ctypes.c_int64 * 3)(*v))
    return d


def forward(lib, d, q=P, k=P, v=P, gate=P, s0=None, out=P, sT=None, ws=None, n=0):
    return lib.gscan_state_scan_forward(d and ctypes.byref(d), q, k, v, gate, s0, out, sT, ws, n, None)


def backward(lib, d, q=P, k=P, v=P, gate=P, s0=None, do=P, dsT=None, dq=P, dk=P, dv=P, dg=P, ds0=None,
             ws=None, n=0):
    return lib.gscan_state_scan_backward(d and ctypes.byref(d), q, k, v, gate, s0, do, dsT, dq, dk, dv, dg,
                                         ds0, ws, n, None)


def step(lib, d, q=P, k=P, v=P, gate=P, state=P, pool=8, slots=P, out=P):
    return lib.gscan_state_scan_step(d and ctypes.byref(d), q, k, v, gate, state, pool, slots, out, None)


BAD_SHAPES = [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID),
    (dict(Dk=0), INVALID), (dict(Dv=-8), INVALID),
    (dict(dtype=7), INVALID), (dict(gate_dtype=-1), INVALID), (dict(gate_form=2), INVALID),
    (dict(Dk=20), UNSUPPORTED), (dict(Dv=12), UNSUPPORTED), (dict(Dk=136), UNSUPPORTED),
    (dict(Dv=136), UNSUPPORTED), (dict(Hk=3), UNSUPPORTED), (dict(H=16392, Hk=1), UNSUPPORTED),
    (dict(B=2**31), UNSUPPORTED),
    (dict(q_stride=(6400, 260, 64)), MISALIGNED), (dict(k_stride=(25600, 256, 68)), MISALIGNED),
    (dict(v_stride=(38404, 384, 48)), MISALIGNED),
    (dict(q_stride=(25600, -256, 64)), UNSUPPORTED), (dict(gate_stride=(800, 8, -1)), UNSUPPORTED),
    (dict(k_stride=(25600, 2**23, 64)), UNSUPPORTED), (dict(v_stride=(38400, 384, 2**31)), UNSUPPORTED),
]


@pytest.mark.parametrize("change,want", BAD_SHAPES)
def test_scan_refuses_descriptors(lib, change, want):
    d = scan_desc(**change)
    assert forward(lib, d) == want
    assert lib.gscan_last_error() != b""
    assert backward(lib, d) == want
    assert step(lib, d) == (want if d.T == 1 or want != OK else INVALID)
    assert lib.gscan_state_scan_forward_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.gscan_state_scan_backward_workspace_bytes(ctypes.byref(d)) == 0


def test_scan_refuses_the_token_count(lib):
    for d in (scan_desc(B=1, T=2**31 - 1, q_stride=(0, 256, 64)), scan_desc(B=2**20, T=2**20)):
        assert forward(lib, d) == UNSUPPORTED and backward(lib, d) == UNSUPPORTED


def test_scan_refuses_null_descriptor(lib):
    assert forward(lib, None) == INVALID and backward(lib, None) == INVALID and step(lib, None) == INVALID
    assert lib.gscan_state_scan_forward_workspace_bytes(None) == 0
    assert lib.gscan_state_scan_backward_workspace_bytes(None) == 0
    assert lib.gscan_qk_norm_rope_workspace_bytes(None) == 0


@pytest.mark.parametrize("name", ["q", "k", "v", "gate", "out"])
def test_forward_refuses_null_and_misaligned(lib, name):
    d = scan_desc()
    assert forward(lib, d, **{name: None}) == INVALID
    assert forward(lib, d, **{name: P + 2}) == MISALIGNED
    if name != "gate":  # the gate is aligned to its elements only
        assert forward(lib, d, **{name: P + 8}) == MISALIGNED


@pytest.mark.parametrize("name", ["q", "k", "v", "gate", "do", "dq", "dk", "dv", "dg"])
def test_backward_refuses_null_and_misaligned(lib, name):
    d = scan_desc()
    assert backward(lib, d, **{name: None}) == INVALID
    assert backward(lib, d, **{name: P + 2}) == MISALIGNED


def test_scan_refuses_misaligned_states_and_offsets(lib):
    d = scan_desc()
    assert forward(lib, d, s0=P + 4) == MISALIGNED and forward(lib, d, sT=P + 8) == MISALIGNED
    assert backward(lib, d, s0=P + 4) == MISALIGNED and backward(lib, d, dsT=P + 4) == MISALIGNED
    assert backward(lib, d, ds0=P + 4) == MISALIGNED
    assert backward(lib, scan_desc(d_out_stride=(38400, 384, 44))) == MISALIGNED
    d = scan_desc(B=3, T=50, seq_offsets=P + 2)
    assert forward(lib, d) == MISALIGNED and backward(lib, d) == MISALIGNED


def test_scan_workspace(lib):
    d = scan_desc()
    need = lib.gscan_state_scan_backward_workspace_bytes(ctypes.byref(d))
    # the states before and the gradients after each of 2 chunks of 64 tokens, 16 bits, widths 64 x 64,
    # and a factor for each of their tiles of 16 keys
    assert need == 2 * (2 * 2 * 8 * (64 * 64 * 2 + 4 * 4))
    assert backward(lib, d, ws=P, n=need - 1) == WS_SMALL
    assert backward(lib, d, ws=P + 16, n=need) == MISALIGNED
    # short or many sequences are walked whole; one long one is divided
    assert lib.gscan_state_scan_forward_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.gscan_state_scan_forward_workspace_bytes(ctypes.byref(scan_desc(B=64, T=4096))) == 0
    d = scan_desc(B=1, T=50000)
    need = lib.gscan_state_scan_forward_workspace_bytes(ctypes.byref(d))
    assert need >= 2 * 8 * (64 * 48 + 1) * 4
    assert forward(lib, d, ws=P, n=need - 1) == WS_SMALL
    assert forward(lib, d, ws=P + 128, n=need) == MISALIGNED


def test_scan_of_nothing_needs_nothing(lib):
    d = scan_desc(T=0)
    assert forward(lib, d, q=None, k=None, v=None, gate=None, out=None) == OK
    assert backward(lib, d, q=None, k=None, v=None, gate=None, do=None, dq=None, dk=None, dv=None,
                    dg=None) == OK


def test_step_refuses(lib):
    d = scan_desc(T=1, B=4)
    assert step(lib, scan_desc(T=2)) == INVALID
    assert step(lib, scan_desc(T=1, seq_offsets=P)) == INVALID
    for name in ("q", "k", "v", "gate", "state", "out"):
        assert step(lib, d, **{name: None}) == INVALID
        assert step(lib, d, **{name: P + 2}) == MISALIGNED
    assert step(lib, d, slots=P + 2) == MISALIGNED
    assert step(lib, d, pool=0) == INVALID and step(lib, d, pool=3, slots=None) == INVALID
    assert step(lib, scan_desc(T=1, B=2**20, H=16384, Hk=1)) == UNSUPPORTED


def norm_desc(**kw):
    c = dict(tokens=10, Hq=8, Hk=2, D=64, rot=32, dtype=BF, layout=0, pos_int64=1, eps=1e-6, magnitude=1.0)
    c.update({k: v for k, v in kw.items() if k in c})
    d = qn._Desc(**c)
    for name, heads in (("q", c["Hq"]), ("k", c["Hk"]), ("dy_q", c["Hq"]), ("dy_k", c["Hk"])):
        setattr(d, name + "_stride", (ctypes.c_int64 * 2)(heads * c["D"], c["D"]))
    for k, v in kw.items():
        if k.endswith("_stride"):
            setattr(d, k, (ctypes.c_int64 * 2)(*v))
    return d


def norm(lib, d, q=P, k=P, wq=P, wk=P, pos=P, freq=P, yq=P, yk=P):
    return lib.gscan_qk_norm_rope_forward(d and ctypes.byref(d), q, k, wq, wk, pos, freq, yq, yk, None)


def dnorm(lib, d, q=P, k=P, wq=P, wk=P, pos=P, freq=P, gq=P, gk=P, dq=P, dk=P, dwq=P, dwk=P, ws=None, n=0):
    return lib.gscan_qk_norm_rope_backward(d and ctypes.byref(d), q, k, wq, wk, pos, freq, gq, gk, dq, dk,
                                           dwq, dwk, ws, n, None)


@pytest.mark.parametrize("change,want", [
    (dict(tokens=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID), (dict(D=0), INVALID),
    (dict(rot=-8), INVALID), (dict(eps=0.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(dtype=5), INVALID), (dict(layout=2), INVALID),
    (dict(D=68), UNSUPPORTED), (dict(D=264), UNSUPPORTED), (dict(rot=72), UNSUPPORTED),
    (dict(rot=12), UNSUPPORTED), (dict(tokens=2**31), UNSUPPORTED), (dict(Hq=2**20 + 1), UNSUPPORTED),
    (dict(q_stride=(516, 64)), MISALIGNED), (dict(k_stride=(128, 68)), MISALIGNED),
])
def test_norm_refuses_descriptors(lib, change, want):
    d = norm_desc(**change)
    assert norm(lib, d) == want and dnorm(lib, d) == want
    assert lib.gscan_last_error() != b""


def test_norm_refuses_pointers(lib):
    assert norm(lib, None) == INVALID and dnorm(lib, None) == INVALID
    d = norm_desc()
    for name in ("q", "k", "pos", "freq", "yq", "yk"):
        assert norm(lib, d, **{name: None}) == INVALID, name
        assert norm(lib, d, **{name: P + 2}) == MISALIGNED, name
    for name in ("wq", "wk"):
        assert norm(lib, d, **{name: P + 4}) == MISALIGNED, name
    for name in ("gq", "gk", "dq", "dk"):
        assert dnorm(lib, d, **{name: None}) == INVALID, name
        assert dnorm(lib, d, **{name: P + 4}) == MISALIGNED, name
    assert dnorm(lib, d, dwq=P + 2) == MISALIGNED
    assert dnorm(lib, norm_desc(dy_q_stride=(508, 64))) == MISALIGNED
    need = lib.gscan_qk_norm_rope_workspace_bytes(ctypes.byref(d))
    assert 0 < need <= 10 * 2 * 64 * 4
    assert dnorm(lib, d, ws=P, n=need - 1) == WS_SMALL
    assert dnorm(lib, d, ws=P + 64, n=need) == MISALIGNED


def test_norm_of_nothing_needs_nothing(lib):
    d = norm_desc(tokens=0)
    assert norm(lib, d, q=None, k=None, pos=None, freq=None, yq=None, yk=None) == OK


# ------------------------------------------------------------ the binding

GPU = torch.device("cuda", 0)


def layout(*shape, stride=None):
    if stride is None:
        stride, n = [], 1
        for s in reversed(shape):
            stride.insert(0, n)
            n *= s
    return torch.Size(shape), tuple(stride)


def scan_template(q=layout(2, 9, 2, 16), k=None, v=layout(2, 9, 4, 24), gate=layout(2, 9, 4),
                  dtypes=(torch.bfloat16,) * 4, devices=(GPU,) * 4, form="sigmoid", n=0, single=False):
    return ms._Desc.from_buffer_copy(ms._template(q, q if k is None else k, v, gate, dtypes, devices, 0.5,
                                                  form, 0.25, n, single))


def test_scan_descriptor_fields():
    d = scan_template()
    assert (d.B, d.T, d.H, d.Hk, d.Dk, d.Dv) == (2, 9, 4, 2, 16, 24)
    assert tuple(d.q_stride) == (288, 32, 16) and tuple(d.v_stride) == (864, 96, 24)
    assert tuple(d.gate_stride) == (36, 4, 1) and (d.scale, d.gate_shift) == (0.5, 0.25)
    # packed: tokens and heads; a slice of a projection's output keeps its strides
    d = scan_template(layout(9, 2, 16, stride=(512, 16, 1)), None, layout(9, 4, 24, stride=(512, 24, 1)),
                      layout(9, 4, stride=(512, 1)), n=3)
    assert (d.B, d.T) == (3, 9) and tuple(d.q_stride) == (0, 512, 16) and tuple(d.gate_stride) == (0, 512, 1)
    # one token of each request: requests are the batch
    d = scan_template(layout(9, 2, 16), None, layout(9, 4, 24), layout(9, 4), single=True)
    assert (d.B, d.T) == (9, 1) and tuple(d.v_stride) == (96, 0, 24)
    # a dimension of one element has no stride that counts
    d = scan_template(layout(1, 9, 1, 16, stride=(7, 16, 5, 1)), None, layout(1, 9, 4, 24), layout(1, 9, 4))
    assert tuple(d.q_stride) == (0, 16, 0)


@pytest.mark.parametrize("kw,error", [
    (dict(devices=(torch.device("cpu"),) * 4), TypeError),
    (dict(devices=(GPU, GPU, torch.device("cuda", 1), GPU)), ValueError),
    (dict(dtypes=(torch.float16,) * 4), TypeError),
    (dict(dtypes=(torch.bfloat16, torch.float32, torch.bfloat16, torch.float32)), TypeError),
    (dict(dtypes=(torch.bfloat16,) * 3 + (torch.float16,)), TypeError),
    (dict(form="tanh"), ValueError),
    (dict(n=3), ValueError),                                   # packed takes [tokens, heads, width]
    (dict(single=True), ValueError),
    (dict(k=layout(2, 9, 4, 16)), ValueError),
    (dict(v=layout(2, 8, 4, 24)), ValueError),
    (dict(gate=layout(2, 9, 2)), ValueError),
    (dict(v=layout(2, 9, 4, 24, stride=(864, 96, 1, 4))), ValueError),
])
def test_scan_binding_refuses(kw, error):
    with pytest.raises(error):
        scan_template(**kw)


def test_public_calls_refuse_cpu_tensors():
    q, v, a = torch.zeros(1, 4, 2, 16), torch.zeros(1, 4, 2, 16), torch.zeros(1, 4, 2)
    for call in (lambda: gs.state_scan_forward(q, q, v, a), lambda: gs.state_scan(q, q, v, a),
                 lambda: gs.state_scan_backward(q, q, v, a, v),
                 lambda: gs.state_scan_forward_workspace_bytes(q, q, v, a),
                 lambda: gs.state_scan_backward_workspace_bytes(q, q, v, a),
                 lambda: gs.state_scan_step(q[0], q[0], v[0], a[0], torch.zeros(4, 2, 16, 16)),
                 lambda: gs.state_scan_forward(q.numpy(), q, v, a),
                 lambda: gs.qk_norm_rope_forward(q[0], q[0], None, None, None, None),
                 lambda: gs.qk_norm_rope(q[0], None, None, None, None, None),
                 lambda: gs.qk_norm_rope_backward(q[0], None, None, None, None, None, q[0], None)):
        with pytest.raises(TypeError):
            call()


def norm_template(q=layout(5, 4, 32), k=layout(5, 2, 32), qdt=torch.float32, kdt=torch.float32, dev=GPU,
                  kdev=GPU, form="half"):
    return qn._Desc.from_buffer_copy(qn._template(q, k, qdt, kdt, dev, kdev, 1e-6, form, 1.0))


def test_norm_binding():
    d = norm_template()
    assert (d.tokens, d.Hq, d.Hk, d.D, d.rot) == (5, 4, 2, 32, 0) and tuple(d.q_stride) == (128, 32)
    assert norm_template(k=None, kdt=None, kdev=None).Hk == 0
    for kw, error in ((dict(dev=torch.device("cpu")), TypeError), (dict(kdev=torch.device("cuda", 1)), ValueError),
                      (dict(form="none"), ValueError), (dict(qdt=torch.float16), TypeError),
                      (dict(kdt=torch.bfloat16), ValueError), (dict(k=layout(4, 2, 32)), ValueError),
                      (dict(k=layout(5, 2, 24)), ValueError), (dict(k=layout(5, 0, 32)), ValueError),
                      (dict(q=layout(5, 4, 32, stride=(128, 1, 4))), ValueError), (dict(q=layout(5, 32)), ValueError)):
        with pytest.raises(error):
            norm_template(**kw)


# --------------------------------------------------------- rotary frequencies

def test_frequencies_plain_linear_base():
    f, m = gs.rotary_frequencies(64)
    assert f.dtype == torch.float32 and f.shape == (32,) and m == 1.0
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert torch.equal(f, want.float())
    f, m = gs.rotary_frequencies(64, base=500000.0, scaling="linear", factor=8.0)
    want = torch.tensor([500000.0 ** (-2 * i / 64) / 8 for i in range(32)], dtype=torch.float64)
    assert torch.equal(f, want.float()) and m == 1.0
    # the fastest pair as before, the slowest divided by the factor (each rounded once to float32)
    f, _ = gs.rotary_frequencies(64, scaling="base", factor=4.0)
    slow = 10000.0 ** (-62 / 64) / 4
    assert f[0] == 1.0 and abs(float(f[-1]) - slow) <= 2.0 ** -24 * slow + 1e-15


def test_frequencies_by_parts():
    rot, base, factor, length = 64, 10000.0, 4.0, 2048
    f, m = gs.rotary_frequencies(rot, base, "parts", factor, length, 32.0, 1.0)
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
    assert m == 0.1 * math.log(factor) + 1.0
    for i, p in enumerate(plain):
        turns = length * p / (2 * math.pi)
        # the ramp's ends are whole pairs, at most one pair outside the two turn counts
        if turns > 32.0 * base ** (2 / rot):
            assert abs(float(f[i]) - p) <= 2.0 ** -24 * p
        elif turns < 1.0 / base ** (2 / rot):
            assert abs(float(f[i]) - p / factor) <= 2.0 ** -24 * p / factor
        assert p / factor * (1 - 2.0 ** -23) <= float(f[i]) <= p * (1 + 2.0 ** -23)
    assert all(x > y for x, y in zip(f.tolist(), f.tolist()[1:]))
    # a factor of one changes nothing
    f1, m1 = gs.rotary_frequencies(rot, base, "parts", 1.0, length)
    assert m1 == 1.0 and torch.allclose(f1.double(), torch.tensor(plain, dtype=torch.float64), rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=8, base=1.0), dict(rot=8, factor=0.5),
                                dict(rot=8, scaling="other"), dict(rot=2, scaling="base"),
                                dict(rot=8, base=math.nan)])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        gs.rotary_frequencies(**kw)
