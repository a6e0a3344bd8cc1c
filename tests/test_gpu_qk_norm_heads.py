"""The query/key norm with few heads, one in all among them, where several
tokens share a workgroup and their rows are divided into tokens and heads by a
multiplier.  Tolerances are those of test_gpu_qk_norm.py, which do not depend
on heads or tokens."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests import state_ref as sr
from tests.test_gpu_qk_norm import BF, DEV, F32, TOL, call_args, close, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D", [8, 64, 72, 128, 256])
@pytest.mark.parametrize("Hq,Hk", [(1, 0), (1, 1), (2, 0), (3, 0)])
@pytest.mark.parametrize("n", [1, 29])
def test_few_heads(n, Hq, Hk, D, layout, dtype):
    print(f"case norm, few heads: {n} tokens, {Hq} + {Hk} heads of {D} {layout} {dtype}", flush=True)
    m = make(n, Hq, Hk, D, 8, dtype)
    args, kw = call_args(m), dict(eps=1e-5, layout=layout)
    out = gs.qk_norm_rope_forward(*args, **kw)
    dy = [None if x is None else x.to(DEV) for x in m["dy"]]
    g = gs.qk_norm_rope_backward(*args, *dy, **kw)
    torch.cuda.synchronize()
    pos, freq = m["pos"].numpy(), m["freq"].numpy()
    for i in range(2 if Hk else 1):
        x, w = m["host"][i].double().numpy(), m["w"][i].double().numpy()
        close(out[i], sr.norm_rope(x, w, pos, freq, 1e-5, layout), TOL[dtype], f"y{i}")
        dx, dw = sr.norm_rope_grad(x, w, pos, freq, m["dy"][i].double().numpy(), 1e-5, layout)
        close(g[i], dx, TOL[dtype], f"dx{i}")
        close(g[2 + i], dw, 32 * 2.0 ** -24, f"dw{i}")
    if not Hk:
        assert out[1] is None and g[1] is None and g[3] is None
