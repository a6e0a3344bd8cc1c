"""The token embedding (gscan_embed_*, through the package) against its 64-bit form.

Tolerances.  Forward: one product, rounded once to the output's type: equal to the
float32 product rounded, bit by bit.  Backward: a row's sum in float32 in the order of
the positions, in chunks: of n terms sqrt(n) / 2 roundings' size; four times that of
the norm (lm_ref.product with K = n terms holds it), and one rounding to bf16."""
import pytest
import torch

import gated_linear_recurrence_history_amd as gs
from tests import lm_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def tokens_of(n, vocabulary, gen, often=0.3):
    """Some outside the vocabulary, one that is frequent, runs in the middle."""
    t = torch.randint(-2, vocabulary + 2, (n,), generator=gen)
    t[torch.rand(n, generator=gen) < often] = vocabulary // 2
    t[n // 3:n // 2] = vocabulary - 1
    return t


CASES = {  # tokens, vocabulary, width
    "one": (1, 5, 8),
    "one row": (9, 1, 16),
    "a chunk": (8, 40, 24),
    "chunks end inside runs": (131, 7, 200),
    "one sort": (777, 1003, 136),
    "wide": (300, 64, 1544),
    "widest": (3, 4, 65536),
    "several keys a lane": (5000, 300, 72),
    "largest single sort": (16384, 32000, 64),
    "sort of two workgroups": (16385, 70000, 16),
    "large vocabulary": (100, 2 ** 18, 8),
    "three digits": (20000, 2 ** 17, 8),
    "a frequent token": (70001, 3, 24),
    "many workgroups": (600001, 256, 8),
    # up to 2048 tokens (wide rows: 64) at once, up to 32768 of fewer than 2^20 rows sorted by one launch
    "a wavefront's own row": (32, 1, 24),
    "a shared row": (33, 1, 24),
    "most at once": (2048, 5, 512),
    "one more": (2049, 5, 512),
    "most at once, 256 rows a workgroup": (2048, 65535, 8),
    "most wide rows at once": (64, 300, 4096),
    "one more wide row": (65, 300, 520),
    "wider rows": (64, 7, 4104),
    "most in one sort": (32768, 1003, 8),
    "one more than one sort": (32769, 1003, 8),
    "most in one sort, many rows": (32767, 2 ** 19, 8),
    "one more than that": (32768, 2 ** 19, 8),
    "eight workgroups' blocks": (65536, 1003, 8),
    "one more than those": (65537, 1003, 8),
    "most rows of one sort": (3000, 2 ** 20 - 1, 8),
    "one more row": (50, 2 ** 20, 8),
}


@pytest.mark.parametrize("table_dtype,dtype", [(F32, BF), (BF, F32), (F32, F32), (BF, BF)])
@pytest.mark.parametrize("name", CASES)
def test_forward_and_backward(name, table_dtype, dtype):
    n, V, D = CASES[name]
    print(f"case embed: {name} {table_dtype} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(4)
    t = tokens_of(n, V, gen).to(torch.int32 if n % 2 else torch.int64)
    table = torch.randn(V, D + 8, generator=gen).to(table_dtype).to(DEV)[:, 8:]  # rows of a wider matrix
    y = gs.embed_forward(table, t.to(DEV), scale=1.5, dtype=dtype)
    ok = ((t >= 0) & (t < V)).to(DEV)
    want = torch.where(ok[:, None], table.float()[t.to(DEV).clamp(0, V - 1).long()] * 1.5, torch.zeros((), device=DEV))
    assert torch.equal(y, want.to(dtype))

    d = torch.randn(n, D, generator=gen).to(dtype).to(DEV)
    out = torch.full((V, D), float("nan"), dtype=table_dtype, device=DEV)  # every row is written
    g = gs.embed_backward(d, t.to(DEV), V, scale=0.5, dtype=table_dtype, out=out)
    assert g is out
    assert torch.equal(g, gs.embed_backward(d, t.to(DEV), V, scale=0.5, dtype=table_dtype))
    exact = torch.zeros(V, D, dtype=torch.float64, device=DEV)
    exact.index_add_(0, t.to(DEV)[ok].long(), d[ok].double())
    ref.close(g, exact * 0.5, ref.product(n) + ref.rounding(table_dtype), "gradient")
    absent = torch.ones(V, dtype=torch.bool, device=DEV)
    absent[t.to(DEV)[ok].long()] = False
    assert bool((g[absent] == 0).all())


def test_shapes_and_order():
    """A batch of sequences; the gradient of one token is the sum in the order of its positions."""
    gen = torch.Generator().manual_seed(5)
    t = torch.randint(0, 50, (3, 4, 7), generator=gen)
    table = torch.randn(50, 40, generator=gen)
    y = gs.embed_forward(table.to(DEV), t.to(DEV), scale=2.0)
    ref.close(y, ref.embed(table, t, 2.0), 2.0 ** -23, "rows")
    d = torch.randn(3, 4, 7, 40, generator=gen)
    ref.close(gs.embed_backward(d.to(DEV), t.to(DEV), 50), ref.embed_grad(d, t, 50, 1.0), ref.product(84), "gradient")
    one = torch.zeros(6, dtype=torch.int64, device=DEV)
    big = torch.tensor([2.0 ** 24, 1.0, -2.0 ** 24, 1.0, 1.0, 1.0], device=DEV)[:, None].expand(6, 8).contiguous()
    assert gs.embed_backward(big, one, 1)[0, 0] == 3.0  # 2^24 + 1 is 2^24: in order, the first 1 is lost


def test_nothing():
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    table = torch.ones(5, 16, device=DEV)
    assert gs.embed_forward(table, t).shape == (0, 16)
    assert bool((gs.embed_backward(torch.empty(0, 16, device=DEV), t, 5) == 0).all())
    outside = torch.tensor([-1, 5, 2 ** 40, -2 ** 40], device=DEV)
    assert bool((gs.embed_forward(table, outside) == 0).all())
    assert bool((gs.embed_backward(torch.ones(4, 16, device=DEV), outside, 5) == 0).all())


def test_nonfinite_rows_stay_alone():
    t = torch.tensor([3, 1, 3, 0, 9], device=DEV)
    table = torch.ones(4, 24, device=DEV)
    table[3, 5] = float("nan")
    y = gs.embed_forward(table, t)
    assert bool(torch.isnan(y[[0, 2], 5]).all()) and int(torch.isnan(y).sum()) == 2
    d = torch.ones(5, 24, device=DEV)
    d[4] = float("nan")  # padding
    d[1, 7] = float("inf")
    g = gs.embed_backward(d, t, 4)
    assert bool(torch.isinf(g[1, 7])) and int(torch.isfinite(g).sum()) == 4 * 24 - 1


def test_table_past_32_bits():
    V, D = 300001, 8192  # 4.9 GB
    table = torch.zeros(V, D, dtype=BF, device=DEV)
    table[-1], table[-2, 5] = 3.0, 7.0
    t = torch.tensor([V - 1, 0, V - 2], device=DEV)
    y = gs.embed_forward(table, t)
    assert bool((y[0] == 3).all()) and bool((y[1] == 0).all()) and float(y[2, 5]) == 7.0 and float(y[2].sum()) == 7.0
    d = torch.full((3, D), 2.0, dtype=BF, device=DEV)
    g = gs.embed_backward(d, t, V, out=table)
    assert bool((g[-1] == 2).all()) and bool((g[-2] == 2).all()) and bool((g[0] == 2).all())
    assert float(g[1:-2].abs().amax()) == 0.0


def test_gradient_of_more_rows_than_a_launch_has_threads():
    V, D = 2 ** 30 + 65, 8
    t = torch.tensor([0, V - 1, 2 ** 30, V - 1], device=DEV)
    d = torch.ones(4, D, dtype=BF, device=DEV)
    out = torch.full((V, D), float("nan"), dtype=BF, device=DEV)
    gs.embed_backward(d, t, V, out=out)
    assert out[0, 0] == 1 and out[2 ** 30, 0] == 1 and out[V - 1, 0] == 2
    out[t] = 0
    step = 2 ** 27
    assert all(bool((out[i:i + step] == 0).all()) for i in range(0, V, step))


def test_more_tokens_than_a_launch_has_groups():
    n, D = 2 ** 30 + 1025, 8  # 1024 tokens a workgroup
    table = torch.randn(3, D, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    t = (torch.arange(n, device=DEV, dtype=torch.int32) % 4) - 1
    y = gs.embed_forward(table, t)
    want = torch.cat([torch.zeros(1, D, dtype=BF, device=DEV), table])
    step = 2 ** 26
    for i in range(0, n, step):
        part = y[i:i + step]
        assert torch.equal(part[:len(part) // 4 * 4].view(-1, 4, D), want.expand(len(part) // 4, 4, D))
    assert torch.equal(y[-1], want[(n - 1) % 4])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_autograd(dtype):
    gen = torch.Generator().manual_seed(6)
    base = torch.randn(30, 45, generator=gen).to(DEV)
    t = torch.randint(0, 30, (4, 9), generator=gen).to(DEV)
    for table in (base[:, :40].contiguous(), base[:, 3:43]):  # the second on no multiple of 16 bytes
        leaf = table.detach().requires_grad_()
        y = gs.embed(leaf, t, scale=3.0, dtype=dtype)
        assert torch.equal(y, (leaf.detach()[t] * 3.0).to(dtype))
        d = torch.randn(y.shape, generator=gen).to(dtype).to(DEV)
        y.backward(d.transpose(0, 1).contiguous().transpose(0, 1))  # strides of its own
        assert leaf.grad.dtype == F32
        ref.close(leaf.grad, ref.embed_grad(d.cpu(), t.cpu(), 30, 3.0), ref.product(36), "gradient")
    frozen = gs.embed(base[:, :40].contiguous(), t)
    assert not frozen.requires_grad


def test_a_batch_without_its_last_tokens():
    gen = torch.Generator().manual_seed(7)
    table = torch.randn(11, 16, generator=gen).to(DEV).requires_grad_()
    t = torch.randint(0, 11, (3, 9), generator=gen).to(DEV)
    y = gs.embed(table, t[:, :-1])
    assert torch.equal(y, table.detach()[t[:, :-1]])
    y.sum().backward()
    assert torch.equal(table.grad[:, 0].long(), torch.bincount(t[:, :-1].reshape(-1), minlength=11))
    with pytest.raises(ValueError):
        gs.embed_forward(table.detach(), t[:, :-1])


def test_other_stream_and_graph():
    gen = torch.Generator(device=DEV).manual_seed(7)
    t = torch.randint(0, 90, (2500,), generator=gen, device=DEV)
    table, d = torch.randn(90, 64, generator=gen, device=DEV), torch.randn(2500, 64, generator=gen, device=DEV)
    ws = torch.empty(gs.embed_backward_workspace_bytes(d, t, 90), dtype=torch.uint8, device=DEV)

    def work(stream=None):
        return (gs.embed_forward(table, t, dtype=BF, stream=stream),
                gs.embed_backward(d, t, 90, workspace=ws, stream=stream))

    a = work()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = work(s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for _ in range(3):
        d.copy_(torch.randn(2500, 64, device=DEV))
        t.copy_(torch.randint(-1, 91, (2500,), device=DEV))
        torch.randn(1 << 16, device=DEV).add_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        assert all(torch.equal(x, y) for x, y in zip(got, work()))


def test_refusals():
    table, t = torch.zeros(5, 16, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    for bad in (dict(table=table.half()), dict(dtype=torch.float16), dict(tokens=t.float()),
                dict(tokens=t.cpu()), dict(table=table.T), dict(out=torch.zeros(3, 8, device=DEV))):
        args = dict(table=table, tokens=t, **{k: v for k, v in bad.items() if k not in ("table", "tokens")})
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            gs.embed_forward(**args)
    with pytest.raises(gs.GScanError):
        gs.embed_forward(torch.zeros(5, 12, device=DEV), t)
    with pytest.raises(gs.GScanError):
        gs.embed_forward(torch.zeros(5, 24, device=DEV)[:, 2:18], t)
    d = torch.zeros(3, 16, device=DEV)
    with pytest.raises(ValueError):
        gs.embed_backward(d[:2], t, 5)
    for V in (0, -1):
        with pytest.raises(gs.GScanError):
            gs.embed_backward(d, t, V)
    many, dmany = t.repeat(1000), d.repeat(1000, 1)  # few tokens need no workspace
    with pytest.raises((ValueError, gs.GScanError)):
        gs.embed_backward(dmany, many, 5, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
