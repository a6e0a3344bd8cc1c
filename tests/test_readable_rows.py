"""What the binding takes for readable in place of an upstream gradient: the last
dimension contiguous, rows on 16 bytes.  Anything else becomes a dense copy (no
GPU)."""
import pytest
import torch

from gated_linear_recurrence_history_amd.matrix_state import _readable


@pytest.mark.parametrize("dtype,columns", [(torch.bfloat16, 8), (torch.float32, 4)])
def test_rows(dtype, columns):
    wide = torch.arange(6 * 52 * columns, dtype=torch.float32).remainder(97).to(dtype).view(6, 52 * columns)
    width = 16 * columns

    def part(x, at):  # [6, 2, width] behind `at` columns of a wider row
        return x[:, at:at + 2 * width].unflatten(1, (2, width))

    ok = [part(wide, 0), part(wide, columns), part(wide, 3 * columns)[:, :1], wide.new_empty(0, 2, width),
          part(wide, 0)[:1].expand(6, 2, width), part(wide, 0).transpose(0, 1)]
    for x in ok:
        assert _readable(x, x) is x
    odd = wide[:, :-4 if dtype == torch.bfloat16 else -2].contiguous()  # rows of 8 bytes' multiple
    flat = wide.reshape(-1)[1:1 + 4 * width].view(2, 2, width)  # dense, its first byte on no 16
    bad = [part(wide, 1), part(odd, 0), part(odd, columns), flat, part(wide, 0).transpose(1, 2)]
    for x in bad:
        y = _readable(x, x)
        assert y is not x and y.is_contiguous() and y.data_ptr() % 16 == 0 and torch.equal(x, y)
    one = part(odd, 0)[:1]  # a single row has no stride that counts
    assert _readable(one, one) is one
