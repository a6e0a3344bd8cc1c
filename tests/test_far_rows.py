"""Rows further apart than the library reads them: the differentiable calls' operands
become dense copies there, and only there (no GPU)."""
import pytest
import torch

from gated_linear_recurrence_history_amd import embedding, matrix_state

FAR = 2 ** 21  # elements between rows of the matrix products' operands, at most


def rows(stride, n=2, width=16, dtype=torch.bfloat16):
    return torch.arange(stride * (n - 1) + width, dtype=torch.int32).remainder_(97).to(dtype).as_strided(
        (n, width), (stride, 1))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_the_products(dtype):
    far = rows(FAR + 8, dtype=dtype)
    y = embedding._product_rows(far)
    assert y is not far and y.is_contiguous() and y.data_ptr() % 16 == 0 and torch.equal(far, y)
    last = torch.zeros(3, 2049, 1024, dtype=dtype)[:, -1]  # the last token of each sequence
    y = embedding._product_rows(last)
    assert y is not last and y.is_contiguous()
    for x in (rows(FAR, dtype=dtype), rows(FAR + 8, dtype=dtype)[:1], rows(64, dtype=dtype),
              rows(8, dtype=dtype)[:1].expand(5, 16)):
        assert embedding._product_rows(x) is x
    assert not embedding._product_rows(rows(FAR + 8, dtype=dtype)[:, 1:9]).storage_offset()
    assert embedding._product_rows(None) is None


def test_rows_of_the_embedding():
    """Its own limit is 2^31; these tensors have no memory."""
    x = torch.empty_strided((2, 16), (2 ** 31, 1), dtype=torch.bfloat16, device="meta")
    assert embedding._rows(x) is x
    x = torch.empty_strided((2, 16), (2 ** 31 + 8, 1), dtype=torch.bfloat16, device="meta")
    assert embedding._rows(x).is_contiguous()


def test_operands_of_other_layers_stay():
    x = rows(FAR + 8)
    assert matrix_state._readable(x, x) is x


def test_a_number_is_refused_as_the_calls_refuse_it():
    """No dimension at all: left to the checks, whose error it is."""
    x = torch.tensor(1.0)
    assert embedding._rows(x) is x
