"""Sizes and layouts that the binding of the gated projection works out for itself (no GPU needed)."""
import pytest
import torch

from transposed_convolution_convtranspose1_gb300 import block


@pytest.mark.parametrize("shape", [(0,), (5, 0), (0, 0), (2, 3, 0), (2, 0, 4), (0, 3, 7), (6,), (2, 3, 4, 5)], ids=str)
def test_rows_are_the_leading_axes(shape):
    rows = 1
    for n in shape[:-1]:
        rows *= n
    assert tuple(block._extent(torch.empty(shape))) == (rows, shape[-1])
