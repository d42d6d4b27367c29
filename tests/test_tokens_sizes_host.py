"""Sizes and layouts that the binding of the gated projection works out for itself (no GPU needed)."""
import ctypes

import pytest
import torch

from transposed_convolution_convtranspose1_gb300 import block


@pytest.mark.parametrize("shape", [(0,), (5, 0), (0, 0), (2, 3, 0), (2, 0, 4), (0, 3, 7), (6,), (2, 3, 4, 5)], ids=str)
def test_rows_are_the_leading_axes(shape):
    rows = 1
    for n in shape[:-1]:
        rows *= n
    assert tuple(block._extent(torch.empty(shape))) == (rows, shape[-1])


@pytest.fixture(scope="module")
def workspace():
    from transposed_convolution_convtranspose1_gb300 import _build
    from transposed_convolution_convtranspose1_gb300 import ct as ctb
    _build.build_library()

    def bytes_of(rows, C, F, dtype, aligned, backward=0):
        n = ctypes.c_size_t(1)
        assert ctb.lib().ct_gated_projection_workspace_bytes(rows, C, F, dtype, backward, aligned, ctypes.byref(n)) == ctb.CT_OK
        return n.value
    return bytes_of


ALIGNED, BY_F, BY_C = 1, 2, 4


@pytest.mark.parametrize("dtype,most", [(0, 16), (1, 4), (2, 4)])
def test_few_rows_ask_for_no_workspace(workspace, dtype, most):
    """As many rows as go past the tensor cores, with weights in place; one more, or other weights, and it is as before."""
    for rows in (1, 2, most):
        for layout in (BY_F, BY_C):
            assert workspace(rows, 2048, 8192, dtype, layout | ALIGNED) == workspace(rows, 2048, 8192, dtype, layout) == 0
        assert workspace(rows, 2048, 8192, dtype, 0) > 2 * 2048 * 8192 * 2
        assert workspace(rows, 2048, 8192, dtype, layout | ALIGNED, backward=1) > 0
    for layout in (BY_F, BY_C):
        assert workspace(most + 1, 2048, 8192, dtype, layout | ALIGNED) == workspace(most + 1, 2048, 8192, dtype, ALIGNED) > 0
    # rows of the weights that end inside a vector go to the tensor cores: F in one layout, C in the other
    assert workspace(1, 2048, 8196, dtype, BY_F) > 0 == workspace(1, 2048, 8196, dtype, BY_C)
    assert workspace(1, 2050, 8192, dtype, BY_C) > 0 == workspace(1, 2050, 8192, dtype, BY_F)
