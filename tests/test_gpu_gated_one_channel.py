"""The gated projection of one channel or to one column: an axis of one value counts as dense whatever its stride."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn
from _tokens import check_gated, check_gated_back

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def spread(g, C, F, rows, cols, dtype):
    """[C, F] with `rows` and `cols` elements between its neighbours."""
    return randn(g, (C - 1) * rows + (F - 1) * cols + 1, dtype=dtype).as_strided((C, F), (rows, cols))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 5, 150])
@pytest.mark.parametrize("C,F", [(1, 64), (1, 5), (64, 1), (1, 1)])
@pytest.mark.parametrize("gate,up", [((64, 1), (512, 8)), ((512, 8), (64, 1)), ((64, 1), (1, 1)), ((1, 64), (8, 1)), ((8, 64), (3, 64)),
                                     ((8, 1), (1, 16)), ((1, 16), (1, 1))], ids=str)
def test_strides_of_an_axis_of_one(dtype, rows, C, F, gate, up):
    g = gen(rows + C)
    x, dy = randn(g, rows, C, dtype=dtype), randn(g, rows, F, dtype=dtype)
    wg, wu = spread(g, C, F, *gate, dtype), spread(g, C, F, *up, dtype)
    check_gated(x, wg, wu, "silu", dtype, ct.gated_projection(x, wg, wu))
    check_gated_back(dy, x, wg, wu, "silu", dtype, *ct.gated_projection_backward(dy, x, wg, wu))
