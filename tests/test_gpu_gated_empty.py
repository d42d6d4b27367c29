"""The gated projection of rows without channels."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import DT, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


@pytest.mark.parametrize("shape", [(3, 0), (2, 3, 0), (1, 0), (2, 2, 2, 0)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_channels(shape, dtype):
    """y is act(0) * 0 in every row, whatever memory it lands in."""
    w = torch.empty(0, 48, dtype=DT[dtype], device="cuda")
    x = torch.empty(shape, dtype=DT[dtype], device="cuda")
    for _ in range(3):
        dirt = [torch.full((*shape[:-1], 48), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(4)]
        del dirt
        y = ct.gated_projection(x, w, w)
        assert y.shape == (*shape[:-1], 48) and not y.any()
    dx, dwg, dwu = ct.gated_projection_backward(y, x, w, w)
    assert dx.shape == shape and dwg.shape == dwu.shape == (0, 48)
