"""The activations of checkpointed inputs in fp32 over the whole range of their exponentials."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import E, act_ref, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


@pytest.mark.parametrize("cols", [4096, 4099])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_fp32_sigmoid_is_good_to_its_roundings(act, cols):
    """Also where it is smallest: exp is good to 2 units in the last place, the sum, the quotient and the product to half of one
    each (subnormal results to a step of 2^-149); down to where exp(-x) leaves the type."""
    x = torch.linspace(-88.5, 88.5, 8 * cols, device="cuda").view(8, cols)
    y, kept, _ = ct.checkpointed_activation(x, activation=act)
    ref = act_ref(x.double(), act)
    off = (y.double() - ref).abs() - (ref.abs() * 8 * E + 90 * 2.0 ** -149)
    assert off.max().item() <= 0
    # the gradient's own: codes 1 and a scale for each 32 values of x
    codes = torch.ones(8, cols, dtype=torch.int8, device="cuda")
    scales = x[:, ::32].contiguous()
    again = ct.checkpointed_activation_backward(None, ct.Checkpoint(codes, scales, 32, torch.float32), activation=act, need=("y",))[2]
    ref = act_ref(scales.double(), act).repeat_interleave(32, 1)[:, :cols]
    off = (again.double() - ref).abs() - (ref.abs() * 8 * E + 90 * 2.0 ** -149)
    assert off.max().item() <= 0
