"""What the recorded norm, activation and attention calls refuse (no GPU needed)."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct


def test_decays_that_ask_for_a_gradient_are_refused():
    q, ld = torch.zeros(1, 5, 2, 8), (-torch.ones(2)).requires_grad_()
    with pytest.raises(ct.CtError, match="detach"):
        ct.linear_attention_autograd(q, q, q, ld)
    for call in (lambda: ct.linear_attention_autograd(q, q, q, ld.detach()), lambda: no_grad(q, ld)):
        with pytest.raises(ct.CtError, match="device tensors"):  # as far as these get without a device
            call()


def no_grad(q, ld):
    with torch.no_grad():
        ct.linear_attention_autograd(q, q, q, ld)


@pytest.mark.parametrize("checkpoint", ["int4", "none"])
@pytest.mark.parametrize("dw", [False, True])
def test_formats_of_the_kept_input(checkpoint, dw):
    x, w = torch.zeros(1, 2, 8, requires_grad=True), torch.zeros(2, 2, 4, requires_grad=dw)
    with pytest.raises(ct.CtError, match="int8"):
        ct.conv_transpose_autograd(x, w, checkpoint=checkpoint)
