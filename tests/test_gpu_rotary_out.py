"""Rotary positions written into tensors that autograd knows."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn
from _tokens import check_rotary


def test_out_that_asks_for_a_gradient_is_refused():
    """No device is reached: the values would change behind autograd's back, the gradient pass through as if they had not."""
    q, pos, table = torch.zeros(1, 5, 2, 8), torch.zeros(5, 1, dtype=torch.int32), ct.rotary_table((4,), device="cpu")
    leaf = q.clone().requires_grad_()
    inner = leaf * 2
    for out, k in (((leaf, None), None), ((inner, None), None), ((q, leaf), q), ((leaf, q), q)):
        with pytest.raises(ct.CtError, match="gradient"):
            ct.rotary(q, k, pos, table, out=out)
    with torch.no_grad(), pytest.raises(ct.CtError, match="device tensors"):  # as far as it gets without a device
        ct.rotary(q, None, pos, table, out=(leaf, None))
    with pytest.raises(ct.CtError, match="device tensors"):
        ct.rotary(leaf, None, pos, table, out=(q, None))


@pytest.mark.gpu
def test_a_tensor_kept_for_a_backward_pass():
    need_gpu()
    g = gen(1)
    q, k, w = randn(g, 2, 5, 3, 16), randn(g, 2, 5, 1, 16), randn(g, 16).requires_grad_()
    pos, table = torch.arange(5, device="cuda")[:, None], ct.rotary_table((8,))
    start = q.clone()
    loss = (q * w).sum()  # keeps q
    assert ct.rotary(q, k, pos, table, out=(q, k))[0] is q
    check_rotary(start, pos, table, False, False, "f32", q)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        a = start.clone()
        ct.rotary(a, None, pos, table, out=(a, None))
    assert torch.equal(a, q)
    leaf = start.clone().requires_grad_()
    with torch.no_grad():
        ct.rotary(leaf, None, pos, table, out=(leaf, None))
    assert torch.equal(leaf, q)
