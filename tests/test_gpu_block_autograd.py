"""The recorded norm, activation, attention and convolution calls: what they keep, and what they refuse."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def recorded():
    g = gen(1)
    x, r, w = randn(g, 6, 64), randn(g, 6, 64), randn(g, 64)
    q, k, v = (randn(g, 2, 5, 2, 16) for _ in range(3))
    ld = -torch.ones(2, device="cuda")
    cx, cw = randn(g, 2, 8, 9), randn(g, 8, 4, 4)
    return {"norm": ((x, w), lambda x, w: ct.rms_norm_autograd(x, w)),
            "norm with residual": ((x, w, r), lambda x, w, r: sum(ct.rms_norm_autograd(x, w, r))),
            "activation": ((x, r), lambda x, r: ct.checkpointed_activation_autograd(x, r)),
            "attention": ((q, k, v), lambda q, k, v: ct.linear_attention_autograd(q, k, v, ld)[0]),
            "convolution": ((cx, cw), lambda x, w: ct.conv_transpose_autograd(x, w, stride=2)),
            "convolution, kept": ((cx, cw), lambda x, w: ct.conv_transpose_autograd(x, w, stride=2, checkpoint="int8"))}


@pytest.mark.parametrize("name", ["norm", "norm with residual", "activation", "attention", "convolution", "convolution, kept"])
def test_a_second_derivative_is_refused(name):
    """A penalty on a gradient next to another loss: an error, not the other loss's gradient alone."""
    inputs, f = recorded()[name]
    leaves = [t.clone().requires_grad_() for t in inputs]
    first = torch.autograd.grad(f(*leaves).square().sum(), leaves, create_graph=True)
    for grad in first:
        loss = sum(t.square().sum() for t in leaves)
        loss.backward(retain_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (loss + grad.square().sum()).backward(retain_graph=True)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("positions", [4, 300])
def test_what_the_convolution_keeps(positions, quant):
    """8-bit codes and a scale for each 128 positions of a channel where dw is asked for, nothing of x where it is not."""
    g = gen(3)
    x, w = randn(g, 3, 16, positions, dtype="bf16"), randn(g, 16, 8, 4, dtype="bf16")
    dy = randn(g, 3, 8, 2 * positions, dtype="bf16")
    grads = {}
    for dw in (True, False):
        leaf, weight = x.clone().requires_grad_(), w.clone().requires_grad_(dw)
        y = ct.conv_transpose_autograd(leaf, weight, stride=2, padding=1, checkpoint=quant)
        kept = [t for t in y.grad_fn.saved_tensors if t is not None and t.data_ptr() != weight.data_ptr()]
        assert sum(t.numel() * t.element_size() for t in kept) == (3 * 16 * (positions + 4 * -(-positions // 128)) if dw else 0)
        y.backward(dy)
        grads[dw] = leaf.grad
        assert (weight.grad is not None) == dw
    assert torch.equal(grads[True], grads[False])
