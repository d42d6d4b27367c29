"""NaN through the activations: no operator answers with a finite number for it."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn

pytestmark = pytest.mark.gpu
ACTS = [None, "relu", "leaky_relu", "silu", "gelu", "tanh", "sigmoid"]


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("shape", [(2, 40, 64), (2, 40, 63), (1, 70000, 64), (3, 20000, 33)], ids=str)  # in one pass, in two; vectors, single values
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_group_that_is_not_finite(act, bad, shape, dtype):
    """It is NaN throughout, its gradient too; the others are as without it."""
    g = gen(1)
    B, S, C = shape
    G = 8 if C == 64 else 3
    n = C // G
    x, w, b, dy = randn(g, *shape, dtype=dtype), randn(g, C, dtype=dtype), randn(g, C, dtype=dtype), randn(g, *shape, dtype=dtype)
    clean, mean, rstd = ct.group_norm(x, G, w, b, activation=act, alpha=0.0)
    want = ct.group_norm_backward(dy, x, mean, rstd, w, b, act, 0.0)
    x[0, S // 2, n] = bad  # a value of sample 0, group 1
    y, mean, rstd = ct.group_norm(x, G, w, b, activation=act, alpha=0.0)
    dx, dw, db = ct.group_norm_backward(dy, x, mean, rstd, w, b, act, 0.0)
    for got, ref in ((y, clean), (dx, want[0])):
        assert torch.isnan(got[0, :, n:2 * n]).all()
        got, ref = got.clone(), ref.clone()
        got[0, :, n:2 * n] = ref[0, :, n:2 * n] = 0
        assert torch.equal(got, ref)
    assert torch.isnan(dw[n:2 * n]).all()
    if act is not None:
        assert torch.isnan(db[n:2 * n]).all()
    for got, ref in ((dw, want[1]), (db, want[2])):
        assert torch.equal(got[:n], ref[:n]) and torch.equal(got[2 * n:], ref[2 * n:])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [1, 3, 40, 200])  # without tiles, on one SM a tile, on pairs
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_gate_that_is_not_a_number(act, rows, layout, dtype):
    """A NaN in one column of the gate's weights: that column of y, and all of dx and that column's gradients."""
    g = gen(2)
    x, dy = randn(g, rows, 64, dtype=dtype), randn(g, rows, 96, dtype=dtype)
    wg, wu = (randn(g, 64, 96, std=0.125, dtype=dtype) if layout == "in_out" else randn(g, 96, 64, std=0.125, dtype=dtype).t() for _ in range(2))
    clean = ct.gated_projection(x, wg, wu, act, 0.0)
    want = ct.gated_projection_backward(dy, x, wg, wu, act, 0.0)
    wg[7, 11] = float("nan")
    y = ct.gated_projection(x, wg, wu, act, 0.0)
    dx, dwg, dwu = ct.gated_projection_backward(dy, x, wg, wu, act, 0.0)
    assert torch.isnan(y[:, 11]).all() and torch.isnan(dx).any(1).all() and torch.isnan(dwu[:, 11]).all()
    if act is not None:
        assert torch.isnan(dwg[:, 11]).all()
    for got, ref in ((y, clean), (dwg, want[1]), (dwu, want[2])):
        got, ref = got.clone(), ref.clone()
        got[:, 11] = ref[:, 11] = 0
        assert torch.equal(got, ref)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("cols", [64, 33])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_checkpointed_activation_of_not_a_number(act, cols, dtype):
    g = gen(3)
    gate, up, dy = (randn(g, 5, cols, dtype=dtype) for _ in range(3))
    gate[2, 3] = float("nan")
    act = act or "none"
    y, kept_gate, kept_up = ct.checkpointed_activation(gate, up, act, 0.0, "int8", 32)
    assert torch.isnan(y[2, 3]) and torch.isnan(y).sum() == 1
    dgate, dup = ct.checkpointed_activation_backward(dy, kept_gate, kept_up, act, 0.0)
    # what is kept of the group is NaN throughout
    assert torch.isnan(dup[2, :32]).all() and torch.isnan(dup).sum() == 32
    if act != "none":
        assert torch.isnan(dgate[2, :32]).all() and torch.isnan(dgate).sum() == 32
