"""8-bit checkpoints, the activation that keeps them and its gradient from them, against the format's rule and 64 bits."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import DT, E, TINY, U, act_ref, decoded, gen, need_gpu, q8_ref, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


SHAPES = [(1, 1), (1, 128), (3, 31), (5, 33), (16, 512), (7, 1000), (64, 2049), (9, 4096), (2, 10007), (700, 64)]
ACTS = ["none", "relu", "leaky_relu", "silu", "gelu", "tanh", "sigmoid"]


def same_codes(c, codes, scales):
    assert torch.equal(c.codes.float(), codes) and torch.equal(torch.isnan(c.scales), torch.isnan(scales))
    assert torch.equal(c.scales.nan_to_num(-1), scales.nan_to_num(-1))


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_store_and_load(rows, cols, dtype, group, quant):
    """Codes and scales are the format's, exactly: they are computed from exact fp32 values by single roundings."""
    x = randn(gen(cols + group), rows, cols, std=3, dtype=dtype)
    c = ct.checkpoint_store(x, quant, group)
    same_codes(c, *q8_ref(x.float(), quant, group))
    back = ct.checkpoint_load(c)
    assert back.dtype == x.dtype
    ref = decoded(c)
    within(back, ref, ref.abs() * (U[dtype] + 2 * E) + TINY[dtype], "load")
    wide = ct.checkpoint_load(c, torch.float32)
    within(wide, ref, ref.abs() * 2 * E + TINY["f32"], "load f32")


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
def test_groups_without_a_scale(quant):
    """Zero groups, groups too small for a scale, infinities and NaN."""
    for cols in (512, 515):
        x = torch.randn(4, cols, generator=gen(1), device="cuda")
        x[0, :32] = 0
        x[0, 32:64] = 1e-38
        x[0, 64:96] *= 1e-30
        x[1, 40] = float("inf")
        x[2, 100] = float("-inf")
        x[3, 511] = float("nan")
        c = ct.checkpoint_store(x, quant, 32)
        same_codes(c, *q8_ref(x, quant, 32))
        back = ct.checkpoint_load(c)
        assert (back[0, :64] == 0).all() and torch.isnan(back[1, 32:64]).all() and torch.isfinite(back[1, 64:]).all()
        assert torch.isnan(back[2, 96:128]).all() and torch.isnan(back[3, 480:512]).all()
        assert torch.isfinite(back[0]).all()


def act_bound(x, u, y, dtype):
    # expf, erff, tanhf and the divisions are each good to a few roundings;
    # 1 + erf(x / sqrt 2) and tanh lose what cancels, bounded by the factor's
    # size before it: |x| * 8 E
    w = x.abs() if u is None else x.abs() * u.abs()
    one = torch.ones_like(x) if u is None else u.abs()
    return y.abs() * (U[dtype] + 16 * E) + (w + one) * 8 * E + TINY[dtype]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", [(1, 1), (16, 512), (7, 1000), (5, 2049), (33, 96)])
def test_activation(rows, cols, dtype, gated, act):
    g = gen(cols)
    x, up = randn(g, rows, cols, std=2, dtype=dtype), randn(g, rows, cols, std=2, dtype=dtype) if gated else None
    quant, group = ("int8", 64) if act in ("silu", "relu", "none") else ("e4m3", 128)
    y, cg, cu = ct.checkpointed_activation(x, up, act, 0.2, quant, group)
    xd, ud = x.double(), up.double() if gated else None
    ref = act_ref(xd, act, 0.2) * (ud if gated else 1.0)
    within(y, ref, act_bound(xd, ud, ref, dtype), "y")
    same_codes(cg, *q8_ref(x.float(), quant, group))
    assert (cu is None) == (not gated)
    if gated:
        same_codes(cu, *q8_ref(up.float(), quant, group))
    # the gradient, at the kept values
    dy = randn(g, rows, cols, dtype=dtype)
    kg, ku = decoded(cg), decoded(cu) if gated else None
    leaf = kg.clone().requires_grad_()
    slope = torch.autograd.grad(act_ref(leaf, act, 0.2).sum(), leaf)[0]
    f = act_ref(kg, act, 0.2)
    dyd = dy.double()
    dgate, dup, y2 = ct.checkpointed_activation_backward(dy, cg, cu, act, 0.2, need=("dgate", "dup", "y"))
    other = ku if gated else torch.ones_like(kg)
    # each slope is a product or a sum of terms of at most 1 + |x| in size
    want = dyd * slope * other
    within(dgate, want, want.abs() * (U[dtype] + 16 * E) + (dyd * other).abs() * (1 + kg.abs()) * 16 * E + TINY[dtype], "dgate")
    want = f * other
    within(y2, want, act_bound(kg, ku, want, dtype), "y again")
    if gated:
        want = dyd * f
        within(dup, want, act_bound(kg, dyd, want, dtype), "dup")
    else:
        assert dup is None
    only = ct.checkpointed_activation_backward(dy, cg, cu, act, 0.2, need=("dup",))
    assert only[0] is None and (not gated or torch.equal(only[1], dup))


@pytest.mark.parametrize("dtype", list(DT))
def test_halves_of_a_projection(dtype):
    """gate and up as halves of one wider matrix, at starts of every alignment; three axes."""
    g = gen(2)
    both = randn(g, 3, 11, 2 * 192 + 9, dtype=dtype)
    for first in (0, 1, 2, 4, 8, 9):
        gate, up = both[..., first:first + 192], both[..., first + 192:first + 384]
        y, cg, cu = ct.checkpointed_activation(gate, up, "silu", quant="int8", group=64)
        y2, cg2, cu2 = ct.checkpointed_activation(gate.contiguous(), up.contiguous(), "silu", quant="int8", group=64)
        assert torch.equal(y, y2)
        for a, b in ((cg, cg2), (cu, cu2)):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        dy = both[..., first:first + 192]
        for a, b in zip(ct.checkpointed_activation_backward(dy, cg, cu), ct.checkpointed_activation_backward(dy.contiguous(), cg, cu)):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y3 = ct.checkpointed_activation(gate, up, "silu", quant="int8", group=64)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y3, y)


def test_gradients_into_one_projection():
    """dgate and dup written into the halves of one matrix, and y over gate, through the C entry points."""
    g = gen(5)
    for cols in (256, 257):
        gate, up, dy = (randn(g, 19, cols, dtype="bf16") for _ in range(3))
        y, cg, cu = ct.checkpointed_activation(gate, up)
        dgate, dup = ct.checkpointed_activation_backward(dy, cg, cu)
        both = torch.empty(19, 2 * cols, dtype=torch.bfloat16, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        kept = [t.data_ptr() for t in (cg.codes, cg.scales, cu.codes, cu.scales)]
        rc = ct.lib().ct_checkpointed_activation_backward(dy.data_ptr(), cols, *kept, both.data_ptr(), 2 * cols,
                                                          both.data_ptr() + 2 * cols, 2 * cols, None, 0, 19, cols,
                                                          ct.CT_ACT_SILU, 0.0, ct.CT_BF16, 1, 128, s)
        assert rc == ct.CT_OK and torch.equal(both[:, :cols], dgate) and torch.equal(both[:, cols:], dup)
        over = gate.clone()
        rc = ct.lib().ct_checkpointed_activation_forward(over.data_ptr(), cols, up.data_ptr(), cols, over.data_ptr(), cols, *kept,
                                                         19, cols, ct.CT_ACT_SILU, 0.0, ct.CT_BF16, 1, 128, s)
        assert rc == ct.CT_OK and torch.equal(over, y)


def test_nothing_to_do():
    for shape in ((0, 64), (3, 0)):
        x = torch.empty(shape, device="cuda")
        y, cg, cu = ct.checkpointed_activation(x, x)
        assert y.shape == shape and cg.codes.shape == shape
        assert ct.checkpoint_load(ct.checkpoint_store(x)).shape == shape
        assert ct.checkpointed_activation_backward(x, cg, cu)[1].shape == shape


def test_autograd_against_differences():
    """The recorded gradient against central differences of the activation at the kept values."""
    g = gen(8)
    gate, up, a = randn(g, 5, 130), randn(g, 5, 130), randn(g, 5, 130).double()
    leaves = [gate.clone().requires_grad_(), up.clone().requires_grad_()]
    y = ct.checkpointed_activation_autograd(*leaves, activation="gelu", quant="int8", group=32)
    (y * a.float()).sum().backward()
    kg, ku = (decoded(ct.checkpoint_store(t, "int8", 32)) for t in (gate, up))

    def f(x, u):
        return (act_ref(x, "gelu") * u * a).sum()

    step = 1e-6
    for i in range(2):
        d = torch.randn(5, 130, generator=g, device="cuda").double()
        lo, hi = [kg, ku], [kg, ku]
        hi[i], lo[i] = hi[i] + step * d, lo[i] - step * d
        want = ((f(*hi) - f(*lo)) / (2 * step)).item()
        terms = leaves[i].grad.double() * d
        assert abs(terms.sum().item() - want) <= 64 * E * terms.abs().sum().item() + 1e-5


@pytest.mark.parametrize("dtype,quant", [("bf16", "int8"), ("f16", "e4m3"), ("f32", "int8")])
def test_convolution_keeps_its_input_in_8_bits(dtype, quant):
    """conv_transpose's weight gradient from an 8-bit x is that of the kept x, exactly; dx, db and y do not change."""
    g = gen(6)
    x, w, b = randn(g, 2, 64, 9, 16, dtype=dtype), randn(g, 64, 32, 4, 4, std=0.05, dtype=dtype), randn(g, 32, dtype=dtype)
    args = dict(stride=2, padding=1)
    plain = [t.clone().requires_grad_() for t in (x, w, b)]
    kept = [t.clone().requires_grad_() for t in (x, w, b)]
    y = ct.conv_transpose_autograd(*plain, **args)
    y8 = ct.conv_transpose_autograd(*kept, **args, checkpoint=quant)
    assert torch.equal(y, y8)
    dy = randn(g, *y.shape, dtype=dtype)
    y.backward(dy)
    y8.backward(dy)
    assert torch.equal(plain[0].grad, kept[0].grad) and torch.equal(plain[2].grad, kept[2].grad)
    x8 = ct.checkpoint_load(ct.checkpoint_store(x.flatten(2).flatten(0, 1), quant)).view(x.shape)
    assert torch.equal(kept[1].grad, ct.conv_transpose_backward(x8, w, dy, **args)[1])
    # only dx asked for
    w2 = w.clone()
    x2 = x.clone().requires_grad_()
    ct.conv_transpose_autograd(x2, w2, **args, checkpoint=quant).backward(dy)
    assert torch.equal(x2.grad, plain[0].grad)
