"""RMS norm with the residual's addition and an 8-bit output, and its gradient, against 64 bits."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import (DT, E, TINY, U, check_norm, decoded, gen, need_gpu, norm_back_ref, norm_chain, q8_ref, randn,
                    within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


SHAPES = [(1, 1), (1, 512), (3, 7), (5, 64), (8, 512), (17, 999), (64, 1000), (33, 1024), (7, 2049), (300, 256), (9, 4096), (5, 4104),
          (3, 8192), (2, 12345), (2, 40000), (2000, 128)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dtype):
    g = gen(rows * 131 + cols)
    x, r, w = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, std=3, dtype=dtype), randn(g, cols, dtype=dtype)
    for res in (None, r):
        for weight in (w, None):
            y, h, rstd, kept = ct.rms_norm(x, weight, res, eps=1e-5)
            assert kept is None and (res is not None or h is x)
            check_norm(x, weight, res, 1e-5, dtype, y, h, rstd)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (8, 512), (5, 999), (64, 1000), (16, 2048), (3, 2050), (3, 5000), (2, 20000)])
@pytest.mark.parametrize("dtype", list(DT))
def test_8_bit_output(rows, cols, group, quant, dtype):
    """The codes are within one rounding step (and the fp32 norm's error) of the exact y."""
    g = gen(cols * 7 + group)
    x, r, w = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype), randn(g, cols, dtype=dtype)
    y, h, rstd, kept = ct.rms_norm(x, w, r, quant=quant, group=group, need=("y", "rstd"))
    exact = check_norm(x, w, r, 1e-6, dtype, y, h, rstd)
    assert kept.codes.shape == x.shape and kept.scales.shape == (rows, -(-cols // group))
    scale = kept.scales.double().repeat_interleave(group, 1)[:, :cols]
    k = norm_chain(cols) * E
    # int8: half a step of the scale; e4m3: a unit roundoff of 2^-4, or half
    # its subnormal step of 2^-9
    step = scale * 0.5 if quant == "int8" else torch.maximum(exact.abs() * 2.0 ** -4, scale * 2.0 ** -10)
    within(decoded(kept), exact, step * 1.0001 + exact.abs() * 4 * k, "8-bit y")
    top = 127.0 if quant == "int8" else 448.0
    # amax of the group over top
    pad = torch.zeros(rows, -(-cols // group) * group, dtype=torch.float64, device="cuda")
    pad[:, :cols] = exact.abs()
    want = pad.view(rows, -1, group).amax(2) / top
    within(kept.scales, want, want * (k + 4 * E), "scales")
    # without y the codes are the same
    none, _, _, again = ct.rms_norm(x, w, r, quant=quant, group=group, need=())
    assert none is None and torch.equal(again.codes.view(torch.uint8), kept.codes.view(torch.uint8))
    assert torch.equal(again.scales, kept.scales)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, dtype):
    g = gen(rows * 17 + cols)
    h, dy = randn(g, rows, cols, std=2, dtype=dtype), randn(g, rows, cols, dtype=dtype)
    w, dres = randn(g, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype)
    rstd = (h.float().square().mean(1) + 1e-6).rsqrt()
    for weight, extra in ((w, dres), (w, None), (None, dres)):
        dx, dw = ct.rms_norm_backward(dy, h, rstd, weight, extra)
        rx, ax, rw, aw = norm_back_ref(dy, h, rstd, weight, extra)
        within(dx, rx, rx.abs() * U[dtype] + ax * norm_chain(cols) * E + TINY[dtype], "dx")
        assert (dw is None) == (weight is None)
        if dw is not None:
            within(dw, rw, rw.abs() * U[dtype] + aw * (rows + 32) * E + TINY[dtype], "dw")
    only, none = ct.rms_norm_backward(dy, h, rstd, w, dres, need=("dx",))
    assert none is None
    none, dw2 = ct.rms_norm_backward(dy, h, rstd, w, dres, need=("dw",))
    assert none is None and torch.equal(dw2, ct.rms_norm_backward(dy, h, rstd, w, dres)[1])


def test_more_rows_than_blocks_and_reproducible():
    g = gen(3)
    h, dy, w = randn(g, 5001, 768, dtype="bf16"), randn(g, 5001, 768, dtype="bf16"), randn(g, 768, dtype="bf16")
    rstd = (h.float().square().mean(1) + 1e-6).rsqrt()
    a, b = ct.rms_norm_backward(dy, h, rstd, w), ct.rms_norm_backward(dy, h, rstd, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    rx, ax, rw, aw = norm_back_ref(dy, h, rstd, w, None)
    within(a[0], rx, rx.abs() * U["bf16"] + ax * norm_chain(768) * E, "dx")
    within(a[1], rw, rw.abs() * U["bf16"] + aw * 5033 * E, "dw")


@pytest.mark.parametrize("dtype", list(DT))
def test_strides_shapes_and_offsets(dtype):
    """Rows of a wider matrix, unaligned starts, three axes, tensors on another stream."""
    g = gen(9)
    wide = randn(g, 6, 5, 3 * 320 + 5, dtype=dtype)
    w = randn(g, 320, dtype=dtype)
    for first in (0, 1, 2, 3, 320, 325):
        x, r = wide[..., first:first + 320], wide[..., first + 320:first + 640]
        y, h, rstd, kept = ct.rms_norm(x, w, r, quant="int8")
        check_norm(x, w, r, 1e-6, dtype, y, h, rstd)
        dx, dw = ct.rms_norm_backward(r, x, rstd, w, x)
        rx, ax, rw, aw = norm_back_ref(r, x, rstd, w, x)
        within(dx, rx, rx.abs() * U[dtype] + ax * norm_chain(320) * E, "dx")
        within(dw, rw, rw.abs() * U[dtype] + aw * 62 * E, "dw")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = ct.rms_norm(x, w, r)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y2, y)
    with pytest.raises(ValueError):
        ct.rms_norm(wide.transpose(1, 2))


def test_outputs_in_place():
    """h written over the residual, and dx over dy, through the C entry points."""
    g = gen(4)
    for cols in (512, 2048, 999):
        x, r, w = randn(g, 33, cols, dtype="bf16"), randn(g, 33, cols, dtype="bf16"), randn(g, cols, dtype="bf16")
        y, h, rstd, _ = ct.rms_norm(x, w, r)
        s = torch.cuda.current_stream().cuda_stream
        stream, y2 = r.clone(), torch.empty_like(x)
        rc = ct.lib().ct_rms_norm_forward(x.data_ptr(), cols, stream.data_ptr(), cols, w.data_ptr(), y2.data_ptr(), cols,
                                          stream.data_ptr(), cols, None, None, None, 33, cols, 1e-6, ct.CT_BF16, 0, 128, s)
        assert rc == ct.CT_OK and torch.equal(stream, h) and torch.equal(y2, y)
        dx, _ = ct.rms_norm_backward(x, h, rstd, w, r)
        d = x.clone()
        rc = ct.lib().ct_rms_norm_backward(d.data_ptr(), cols, h.data_ptr(), cols, rstd.data_ptr(), w.data_ptr(), r.data_ptr(), cols,
                                           d.data_ptr(), cols, None, None, 0, 33, cols, ct.CT_BF16, s)
        assert rc == ct.CT_OK and torch.equal(d, dx)
        # dw with a workspace of the call's own
        dw = torch.empty(cols, dtype=torch.bfloat16, device="cuda")
        rc = ct.lib().ct_rms_norm_backward(x.data_ptr(), cols, h.data_ptr(), cols, rstd.data_ptr(), w.data_ptr(), None, 0, None, 0,
                                           dw.data_ptr(), None, 0, 33, cols, ct.CT_BF16, s)
        assert rc == ct.CT_OK and torch.equal(dw, ct.rms_norm_backward(x, h, rstd, w)[1])


def test_extreme_rows():
    """Zero rows, rows whose squares are subnormal, infinities and NaN stay in their rows."""
    for cols in (64, 1000, 4096):
        x = torch.ones(6, cols, device="cuda")
        x[1], x[2, 3], x[3, 5], x[4] = 0, float("inf"), float("nan"), 1e-18
        y, _, rstd, kept = ct.rms_norm(x, eps=1e-6, quant="int8", group=32)
        check_norm(x[[0, 1, 4, 5]], None, None, 1e-6, "f32", y[[0, 1, 4, 5]], None, rstd[[0, 1, 4, 5]])
        assert torch.isnan(y[3]).all() and torch.isnan(kept.scales[3]).all()
        # inf / inf: NaN at the infinity, 0 beside it
        assert torch.isnan(y[2, 3]) and (y[2, 4:] == 0).all() and torch.isnan(kept.scales[2, 0])
        assert (kept.scales[1] == 0).all() and (kept.codes[1] == 0).all()
        assert torch.isnan(ct.checkpoint_load(kept)[3]).all() and (ct.checkpoint_load(kept)[1] == 0).all()


def test_no_rows():
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, h, rstd, kept = ct.rms_norm(x, w, x, quant="e4m3")
    assert y.shape == h.shape == (0, 64) and rstd.shape == (0,) and kept.scales.shape == (0, 1)
    dx, dw = ct.rms_norm_backward(x, x, rstd, w)
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_autograd_against_differences():
    """The gradient of sum(y * a + h * b) against central differences in 64 bits along random directions."""
    g = gen(21)
    x, r, w = randn(g, 7, 200), randn(g, 7, 200), randn(g, 200)
    a, b = randn(g, 7, 200).double(), randn(g, 7, 200).double()
    leaves = [t.clone().requires_grad_() for t in (x, w, r)]
    y, h = ct.rms_norm_autograd(leaves[0], leaves[1], leaves[2], 1e-5)
    (y * a.float() + h * b.float()).sum().backward()

    def f(x, w, r):
        s = x + r
        return ((s * ((s * s).mean(1, keepdim=True) + 1e-5).rsqrt() * w) * a + s * b).sum()

    base = [t.double() for t in (x, w, r)]
    for i in range(3):
        d = torch.randn(base[i].shape, generator=g, device="cuda").double()
        step = 1e-5
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + step * d, base[i] - step * d
        want = ((f(*up) - f(*down)) / (2 * step)).item()
        terms = leaves[i].grad.double() * d
        # the fp32 gradient: as the bounds above, with 200 + 32 roundings of
        # each term; the difference itself is good to about 1e-9
        assert abs(terms.sum().item() - want) <= 300 * E * terms.abs().sum().item() + 1e-6
    y1 = ct.rms_norm_autograd(leaves[0], leaves[1])
    assert y1.grad_fn is not None and torch.equal(y1, ct.rms_norm(x, w)[0])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [64, 256, 264, 1000, 2048, 2944])
def test_forward_of_many_rows(cols, dtype):
    """Enough rows that the blocks walk them: every row right, h over the residual, reproducible."""
    rows = 45001 if cols < 512 else 21000 if cols <= 1000 else 9001
    g = gen(cols)
    x, r, w = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype), randn(g, cols, dtype=dtype)
    y, h, rstd, kept = ct.rms_norm(x, w, r, quant="int8", group=64)
    exact = check_norm(x, w, r, 1e-6, dtype, y, h, rstd)
    scale = kept.scales.double().repeat_interleave(64, 1)[:, :cols]
    within(decoded(kept), exact, scale * 0.50005 + exact.abs() * 4 * norm_chain(cols) * E, "8-bit y")
    del exact, scale
    stream, y2 = r.clone(), torch.empty_like(x)
    rc = ct.lib().ct_rms_norm_forward(x.data_ptr(), cols, stream.data_ptr(), cols, w.data_ptr(), y2.data_ptr(), cols, stream.data_ptr(),
                                      cols, None, None, None, rows, cols, 1e-6, ct.dtype_code(x.dtype), 0, 128,
                                      torch.cuda.current_stream().cuda_stream)
    assert rc == ct.CT_OK and torch.equal(stream, h) and torch.equal(y2, y)
    assert torch.equal(ct.rms_norm(x, None, None)[0], ct.rms_norm(x, None, None)[0])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [257, 300, 511, 513, 1025, 1500, 2047, 2049, 4097, 8191, 8193, 16385])
def test_odd_widths(cols, dtype):
    """Rows off 16-byte boundaries on both sides of every width at which another kernel takes over."""
    test_forward(37, cols, dtype)
    test_backward(37, cols, dtype)
    test_8_bit_output(9, cols, 128, "int8", dtype)
