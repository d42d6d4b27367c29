"""The gated projection in fp32 at the ends of its range, by both routes: a few rows (fp32 arithmetic) and the tensor cores (three bf16 parts)."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import E, gen, need_gpu, randn, within
from _tokens import gated_parts

pytestmark = pytest.mark.gpu
FEW = 16  # rows of fp32 up to which weights in place go past the tensor cores


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def operands(rows, layout, C=64, F=96):
    g = gen(rows)
    x, dy = randn(g, rows, C), randn(g, rows, F)
    return (x, dy, *(randn(g, C, F, std=0.125) if layout == "in_out" else randn(g, F, C, std=0.125).t() for _ in range(2)))


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("rows", [1, 2, FEW, FEW + 1, 40, 200])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("where", ["x", "gate", "up"])
def test_a_value_that_is_not_finite(where, layout, rows, bad):
    """It reaches its row (of x) or its column (of a weight) alone; a few rows get what the formula has, the others no finite number."""
    x, dy, wg, wu = operands(rows, layout)
    clean = ct.gated_projection(x, wg, wu, None)
    want = ct.gated_projection_backward(dy, x, wg, wu, None)
    {"x": x, "gate": wg, "up": wu}[where][(rows - 1, 5) if where == "x" else (7, 11)] = bad
    y = ct.gated_projection(x, wg, wu, None)
    dx, dwg, dwu = ct.gated_projection_backward(dy, x, wg, wu, None)
    at = (slice(rows - 1, rows),) if where == "x" else (slice(None), slice(11, 12))
    if rows <= FEW:
        ref = ((x.double() @ wg.double()) * (x.double() @ wu.double()))[at]
        assert torch.equal(torch.isnan(y[at]), torch.isnan(ref)) and torch.equal(y[at].double()[~torch.isnan(ref)], ref[~torch.isnan(ref)])
    else:
        assert not torch.isfinite(y[at]).any()
    pairs = [(y, clean, at)]
    if where == "x":  # each row of dx comes from its own row of x; what sums over rows holds it everywhere or in channel 5
        pairs.append((dx, want[0], at))
    else:
        pairs += [(dwg, want[1], at), (dwu, want[2], at)]
    for got, ref, part in pairs:
        got, ref = got.clone(), ref.clone()
        got[part] = ref[part] = 0
        assert torch.equal(got, ref)


@pytest.mark.parametrize("rows", [3, 40, 200])
@pytest.mark.parametrize("e", [60, 109, 114, 120, 126])
@pytest.mark.parametrize("small", ["x", "weights"])
def test_small_factors(small, e, rows):
    """Factors around 2^-e against large ones.  Parts are multiples of 2^-133: a factor is off by 2^-134 at most, and not at all from 2^-110 on."""
    x, _, wg, wu = operands(rows, "in_out")
    down, up = 2.0 ** -e, 2.0 ** min(e, 118)
    x, wg, wu = ((t.double() * (down if (small == "x") == (i == 0) else up)).float() for i, t in enumerate((x, wg, wu)))
    g, u, dg, du = gated_parts(x, wg, wu, "f32")
    off = 0.0 if rows <= FEW else 2.0 ** -134
    ones = torch.ones_like(x, dtype=torch.float64)
    dg, du = (d + off * (ones @ w.double().abs() + x.double().abs() @ torch.ones_like(w, dtype=torch.float64)) for d, w in ((dg, wg), (du, wu)))
    # products of the smallest factors themselves may fall below fp32's own range: 2^-149 for each of the C terms
    y = ct.gated_projection(x, wg, wu, None)
    within(y, g * u, (g * u).abs() * 2 * E + g.abs() * du + u.abs() * dg + dg * du + 64 * 2.0 ** -149, "y")


@pytest.mark.parametrize("rows", [3, 40, 200])
def test_the_largest_factors(rows):
    """3.4e38 has no bf16 neighbour above it: its parts begin below it."""
    x, _, wg, wu = operands(rows, "in_out")
    x[0] = torch.finfo(torch.float32).max
    x[-1, ::2] = -torch.finfo(torch.float32).max
    wg, wu = wg * 2.0 ** -120, wu * 2.0 ** -120
    g, u, dg, du = gated_parts(x, wg, wu, "f32")
    if rows > FEW:  # the weights, around 2^-123, are sums of three multiples of 2^-133: each is off by 2^-134 at most, against |x| up to 2^128
        dg, du = (d + 2.0 ** -134 * x.double().abs().sum(1, keepdim=True) for d in (dg, du))
    # rows of ordinary values: g and u near 2^-120 (no term below 2^-149), their product near 2^-240, which fp32 rounds to 0: off by less than 2^-150
    within(ct.gated_projection(x, wg, wu, None), g * u, (g * u).abs() * 2 * E + g.abs() * du + u.abs() * dg + dg * du + 2.0 ** -150, "y")
