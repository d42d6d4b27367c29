"""fp32 products of the gated projection, held to what three bf16 parts leave, and group norm's bounds with as many chunks as there are.

No activation: y = g u, dg = dy u, du = dy g, so that the products' own errors show.
"""
import pytest
import torch

import _tokens
import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn
from _parts import rms, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def near(got, ref, bound, what):
    off = rms(got.double() - ref) / rms(ref)
    assert off <= bound, f"{what}: {off:.2e} of its size, {bound:.2e} allowed"


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("rows,C,F", [(512, 512, 512), (64, 2048, 512), (100, 512, 640), (1000, 640, 520), (2048, 512, 1024), (17, 1000, 512)])
def test_sums_of_many_blocks(rows, C, F, layout):
    g = gen(rows)
    x, dy = randn(g, rows, C), randn(g, rows, F)
    wg, wu = (randn(g, C, F, std=C ** -0.5) if layout == "in_out" else randn(g, F, C, std=C ** -0.5).t() for _ in range(2))
    xd, wgd, wud, dyd = (t.double() for t in (x, wg, wu, dy))
    gd, ud = xd @ wgd, xd @ wud
    first = tolerance(C)  # of g and u
    near(ct.gated_projection(x, wg, wu, None), gd * ud, 2 * first + 2.0 ** -24, "y")
    dx, dwg, dwu = ct.gated_projection_backward(dy, x, wg, wu, None)
    # dg and du carry u's and g's errors, and their own rounding
    near(dwg, xd.t() @ (dyd * ud), first + tolerance(rows) + 2.0 ** -24, "dw_gate")
    near(dwu, xd.t() @ (dyd * gd), first + tolerance(rows) + 2.0 ** -24, "dw_up")
    near(dx, (dyd * ud) @ wgd.t() + (dyd * gd) @ wud.t(), first + tolerance(F, pairs=2) + 2.0 ** -24, "dx")


@pytest.mark.parametrize("shape,G", [((2, 30000, 64), 8), ((1, 100000, 40), 5), ((3, 20000, 210), 7), ((1, 40000, 512), 1)], ids=str)
def test_group_norm_with_the_chunks_there_are(monkeypatch, shape, G):
    """Two blocks an SM at most share the positions of a sample."""
    most = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    monkeypatch.setattr(_tokens, "norm_chunks", lambda S: min(most, S // 16 + 1))
    g = gen(1)
    x, w, b, dy = 3 + randn(g, *shape), randn(g, shape[2]), randn(g, shape[2]), randn(g, *shape)
    y, mean, rstd = ct.group_norm(x, G, w, b, activation="silu")
    _tokens.check_group_norm(x, G, w, b, 1e-5, "silu", "f32", y, mean, rstd)
    _tokens.check_group_norm_back(dy, x, mean, rstd, G, w, b, "silu", "f32", *ct.group_norm_backward(dy, x, mean, rstd, w, b, "silu"))
