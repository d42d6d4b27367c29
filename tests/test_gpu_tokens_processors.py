"""The layers of an image or video decoder on a stream that has 64 of the GPU's processors: clusters and pairs are placed there, the results the same."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn
from test_gpu_attention_limits import part_of_the_device  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def gated(dtype, rows, C, F):
    g = gen(rows)
    x, dy, wg, wu = randn(g, rows, C, dtype=dtype), randn(g, rows, F, dtype=dtype), randn(g, C, F, std=C ** -0.5, dtype=dtype), randn(g, C, F, std=C ** -0.5, dtype=dtype)
    return lambda: (ct.gated_projection(x, wg, wu), *ct.gated_projection_backward(dy, x, wg, wu))


def norm(dtype, B, S, C, G):
    g = gen(S)
    x, dy, w, b = randn(g, B, S, C, dtype=dtype), randn(g, B, S, C, dtype=dtype), randn(g, C, dtype=dtype), randn(g, C, dtype=dtype)

    def f():
        y, mean, rstd = ct.group_norm(x, G, w, b, activation="silu")
        return (y, mean, rstd, *ct.group_norm_backward(dy, x, mean, rstd, w, b, "silu"))
    return f


@pytest.mark.parametrize("call", [lambda: gated("bf16", 2, 512, 2048), lambda: gated("f32", 9, 512, 2048), lambda: gated("bf16", 3000, 520, 1032),
                                  lambda: gated("f32", 300, 512, 520), lambda: norm("bf16", 1, 12000, 512, 32), lambda: norm("bf16", 1, 4500, 64, 8),
                                  lambda: norm("f32", 2, 70000, 40, 5), lambda: norm("bf16", 16, 4096, 256, 32)],
                         ids=["few", "few f32", "pairs", "pairs f32", "one pass, large", "one pass", "two passes f32", "two passes"])
def test_a_stream_with_part_of_the_processors(part_of_the_device, call):  # noqa: F811
    f = call()
    want = f()
    torch.cuda.synchronize()
    with torch.cuda.stream(part_of_the_device):
        got = f()
    part_of_the_device.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert ct.ct_device_status(clear=True) == (ct.CT_OK, 0)
