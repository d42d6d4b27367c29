"""What a call of the gated projection allocates."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 4, 16])
@pytest.mark.parametrize("layout", ["in_out", "out_in", "halves"])
@pytest.mark.parametrize("kind", ["aligned", "rows off 16 bytes"])
def test_streaming_steps_allocate_their_result_alone(dtype, rows, layout, kind):
    """Calls that go past the tensor cores use no workspace, and none is taken."""
    if dtype != "f32" and rows > 4:
        pytest.skip("those take the tensor cores")
    g = gen(1)
    C, F = 256, 512
    x = randn(g, rows, C + 1, dtype=dtype)[:, 1:] if kind != "aligned" else randn(g, rows, C, dtype=dtype)
    if layout == "halves":
        both = randn(g, C, 2 * F, dtype=dtype)
        wg, wu = both[:, :F], both[:, F:]
    else:
        wg, wu = (randn(g, C, F, dtype=dtype) if layout == "in_out" else randn(g, F, C, dtype=dtype).t() for _ in range(2))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    y = ct.gated_projection(x, wg, wu)
    used = torch.cuda.max_memory_allocated() - before
    # the allocator's blocks are multiples of 512 bytes
    assert used == -(-y.numel() * y.element_size() // 512) * 512
