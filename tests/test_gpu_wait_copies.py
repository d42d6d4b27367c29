"""Tensor-core convolutions whose copies are all on their way when another role gives up: the block still waits for them.

Problems of few taps and channels, so that no tile has more blocks of operands than the ring has places.  What runs next, right
behind the blocks that gave up, is undisturbed.
"""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from transposed_convolution_convtranspose1_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transposed_convolution_convtranspose1_gb300 import _build
    _build.build_library()
    ct.lib()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("k,stride", [(2, 2), (3, 1)])
def test_waits_that_give_up_with_every_copy_issued(k, stride, dtype):
    p = synth.problem("few", 1, 128, 128, (8, 8), k, stride=stride, pad=0, dtype=dtype, seed=5)
    code = ct.dtype_code(p.torch_dtype)
    shape = (p.B, p.C_in, p.C_out, p.spatial, p.k, p.stride, p.pad_lo, p.pad_hi, p.dilation, p.output_padding, p.groups, code)
    want = "tc32_phase_gemm" if dtype == "f32" else "tc_phase_gemm"
    assert ct.ct_conv_transpose_kernel(*shape) == want
    x, w, b = (None if t is None else t.cuda() for t in synth.make_inputs(p))
    args = dict(stride=p.stride, pad_lo=p.pad_lo, pad_hi=p.pad_hi)

    def both():
        y = ct.conv_transpose(x, w, b, **args)
        return (y, *ct.conv_transpose_backward(x, w, torch.ones_like(y), **args))

    good = both()
    torch.cuda.synchronize()
    assert ct.ct_device_status(clear=True) == (ct.CT_OK, 0)
    for _ in range(3):
        before = ct.ct_set_wait_limit_ns(0)
        try:
            both()
            both()
        finally:
            ct.ct_set_wait_limit_ns(before)
        again = both()  # its blocks follow those that gave up
        rc, word = ct.ct_device_status(clear=True)
        assert rc == ct.ct.CT_ERR_DEVICE_TIMEOUT and word != 0 and word & 0x8 == 0
        for a, c in zip(good, again):
            assert torch.equal(a, c)
    assert ct.ct_device_status(clear=True) == (ct.CT_OK, 0)
