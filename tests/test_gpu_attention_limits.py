"""Attention in chunks where its waits give up or the device has fewer processors: it reports, and leaves the device usable."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def calls(B, T, H, Dk, Dv, dtype):
    g = gen(T)
    q, k, v, do = (randn(g, B, T, H, D, dtype=dtype) for D in (Dk, Dk, Dv, Dv))
    s, ds = randn(g, B, H, Dk, Dv), randn(g, B, H, Dk, Dv)
    ld = -torch.exp2(-torch.rand(H, generator=g, device="cuda") * 6)
    return lambda: ct.linear_attention(q, k, v, ld, s) + ct.linear_attention_backward(q, k, v, ld, do, s, ds)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (64, 128)])
@pytest.mark.parametrize("B,T,H", [(2, 33, 3), (2, 128, 3), (40, 200, 8), (1, 1700, 1), (1, 129, 160)])
def test_waits_that_give_up_with_every_copy_issued(B, T, H, Dk, Dv, dtype):
    """Walks of one and two chunks: the copies are all on their way when another warp gives up, and the block still waits for them.
    What runs next on the same processors, again and with other kernels between, is undisturbed."""
    f = calls(B, T, H, Dk, Dv, dtype)
    good = f()
    torch.cuda.synchronize()
    assert ct.ct_device_status(clear=True) == (ct.CT_OK, 0)
    for _ in range(3):
        before = ct.ct_set_wait_limit_ns(0)
        try:
            f()
            f()
        finally:
            ct.ct_set_wait_limit_ns(before)
        again = f()  # no synchronisation between: its blocks follow those that gave up
        rc, code = ct.ct_device_status(clear=True)
        assert rc == ct.ct.CT_ERR_DEVICE_TIMEOUT and code != 0
        for a, b in zip(good, again):
            assert torch.equal(a, b)
    assert ct.ct_device_status(clear=True) == (ct.CT_OK, 0)
