"""Attention in chunks where its waits give up or the device has fewer processors: it reports, and leaves the device usable."""
import ctypes

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


class _Resource(ctypes.Structure):  # CUdevResource
    _fields_ = [("type", ctypes.c_int), ("_", ctypes.c_ubyte * 92), ("sm", ctypes.c_uint * 12)]


@pytest.fixture
def part_of_the_device():
    """A stream that has 64 of the GPU's processors (a green context of this process)."""
    cu = ctypes.CDLL("libcuda.so.1")
    torch.zeros(1, device="cuda")
    every, part, rest, n = _Resource(), _Resource(), _Resource(), ctypes.c_uint(1)
    desc, green, stream = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    by = ctypes.byref
    for rc in (lambda: cu.cuDeviceGetDevResource(torch.cuda.current_device(), by(every), 1),
               lambda: cu.cuDevSmResourceSplitByCount(by(part), by(n), by(every), by(rest), 0, 64),
               lambda: cu.cuDevResourceGenerateDesc(by(desc), by(part), 1),
               lambda: cu.cuGreenCtxCreate(by(green), desc, torch.cuda.current_device(), 1),
               lambda: cu.cuGreenCtxStreamCreate(by(stream), green, 1, 0)):
        code = rc()
        if code:
            pytest.skip(f"no green context here (driver status {code})")
    assert part.sm[0] < every.sm[0]
    yield torch.cuda.ExternalStream(stream.value)
    torch.cuda.synchronize()
    cu.cuStreamDestroy_v2(stream)
    cu.cuGreenCtxDestroy(green)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,T,H,Dk,Dv", [(1, 700, 160, 64, 64), (3, 500, 70, 128, 64), (1, 1700, 1, 64, 64)])
def test_a_stream_with_part_of_the_processors(part_of_the_device, B, T, H, Dk, Dv, dtype):
    """More walks than processors, which then share walks, on a stream that has fewer than the device: the same results."""
    f = calls(B, T, H, Dk, Dv, dtype)
    want = f()
    torch.cuda.synchronize()
    with torch.cuda.stream(part_of_the_device):
        got = f()
    part_of_the_device.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert ct.ct_device_status(clear=True) == (ct.CT_OK, 0)
