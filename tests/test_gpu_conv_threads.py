"""Transposed convolutions of different sizes from several host threads at once, each kernel keeping what it needs of shared memory."""
import ctypes
import threading

import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from transposed_convolution_convtranspose1_gb300 import ct as ctb
from _block import DT, gen, need_gpu, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def entry(form, dtype, C_in, C_out, spatial, k, stride, groups):
    """(a C call on given streams with its arguments laid out beforehand, its outputs, what they should be)."""
    g = gen(C_in + C_out)
    B, nd = 1, len(spatial)
    x, w = randn(g, B, C_in, *spatial, dtype=dtype), randn(g, C_in, C_out // groups, *k, dtype=dtype)
    ax = ctb._Axes(nd, spatial, k, stride, None, None, None, None)
    shape = ctb._shape_args(B, C_in, C_out, ax, groups, ctb.dtype_code(DT[dtype]))
    route = ct.CT_ROUTE_GATHER if form == "gather" else ct.CT_ROUTE_GROUPED
    keep = [x, w, ax]
    if form == "backward":
        O = ctb.ct_conv_transpose_out_shape(spatial, k, stride)
        dy = randn(g, B, C_out, *O, dtype=dtype)
        want = [ct.conv_transpose_backward(x, w, dy, stride=stride, groups=groups, need=("dx",))[0]]
        out = [torch.empty_like(want[0])]
        n = ctb.ct_conv_transpose_backward_workspace_bytes(B, C_in, C_out, spatial, k, stride, groups=groups, dtype=ctb.dtype_code(DT[dtype]))
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        fn = ct.lib().ct_conv_transpose_backward_nd
        args = (x.data_ptr(), w.data_ptr(), dy.data_ptr(), out[0].data_ptr(), None, None, ws.data_ptr(), n, *shape)
        keep += [dy, ws]
    else:
        want = [ct.conv_transpose(x, w, stride=stride, groups=groups, route=route)]
        out = [torch.empty_like(want[0])]
        fn, args = ct.lib().ct_conv_transpose_nd_route, (x.data_ptr(), w.data_ptr(), None, out[0].data_ptr(), None, 0, *shape, route)
    return fn, args, out, want, keep


@pytest.mark.parametrize("form,dtype,small,large", [
    # weights of 64 and 96 KB in shared memory
    ("gather", "f32", (32, 16, (40,), (32,), 2, 1), (48, 16, (40,), (32,), 2, 1)),
    ("gather", "bf16", (32, 16, (40,), (32,), 2, 1), (48, 16, (40,), (32,), 2, 1)),
    # rows of another width
    ("grouped", "bf16", (16, 16, (4, 16, 30), (4, 4, 4), 2, 2), (16, 16, (4, 16, 60), (4, 4, 4), 2, 2)),
    ("grouped", "f32", (16, 16, (4, 16, 32), (2, 4, 4), 2, 2), (16, 16, (4, 16, 32), (4, 4, 4), 2, 2)),
    ("backward", "f32", (32, 64, (40,), (32,), 2, 2), (32, 96, (40,), (32,), 2, 2)),
], ids=["gather f32", "gather bf16", "grouped bf16", "grouped f32", "backward f32"])
def test_sizes_at_once(form, dtype, small, large):
    calls = [entry(form, dtype, *p) for p in (small, large, small, large)]
    torch.cuda.synchronize()
    failed, why = [0] * 4, set()
    start = threading.Barrier(4)

    def work(i):
        fn, args = calls[i][:2]
        stream = torch.cuda.Stream()
        stream.synchronize()  # the thread has the device's context
        start.wait()
        for _ in range(4000):
            if fn(*args, stream.cuda_stream) != ct.CT_OK:
                failed[i] += 1
                why.add(ctb.ct_last_error())
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * 4, why
    for _, _, out, want, _ in calls:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
