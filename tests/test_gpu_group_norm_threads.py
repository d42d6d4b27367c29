"""Group norm of different sizes from several host threads at once, each kernel keeping what it needs of shared memory."""
import ctypes
import threading

import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def entry(form, B, S, C=512, G=32):
    """(a C call on given streams with its arguments laid out beforehand, its outputs, what they should be)."""
    g = gen(S)
    x, dy, w, b = randn(g, B, S, C, dtype="bf16"), randn(g, B, S, C, dtype="bf16"), randn(g, C, dtype="bf16"), randn(g, C, dtype="bf16")
    y, mean, rstd = ct.group_norm(x, G, w, b, activation="silu")
    want = [y, mean, rstd] if form == "forward" else list(ct.group_norm_backward(dy, x, mean, rstd, w, b, "silu"))
    out = [torch.empty_like(t) for t in want]
    strides = (ctypes.c_int64 * 2)(S * C, C)
    need = ctypes.c_size_t(0)
    assert ct.lib().ct_group_norm_workspace_bytes(B, S, C, G, ct.CT_BF16, int(form != "forward"), ctypes.byref(need)) == ct.CT_OK
    ws = torch.empty(max(need.value, 1), dtype=torch.uint8, device="cuda")
    if form == "forward":
        fn, args = ct.lib().ct_group_norm_forward, (x.data_ptr(), strides, w.data_ptr(), b.data_ptr(), out[0].data_ptr(), strides, out[1].data_ptr(),
                                                    out[2].data_ptr(), ws.data_ptr(), need.value, B, S, C, G, 1e-5, 3, 0.0, ct.CT_BF16)
    else:
        fn, args = ct.lib().ct_group_norm_backward, (dy.data_ptr(), strides, x.data_ptr(), strides, mean.data_ptr(), rstd.data_ptr(), w.data_ptr(),
                                                     b.data_ptr(), out[0].data_ptr(), strides, out[1].data_ptr(), out[2].data_ptr(), ws.data_ptr(),
                                                     need.value, B, S, C, G, 3, 0.0, ct.CT_BF16)
    return fn, args, out, want, (x, dy, w, b, ws, mean, rstd)


@pytest.mark.parametrize("form", ["forward", "gradient"])
def test_sizes_at_once(form):
    """One kernel (bf16, vectors of 8), 48 KB of shared memory a block in two threads' calls and 96 KB (gradient: 208 KB) in the others'."""
    large = 20000 if form == "forward" else 12000
    calls = [entry(form, 4, 1024), entry(form, 1, large), entry(form, 4, 1024), entry(form, 1, large)]
    torch.cuda.synchronize()
    failed = [0] * 4
    start = threading.Barrier(4)

    def work(i):
        fn, args = calls[i][:2]
        stream = torch.cuda.Stream()
        start.wait()
        for _ in range(4000):
            failed[i] += fn(*args, stream.cuda_stream) != ct.CT_OK
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * 4
    for _, _, out, want, _ in calls:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
