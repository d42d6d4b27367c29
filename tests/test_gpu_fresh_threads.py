"""C entry points called as a host thread's first use of the GPU."""
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


def conv(dtype, C_in, C_out, spatial, k, stride, groups=1):
    g = gen(1)
    x, w = randn(g, 1, C_in, *spatial, dtype=dtype), randn(g, C_in, C_out // groups, *k, dtype=dtype)
    ax = ctb._Axes(len(spatial), spatial, k, stride, None, None, None, None)
    want = ct.conv_transpose(x, w, stride=stride, groups=groups)
    out = torch.empty_like(want)
    args = (x.data_ptr(), w.data_ptr(), None, out.data_ptr(), None, 0, *ctb._shape_args(1, C_in, C_out, ax, groups, ctb.dtype_code(DT[dtype])))
    return ct.lib().ct_conv_transpose_nd, args, out, want, (x, w, ax)


def gated(dtype, rows):
    g = gen(2)
    x, wg, wu = (randn(g, *s, dtype=dtype) for s in ((rows, 64), (64, 96), (64, 96)))
    want = ct.gated_projection(x, wg, wu)
    out = torch.empty_like(want)
    s = (ctypes.c_int64 * 2)(96, 1)
    return ct.lib().ct_gated_projection_forward, (x.data_ptr(), 64, wg.data_ptr(), s, wu.data_ptr(), s, out.data_ptr(), 96, None, 0, rows, 64, 96, 3, 0.0,
                                                  ctb.dtype_code(DT[dtype])), out, want, (x, wg, wu)


def attention(dtype):
    g = gen(3)
    q, k, v = (randn(g, 1, 200, 2, 64, dtype=dtype) for _ in range(3))
    decay = torch.full((2,), -0.05, device="cuda")
    want = ct.linear_attention(q, k, v, decay)[0]
    out = torch.empty_like(want)
    s = (ctypes.c_int64 * 3)(200 * 128, 128, 64)
    return ct.lib().ct_linear_attention_forward, (q.data_ptr(), s, k.data_ptr(), s, v.data_ptr(), s, out.data_ptr(), s, decay.data_ptr(), None, None, None,
                                                  None, 0, 1, 200, 2, 64, 64, 64 ** -0.5, ctb.dtype_code(DT[dtype])), out, want, (q, k, v, decay)


def norm():
    g = gen(4)
    x = randn(g, 2, 70000, 64, dtype="bf16")
    want = ct.group_norm(x, 8)[0]
    out = torch.empty_like(want)
    s = (ctypes.c_int64 * 2)(70000 * 64, 64)
    return ct.lib().ct_group_norm_forward, (x.data_ptr(), s, None, None, out.data_ptr(), s, None, None, None, 0, 2, 70000, 64, 8, 1e-5, 0, 0.0,
                                            ct.CT_BF16), out, want, (x,)


CALLS = {"conv bf16": lambda: conv("bf16", 64, 64, (40,), (4,), 2), "conv f32": lambda: conv("f32", 64, 64, (40,), (4,), 2),
         "conv grouped": lambda: conv("f32", 16, 16, (4, 16, 32), (2, 4, 4), 2, 2), "gated bf16": lambda: gated("bf16", 200),
         "gated f32": lambda: gated("f32", 200), "gated few": lambda: gated("bf16", 2), "attention": lambda: attention("bf16"), "norm": norm}


@pytest.mark.parametrize("name", CALLS)
def test_a_first_call(name):
    fn, args, out, want, keep = CALLS[name]()
    torch.cuda.synchronize()
    rc = []
    thread = threading.Thread(target=lambda: rc.append((fn(*args, None), ctb.ct_last_error())))
    thread.start()
    thread.join()
    assert rc[0][0] == ct.CT_OK, rc
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_context_of_the_callers_stays_current():
    """A query that looks at the tensor-map route, in a thread whose current context is not the runtime's; nothing is launched there."""
    torch.zeros(1, device="cuda")
    cu = ctypes.CDLL("libcuda.so.1")
    found = []

    def work():
        mine, now = ctypes.c_void_p(), ctypes.c_void_p()
        code = cu.cuCtxCreate_v2(ctypes.byref(mine), 0, 0)
        if code:
            found.append(f"no second context here (driver status {code})")
            return
        name = ctb.ct_conv_transpose_kernel(1, 16, 16, (4, 16, 32), (2, 4, 4), 2, groups=2)
        cu.cuCtxGetCurrent(ctypes.byref(now))
        found.append((name, now.value == mine.value))
        cu.cuCtxDestroy_v2(mine)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    if isinstance(found[0], str):
        pytest.skip(found[0])
    assert found[0][0].startswith("grouped") and found[0][1]
