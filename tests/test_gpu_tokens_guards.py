"""The C entry points with results inside larger buffers and workspaces of exactly the size asked for: nothing else is written."""
import ctypes
import random

import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import DT, gen, need_gpu, randn

pytestmark = pytest.mark.gpu
MARK = 0x5A


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


class Inside:
    """A [..., cols] result at an odd place of a larger buffer of marks, its leading axes at given strides (elements)."""

    def __init__(self, dtype, shape, strides, offset):
        e = torch.empty((), dtype=dtype).element_size()
        span = 1 + sum((n - 1) * s for n, s in zip(shape, strides)) if all(shape) else 1
        self.bytes = torch.full(((span + 2 * offset + 64) * e,), MARK, dtype=torch.uint8, device="cuda")
        self.t = self.bytes.view(dtype).as_strided(shape, strides, offset)
        self.ptr = self.t.data_ptr()

    def check(self, want):
        assert torch.equal(self.t, want)
        self.t.view(torch.uint8 if self.t.element_size() == 1 else {2: torch.int16, 4: torch.int32}[self.t.element_size()]).fill_(
            MARK * (0x0101 if self.t.element_size() == 2 else 0x01010101))
        assert (self.bytes == MARK).all(), "something beside the result was written"


class Workspace:
    """As many bytes as were asked for, between marks."""

    def __init__(self, n):
        self.n, self.all = n, torch.full((n + 2048,), MARK, dtype=torch.uint8, device="cuda")
        self.ptr = self.all.data_ptr() + 1024 if n else None

    def check(self):
        assert (self.all[:1024] == MARK).all() and (self.all[1024 + self.n:] == MARK).all(), "written outside the workspace"


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def asked(fn, *args):
    n = ctypes.c_size_t(0)
    assert fn(*args, ctypes.byref(n)) == ct.CT_OK
    return n.value


def pick(rng, dense):
    """(row stride, offset): aligned, wide, odd."""
    return rng.choice([(dense, 8), (dense + 8, 16), ((dense + 7) // 8 * 8, 8), (dense + rng.randint(0, 9), rng.randint(1, 9))])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("seed", range(30))
def test_gated_projection(seed, dtype):
    rng = random.Random(100 * seed + len(dtype))
    g = gen(seed)
    rows, C, F = rng.choice([1, 3, 4, 5, 16, 17, 100, 129, 300, rng.randint(1, 700)]), rng.choice([8, 64, 520, rng.randint(1, 600)]), rng.choice(
        [8, 96, 264, 1000, rng.randint(1, 900)])
    f_dense = rng.random() < 0.5
    x, dy = (randn(g, rows, n + p, dtype=dtype)[:, p:] for n, p in ((C, rng.choice([0, 0, 8, 3])), (F, rng.choice([0, 0, 8, 1]))))
    wg, wu = (randn(g, C, F + p, std=C ** -0.5, dtype=dtype)[:, :F] if f_dense else randn(g, F, C + p, std=C ** -0.5, dtype=dtype)[:, :C].t()
              for p in (rng.choice([0, 0, 8, 5]),) * 2)
    want = ct.gated_projection(x, wg, wu, "gelu"), *ct.gated_projection_backward(dy, x, wg, wu, "gelu")
    dt, code, lib, stream = DT[dtype], ct.dtype_code(DT[dtype]), ct.lib(), torch.cuda.current_stream().cuda_stream
    sy, sx = pick(rng, F), pick(rng, C)
    y, dx = Inside(dt, (rows, F), (sy[0], 1), sy[1]), Inside(dt, (rows, C), (sx[0], 1), sx[1])
    sw = [pick(rng, F if f_dense else C) for _ in range(2)]
    dw = [Inside(dt, (C, F), (s, 1) if f_dense else (1, s), o) for s, o in sw]
    # aligned as the call finds it
    e = x.element_size()
    lies = lambda t, r, s: t.data_ptr() % 16 == 0 and (r <= 1 or s * e % 16 == 0)  # noqa: E731
    on_f = f_dense or F <= 1
    weights = all(lies(w, C if on_f else F, w.stride(0) if on_f else w.stride(1)) for w in (wg, wu))
    flags = (2 if on_f else 4) * weights + (weights and lies(x, rows, x.stride(0)))
    ws = Workspace(asked(lib.ct_gated_projection_workspace_bytes, rows, C, F, code, 0, flags))
    st = [i64(*w.stride()) for w in (wg, wu)]
    assert lib.ct_gated_projection_forward(x.data_ptr(), x.stride(0), wg.data_ptr(), st[0], wu.data_ptr(), st[1], y.ptr, sy[0], ws.ptr, ws.n, rows, C, F, 4,
                                           0.0, code, stream) == ct.CT_OK, ct.ct.ct_last_error()
    y.check(want[0])
    ws.check()
    on_f = F <= 1 or all(t.stride(1) == 1 for t in (wg, wu, dw[0].t, dw[1].t))
    weights = all(lies(w, C if on_f else F, w.stride(0) if on_f else w.stride(1)) for w in (wg, wu))
    ws = Workspace(asked(lib.ct_gated_projection_workspace_bytes, rows, C, F, code, 1,
                         int(weights and lies(x, rows, x.stride(0)) and lies(dy, rows, dy.stride(0)))))
    assert lib.ct_gated_projection_backward(dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), wg.data_ptr(), st[0], wu.data_ptr(), st[1], dx.ptr, sx[0],
                                            dw[0].ptr, i64(*dw[0].t.stride()), dw[1].ptr, i64(*dw[1].t.stride()), ws.ptr, ws.n, rows, C, F, 4, 0.0, code,
                                            stream) == ct.CT_OK, ct.ct.ct_last_error()
    ws.check()
    for got, ref in zip((dx, *dw), want[1:]):
        got.check(ref)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("seed", range(30))
def test_group_norm(seed, dtype):
    rng = random.Random(100 * seed + len(dtype) + 7)
    g = gen(seed)
    G = rng.choice([1, 2, 4, 8, 32])
    C, B = G * rng.choice([1, 2, 3, 8, 17, 64]), rng.choice([1, 2, 5])
    S = rng.choice([1, 2, 15, 300, 3000, 40000]) if C < 200 else rng.choice([1, 40, 2000])
    x, dy, w, b = (randn(g, B, S, C, dtype=dtype), randn(g, B, S, C, dtype=dtype), randn(g, C, dtype=dtype), randn(g, C, dtype=dtype))
    y, mean, rstd = ct.group_norm(x, G, w, b, activation="silu")
    want = ct.group_norm_backward(dy, x, mean, rstd, w, b, "silu")
    dt, code, lib, stream = DT[dtype], ct.dtype_code(DT[dtype]), ct.lib(), torch.cuda.current_stream().cuda_stream
    dense = (C, 8) if rng.random() < 0.5 else None  # a vector width like the dense call's: the same sums in the same order
    (row, off), gap = dense or pick(rng, C), rng.choice([0, 8])
    out = [Inside(dt, (B, S, C), (S * row + gap, row, 1), off) for _ in range(2)]
    stats = [Inside(torch.float32, (B, G), (G, 1), 3) for _ in range(2)]
    dwb = [Inside(dt, (C,), (1,), 5) for _ in range(2)]
    sx, so = i64(S * C, C), i64(S * row + gap, row)
    ws = Workspace(asked(lib.ct_group_norm_workspace_bytes, B, S, C, G, code, 0))
    assert lib.ct_group_norm_forward(x.data_ptr(), sx, w.data_ptr(), b.data_ptr(), out[0].ptr, so, stats[0].ptr, stats[1].ptr, ws.ptr, ws.n, B, S, C, G, 1e-5,
                                     3, 0.0, code, stream) == ct.CT_OK
    ws.check()
    ws = Workspace(asked(lib.ct_group_norm_workspace_bytes, B, S, C, G, code, 1))
    assert lib.ct_group_norm_backward(dy.data_ptr(), sx, x.data_ptr(), sx, mean.data_ptr(), rstd.data_ptr(), w.data_ptr(), b.data_ptr(), out[1].ptr, so,
                                      dwb[0].ptr, dwb[1].ptr, ws.ptr, ws.n, B, S, C, G, 3, 0.0, code, stream) == ct.CT_OK
    ws.check()
    # another vector width sums in another order: then only that nothing else was written, and values near
    same = C % 8 == 0 and row % 8 == 0 and off % 8 == 0 and gap % 8 == 0
    for got, ref in zip((out[0], *stats, out[1], *dwb), (y, mean, rstd, *want)):
        if not same:
            assert (got.t.double() - ref.double()).abs().max() <= 0.02 * ref.double().abs().max() + 1e-6
        got.check(ref if same else got.t.clone())
