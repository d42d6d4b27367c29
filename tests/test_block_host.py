"""Refusals of the norm, checkpoint and linear-attention calls: every one comes before any device work (no GPU needed)."""
import ctypes

import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from transposed_convolution_convtranspose1_gb300 import _build
from transposed_convolution_convtranspose1_gb300 import ct as ctb

P = 1 << 20  # a pointer that is never read


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return ctb.lib()


def norm(lib, **kw):
    p = dict(x=P, xs=64, r=P, rs=64, w=P, y=P, ys=64, h=P, hs=64, rstd=P, codes=P, scales=P, rows=4, cols=64, eps=1e-6,
             dtype=ctb.CT_BF16, quant=1, group=128)
    p.update(kw)
    return lib.ct_rms_norm_forward(p["x"], p["xs"], p["r"], p["rs"], p["w"], p["y"], p["ys"], p["h"], p["hs"], p["rstd"], p["codes"],
                                   p["scales"], p["rows"], p["cols"], p["eps"], p["dtype"], p["quant"], p["group"], None)


def test_norm_refusals(lib):
    for kw, rc in ((dict(dtype=3), ctb.CT_ERR_DTYPE), (dict(rows=-1), ctb.CT_ERR_SHAPE), (dict(cols=0), ctb.CT_ERR_SHAPE),
                   (dict(cols=1 << 25), ctb.CT_ERR_TOO_LARGE), (dict(quant=3), ctb.CT_ERR_PARAM), (dict(group=48), ctb.CT_ERR_PARAM),
                   (dict(group=256), ctb.CT_ERR_PARAM), (dict(eps=-1.0), ctb.CT_ERR_PARAM), (dict(eps=float("nan")), ctb.CT_ERR_PARAM),
                   (dict(x=None), ctb.CT_ERR_NULL), (dict(codes=None), ctb.CT_ERR_NULL), (dict(scales=None), ctb.CT_ERR_NULL),
                   (dict(x=P + 1), ctb.CT_ERR_ALIGN), (dict(scales=P + 2), ctb.CT_ERR_ALIGN), (dict(rows=0), ctb.CT_OK)):
        assert norm(lib, **kw) == rc, kw
        if rc != ctb.CT_OK:
            assert ctb.ct_last_error()


def norm_back(lib, **kw):
    p = dict(dy=P, h=P, rstd=P, w=P, dres=P, dx=P, dw=P, ws=P, nws=1 << 40, rows=4, cols=64, dtype=ctb.CT_F32)
    p.update(kw)
    return lib.ct_rms_norm_backward(p["dy"], 64, p["h"], 64, p["rstd"], p["w"], p["dres"], 64, p["dx"], 64, p["dw"], p["ws"], p["nws"],
                                    p["rows"], p["cols"], p["dtype"], None)


def test_norm_backward_refusals(lib):
    for kw, rc in ((dict(dtype=9), ctb.CT_ERR_DTYPE), (dict(cols=0), ctb.CT_ERR_SHAPE), (dict(dy=None), ctb.CT_ERR_NULL),
                   (dict(h=None), ctb.CT_ERR_NULL), (dict(rstd=None), ctb.CT_ERR_NULL), (dict(dx=P + 2), ctb.CT_ERR_ALIGN),
                   (dict(dx=None, dw=None), ctb.CT_OK), (dict(rows=0, dw=None), ctb.CT_OK)):
        assert norm_back(lib, **kw) == rc, kw
    n = ctypes.c_size_t(0)
    assert lib.ct_rms_norm_backward_workspace_bytes(1000, 64, 0, ctypes.byref(n)) == ctb.CT_OK and n.value > 0
    assert lib.ct_rms_norm_backward_workspace_bytes(1000, 64, 0, None) == ctb.CT_ERR_NULL


def act(lib, **kw):
    p = dict(gate=P, up=P, y=P, gc=P, gs=P, uc=P, us=P, rows=4, cols=64, act=3, dtype=ctb.CT_F16, quant=1, group=64)
    p.update(kw)
    return lib.ct_checkpointed_activation_forward(p["gate"], 64, p["up"], 64, p["y"], 64, p["gc"], p["gs"], p["uc"], p["us"], p["rows"],
                                                  p["cols"], p["act"], 0.0, p["dtype"], p["quant"], p["group"], None)


def test_activation_refusals(lib):
    for kw, rc in ((dict(dtype=-1), ctb.CT_ERR_DTYPE), (dict(rows=-2), ctb.CT_ERR_SHAPE), (dict(cols=-1), ctb.CT_ERR_SHAPE),
                   (dict(quant=0), ctb.CT_ERR_PARAM), (dict(group=16), ctb.CT_ERR_PARAM), (dict(act=7), ctb.CT_ERR_PARAM),
                   (dict(act=-1), ctb.CT_ERR_PARAM), (dict(gate=None), ctb.CT_ERR_NULL), (dict(gc=None), ctb.CT_ERR_NULL),
                   (dict(us=None), ctb.CT_ERR_NULL), (dict(y=P + 1), ctb.CT_ERR_ALIGN), (dict(cols=1 << 31), ctb.CT_ERR_TOO_LARGE),
                   (dict(rows=0), ctb.CT_OK), (dict(cols=0), ctb.CT_OK)):
        assert act(lib, **kw) == rc, kw
    back = lib.ct_checkpointed_activation_backward
    assert back(None, 0, P, P, P, P, P, 64, None, 0, None, 0, 4, 64, 3, 0.0, 1, 1, 64, None) == ctb.CT_ERR_NULL  # dgate without dy
    assert back(P, 64, P, P, None, None, P, 64, P, 64, None, 0, 4, 64, 3, 0.0, 1, 1, 64, None) == ctb.CT_ERR_NULL  # dup without up
    assert back(P, 64, P, P, P, P, None, 0, None, 0, None, 0, 4, 64, 3, 0.0, 1, 1, 64, None) == ctb.CT_OK
    assert lib.ct_checkpoint_store(P, 64, None, P, 4, 64, 1, 1, 64, None) == ctb.CT_ERR_NULL
    assert lib.ct_checkpoint_load(P, P, None, 64, 4, 64, 1, 1, 64, None) == ctb.CT_ERR_NULL
    assert lib.ct_checkpoint_load(P, P, P, 64, 4, 64, 1, 5, 64, None) == ctb.CT_ERR_PARAM


S3 = (ctypes.c_int64 * 3)(0, 0, 0)


def attention(lib, **kw):
    p = dict(q=P, k=P, v=P, o=P, s=S3, ld=P, lengths=P, si=P, so=P, B=1, T=4, H=2, Dk=8, Dv=8, dtype=ctb.CT_BF16)
    p.update(kw)
    return lib.ct_linear_attention_forward(p["q"], p["s"], p["k"], S3, p["v"], S3, p["o"], S3, p["ld"], p["si"], p["so"], p["lengths"],
                                           None, 0, p["B"], p["T"], p["H"], p["Dk"], p["Dv"], 1.0, p["dtype"], None)


def test_attention_refusals(lib):
    for kw, rc in ((dict(dtype=3), ctb.CT_ERR_DTYPE), (dict(B=-1), ctb.CT_ERR_SHAPE), (dict(Dk=0), ctb.CT_ERR_SHAPE),
                   (dict(Dv=0), ctb.CT_ERR_SHAPE), (dict(T=-1), ctb.CT_ERR_SHAPE), (dict(Dk=257), ctb.CT_ERR_TOO_LARGE),
                   (dict(T=1 << 31), ctb.CT_ERR_TOO_LARGE), (dict(B=1 << 20, H=1 << 15), ctb.CT_ERR_TOO_LARGE),
                   (dict(q=None), ctb.CT_ERR_NULL), (dict(o=None), ctb.CT_ERR_NULL), (dict(ld=None), ctb.CT_ERR_NULL),
                   (dict(s=None), ctb.CT_ERR_NULL), (dict(k=P + 1), ctb.CT_ERR_ALIGN), (dict(lengths=P + 2), ctb.CT_ERR_ALIGN),
                   (dict(si=P + 2), ctb.CT_ERR_ALIGN), (dict(B=0), ctb.CT_OK), (dict(H=0), ctb.CT_OK)):
        assert attention(lib, **kw) == rc, kw
    n = ctypes.c_size_t(0)
    w = lib.ct_linear_attention_workspace_bytes
    assert w(1, 100, 2, 64, 64, 1, 0, ctypes.byref(n)) == ctb.CT_OK
    assert w(1, 100, 2, 64, 64, 1, 0, None) == ctb.CT_ERR_NULL and w(1, 100, 2, 300, 64, 1, 1, ctypes.byref(n)) == ctb.CT_ERR_TOO_LARGE
    back = lib.ct_linear_attention_backward
    args = [P, S3, P, S3, P, S3, None, S3, P, None, None, None, P, S3, P, S3, P, S3, None, None, 0, 1, 4, 2, 8, 8, 1.0, 1, None]
    assert back(*args) == ctb.CT_ERR_NULL  # no upstream gradient
    args[6], args[13] = P, None
    assert back(*args) == ctb.CT_ERR_NULL  # dq without strides


def test_bindings_refuse_before_the_library():
    x = torch.zeros(4, 64)
    for call in (lambda: ct.rms_norm(x), lambda: ct.checkpoint_store(x), lambda: ct.checkpointed_activation(x),
                 lambda: ct.rms_norm(x, torch.ones(63)), lambda: ct.rms_norm(x, residual=torch.zeros(4, 63)),
                 lambda: ct.rms_norm(x, residual=torch.zeros(4, 64, dtype=torch.float16)), lambda: ct.rms_norm(x, quant="int4"),
                 lambda: ct.checkpoint_store(x, None), lambda: ct.checkpointed_activation(x, activation="swish"),
                 lambda: ct.rms_norm_backward(x, x, torch.ones(3)),
                 lambda: ct.checkpoint_load(ct.Checkpoint(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2), 64, torch.float32))):
        with pytest.raises(ct.CtError):
            call()
    with pytest.raises(ValueError):
        ct.rms_norm(x.t())
    q, ld = torch.zeros(2, 5, 3, 8), torch.zeros(3)
    for call in (lambda: ct.linear_attention(q, q, q, ld), lambda: ct.linear_attention(q, q[:, :4], q, ld),
                 lambda: ct.linear_attention(q, q, q.half(), ld), lambda: ct.linear_attention(q, q, q, torch.zeros(2)),
                 lambda: ct.linear_attention(q, q, q, ld.double()), lambda: ct.linear_attention(q[0], q[0], q[0], ld),
                 lambda: ct.linear_attention(q, q, q, ld, state=torch.zeros(2, 3, 8, 7)),
                 lambda: ct.linear_attention(q, q, q, ld, lengths=torch.zeros(2))):
        with pytest.raises(ct.CtError):
            call()
