"""The norm, checkpoint and attention calls on streams other than the current one."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import gen, need_gpu, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def attention(dtype, B, T, H, D):
    g = gen(T)
    q, k, v, do = (randn(g, B, T, H, D, dtype=dtype) for _ in range(4))
    s, ds = randn(g, B, H, D, D), randn(g, B, H, D, D)
    ld = -torch.exp2(-torch.rand(H, generator=g, device="cuda") * 6)
    return (lambda **kw: ct.linear_attention(q, k, v, ld, s, **kw),
            lambda **kw: ct.linear_attention_backward(q, k, v, ld, do, s, ds, **kw))


def calls():
    """Every call that takes a stream, those with a workspace at sizes that use it."""
    g = gen(1)
    x, r, w, dy = (randn(g, *s, dtype="bf16") for s in ((999, 512), (999, 512), (512,), (999, 512)))
    _, h, rstd, kept = ct.rms_norm(x, w, r, quant="int8")
    _, cg, cu = ct.checkpointed_activation(x, r)
    made = {
        "norm": lambda **kw: ct.rms_norm(x, w, r, quant="e4m3", **kw),
        "norm_back": lambda **kw: ct.rms_norm_backward(dy, h, rstd, w, **kw),
        "store": lambda **kw: ct.checkpoint_store(x, "e4m3", 32, **kw),
        "load": lambda **kw: ct.checkpoint_load(kept, **kw),
        "act": lambda **kw: ct.checkpointed_activation(x, r, "gelu", **kw),
        "act_back": lambda **kw: ct.checkpointed_activation_backward(dy, cg, cu, need=("dgate", "dup", "y"), **kw)}
    for dtype in ("bf16", "f16"):
        for name, size in (("segments", (1, 3000, 1, 128)), ("shared", (1, 400, 160, 64)), ("short", (2, 20, 2, 64))):
            made[f"{dtype}_{name}"], made[f"{dtype}_{name}_back"] = attention(dtype, *size)
    made["f32"], made["f32_back"] = attention("f32", 1, 700, 1, 64)
    return made


def tensors(out):
    for t in out if isinstance(out, (tuple, list)) else (out,):
        if isinstance(t, torch.Tensor):
            yield t
        elif isinstance(t, tuple):
            yield from tensors(t)


@pytest.mark.parametrize("form", ["stream", "handle"])
def test_a_given_stream_keeps_its_workspace(form):
    """A call on a stream that is still busy: what the current stream allocates and fills right after it is not the call's memory."""
    made = calls()
    want = {name: [t.clone() for t in tensors(f())] for name, f in made.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for name, f in made.items():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms: the call's kernels start after the fills below
        got = f(stream=side if form == "stream" else side.cuda_stream)
        for size in (1 << 9, 1 << 12, 1 << 16, 1 << 18, 1 << 20, 1 << 22, 1 << 23, 1 << 24, 1 << 26):
            for _ in range(4):
                torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for a, b in zip(want[name], tensors(got)):
            assert a.shape == b.shape and torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


def test_a_stream_of_0_is_the_default_stream():
    x = randn(gen(2), 4, 64)
    y = ct.rms_norm(x)[0]
    assert torch.equal(ct.rms_norm(x, stream=0)[0], y)
    torch.cuda.synchronize()


def test_host_tensors_are_refused_with_a_stream_too():
    with pytest.raises(ct.CtError):
        ct.rms_norm(torch.zeros(4, 64), stream=torch.cuda.Stream())
