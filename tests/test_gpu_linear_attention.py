"""Linear attention with a decay for each head: forward, streaming steps and gradients against the recurrence in 64 bits."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import (DT, E, check_attention, check_attention_back, gen, need_gpu, randn, scan_ref)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def inputs(seed, B, T, H, Dk, Dv, dtype, layout="bthd"):
    g = gen(seed)

    def heads(D):
        if layout == "bhtd":
            return randn(g, B, H, T, D, dtype=dtype).transpose(1, 2)
        if layout == "offset":  # rows that start off 16-byte boundaries
            return randn(g, B, T, H, D + 3, dtype=dtype)[..., 1:1 + D]
        return randn(g, B, T, H, D, dtype=dtype)

    q, k, v, do = heads(Dk), heads(Dk), heads(Dv), heads(Dv)
    ld = -torch.exp2(-torch.rand(H, generator=g, device="cuda") * 8)
    return q, k, v, do, ld, randn(g, B, H, Dk, Dv), randn(g, B, H, Dk, Dv)


def run_all(seed, B, T, H, Dk, Dv, dtype, layout="bthd", lengths=None, states=True, ld=None):
    q, k, v, do, decays, s, ds = inputs(seed, B, T, H, Dk, Dv, dtype, layout)
    decays = decays if ld is None else ld
    if not states:
        s = ds = None
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    scale = Dk ** -0.5
    o, last = ct.linear_attention(q, k, v, decays, s, n)
    check_attention(dtype, q, k, v, decays, s, n, scale, o, last)
    dq, dk, dv, df = ct.linear_attention_backward(q, k, v, decays, do, s, ds, n)
    check_attention_back(dtype, q, k, v, decays, do, s, ds, n, scale, dq, dk, dv, df)
    assert (df is None) == (s is None)
    return o, last


SIZES = [(1, 1), (16, 16), (40, 72), (64, 64), (128, 128), (128, 64), (64, 128), (33, 65), (96, 48), (130, 20), (256, 256), (8, 200)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("Dk,Dv", SIZES)
def test_head_sizes(Dk, Dv, dtype):
    run_all(Dk * 300 + Dv, 2, 150, 3, Dk, Dv, dtype)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 256, 257, 513])
@pytest.mark.parametrize("D", [64, 128])
def test_lengths_of_all_sizes(T, D, dtype):
    run_all(T, 1, T, 2, D, D, dtype, states=T % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,D", [(4096, 64), (3001, 128), (5000, 80)])
def test_long_sequences_on_few_heads(T, D, dtype):
    run_all(T, 1, T, 1, D, D, dtype)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("layout", ["bthd", "bhtd", "offset"])
@pytest.mark.parametrize("D,T", [(64, 300), (128, 260), (48, 140)])
def test_unequal_lengths_and_layouts(dtype, layout, D, T):
    """Lengths from none to more than T (taken as T); every layout gives the same result."""
    o, last = run_all(D + T, 5, T, 2, D, D, dtype, layout, lengths=[0, 1, T // 2 + 3, T, T + 9])
    assert (o[0] == 0).all() and (o[1, 1:] == 0).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
def test_what_lies_after_the_length_is_not_used(dtype, D):
    """NaN and infinities after a sequence's end change nothing, in no direction."""
    T, lengths = 200, [0, 70, 129, 200]
    q, k, v, do, ld, s, ds = inputs(3, 4, T, 2, D, D, dtype)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    clean = (ct.linear_attention(q, k, v, ld, s, n) + ct.linear_attention_backward(q, k, v, ld, do, s, ds, n))
    for t in (q, k, v, do):
        for b, m in enumerate(lengths):
            t[b, m:] = float("nan")
            t[b, m + 1::2] = float("inf")
    dirty = (ct.linear_attention(q, k, v, ld, s, n) + ct.linear_attention_backward(q, k, v, ld, do, s, ds, n))
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)
    assert torch.equal(dirty[1][0], s[0])  # an empty sequence hands its state on


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
def test_decays_at_their_ends(dtype, D):
    """No decay, decays so strong that their powers vanish, and none left at all (-infinity)."""
    ld = torch.tensor([0.0, -1e-6, -3.0, -40.0, -1e4, float("-inf")], device="cuda")
    run_all(11, 2, 190, 6, D, D, dtype, ld=ld)
    o, _ = ct.linear_attention(*inputs(5, 1, 150, 1, D, D, dtype)[:3], torch.tensor([float("-inf")], device="cuda"))
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cuts", [(1, 1, 1, 1, 1, 1), (64, 1, 1, 129, 1, 63), (150, 109)])
def test_streaming_equals_the_whole(dtype, cuts):
    """A prompt and then single tokens, the state carried in place, against one call on all of it."""
    T, B, H, D = sum(cuts), 3, 2, 64
    q, k, v, _, ld, s, _ = inputs(T, B, T, H, D, D, dtype)
    state, outs, t = s.clone(), [], 0
    for c in cuts:
        o, same = ct.linear_attention(q[:, t:t + c], k[:, t:t + c], v[:, t:t + c], ld, state, state_out=state)
        assert same is state
        outs.append(o)
        t += c
    check_attention(dtype, q, k, v, ld, s, None, D ** -0.5, torch.cat(outs, 1), state)


@pytest.mark.parametrize("dtype", list(DT))
def test_no_tokens(dtype):
    q = torch.empty(2, 0, 3, 64, dtype=DT[dtype], device="cuda")
    s = torch.randn(2, 3, 64, 64, device="cuda")
    ld = -torch.ones(3, device="cuda")
    o, last = ct.linear_attention(q, q, q, ld, s)
    assert o.shape == q.shape and torch.equal(last, s)
    o, last = ct.linear_attention(q, q, q, ld)
    assert (last == 0).all()
    dq, dk, dv, df = ct.linear_attention_backward(q, q, q, ld, q, s, s)
    assert dq.shape == q.shape and torch.equal(df, s)
    e = torch.empty(0, 5, 3, 64, dtype=DT[dtype], device="cuda")
    o, last = ct.linear_attention(e, e, e, ld)
    assert o.shape == e.shape and last.shape == (0, 3, 64, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_projection_for_all_three(dtype):
    """q, k and v as slices of one [B, T, 3, H, D] projection; reproducible; on another stream."""
    g = gen(2)
    p = randn(g, 2, 333, 3, 4, 64, dtype=dtype)
    q, k, v = p[:, :, 0], p[:, :, 1], p[:, :, 2]
    ld = -torch.tensor([0.5, 0.1, 0.01, 0.002], device="cuda")
    o, last = ct.linear_attention(q, k, v, ld, scale=0.25)
    check_attention(dtype, q, k, v, ld, None, None, 0.25, o, last)
    again = ct.linear_attention(q.contiguous(), k.contiguous(), v.contiguous(), ld, scale=0.25)
    assert torch.equal(o, again[0]) and torch.equal(last, again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, last2 = ct.linear_attention(q, k, v, ld, scale=0.25)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(last, last2)
    none = ct.linear_attention(q, k, v, ld, scale=0.25, need=())
    assert none[1] is None and torch.equal(none[0], o)


def test_only_the_gradients_asked_for():
    q, k, v, do, ld, s, ds = inputs(9, 1, 140, 2, 64, 64, "bf16")
    every = ct.linear_attention_backward(q, k, v, ld, do, s, ds)
    for i, name in enumerate(("dq", "dk", "dv", "dstate")):
        got = ct.linear_attention_backward(q, k, v, ld, do, s, ds, need=(name,))
        assert [t is None for t in got] == [j != i for j in range(4)] and torch.equal(got[i], every[i])


def test_autograd_against_differences():
    """The recorded gradient of a scalar of o and the last state against central differences in 64 bits."""
    B, T, H, D = 2, 37, 2, 24
    q, k, v, do, ld, s, ds = inputs(4, B, T, H, D, D, "f32")
    n = torch.tensor([37, 20], dtype=torch.int32, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (q, k, v, s)]
    o, last = ct.linear_attention_autograd(leaves[0], leaves[1], leaves[2], ld, leaves[3], n, 0.3)
    ((o * do).sum() + (last * ds).sum()).backward()

    def f(q, k, v, s):
        o, m = scan_ref(q, k, v, s, torch.exp(ld.double()), n, 1.0, 0.3, False)
        return (o * do.double()).sum() + (m * ds.double()).sum()

    base = [t.double() for t in (q, k, v, s)]
    g = gen(77)
    step = 1e-5
    for i in range(4):
        d = torch.randn(base[i].shape, generator=g, device="cuda").double()
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + step * d, base[i] - step * d
        want = ((f(*up) - f(*down)) / (2 * step)).item()
        terms = leaves[i].grad.double() * d
        assert abs(terms.sum().item() - want) <= 300 * E * terms.abs().sum().item() + 1e-4


def test_f16_scores_and_states_beyond_its_range():
    """Scores and states too large for f16 (the result is not): the heads concerned are computed again, exactly as asked."""
    B, T, H, D = 1, 300, 3, 64
    q, k, v, do, ld, s, ds = inputs(31, B, T, H, D, D, "f16")
    ld = torch.tensor([0.0, -0.01, -0.5], device="cuda")
    q[:, :, 0] *= 60
    k[:, :, 0] *= 60         # scores of 1e5
    v[:, :, 0] *= 2.0 ** -10
    s[:, 1] *= 1e6           # a state of 1e6, queries that bring it back
    q[:, :, 1] *= 1e-3
    o, last = ct.linear_attention(q, k, v, ld, s)
    check_attention("f16", q, k, v, ld, s, None, D ** -0.5, o, last)
    state = s.clone()
    o2, last2 = ct.linear_attention(q, k, v, ld, state, state_out=state)
    assert torch.equal(o, o2) and torch.equal(last, state)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_wait_that_gives_up_is_reported(dtype):
    """With no time to wait the tensor-core kernel stops, reports it and leaves the device usable."""
    q, k, v, do, ld, s, _ = inputs(8, 2, 700, 2, 128, 128, dtype)
    good = ct.linear_attention(q, k, v, ld, s)
    torch.cuda.synchronize()
    assert ct.ct_device_status(clear=True) == (ct.CT_OK, 0)
    before = ct.ct_set_wait_limit_ns(0)
    try:
        ct.linear_attention(q, k, v, ld, s)
        torch.cuda.synchronize()
    finally:
        ct.ct_set_wait_limit_ns(before)
    rc, code = ct.ct_device_status(clear=True)
    assert rc == ct.ct.CT_ERR_DEVICE_TIMEOUT and code != 0
    again = ct.linear_attention(q, k, v, ld, s)
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
    assert ct.ct_device_status(clear=True) == (ct.CT_OK, 0)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128, 48])
def test_unequal_lengths_in_segments(dtype, D):
    """Few heads, so that sequences are cut into segments, some of them behind a sequence's end."""
    run_all(D, 3, 1700, 1, D, D, dtype, lengths=[0, 700, 1700])
    run_all(D + 1, 2, 1100, 1, D, D, dtype, lengths=[1024, 1], states=False)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T", [1, 90, 1500])
def test_first_gradient_over_the_last(dtype, T):
    """dstate_in written over dstate_out, and a workspace of the call's own, through the C entry point."""
    B, H, D = 2, 1, 64
    q, k, v, do, ld, s, ds = inputs(T, B, T, H, D, D, dtype)
    want = ct.linear_attention_backward(q, k, v, ld, do, s, ds)
    st = ct.block._I64x3(T * H * D, H * D, D)
    over, out = ds.clone(), [torch.empty_like(q) for _ in range(3)]
    rc = ct.lib().ct_linear_attention_backward(
        q.data_ptr(), st, k.data_ptr(), st, v.data_ptr(), st, do.data_ptr(), st, ld.data_ptr(), s.data_ptr(), over.data_ptr(), None,
        out[0].data_ptr(), st, out[1].data_ptr(), st, out[2].data_ptr(), st, over.data_ptr(), None, 0, B, T, H, D, D, D ** -0.5,
        ct.dtype_code(q.dtype), torch.cuda.current_stream().cuda_stream)
    assert rc == ct.CT_OK
    n = None
    check_attention_back(dtype, q, k, v, ld, do, s, ds, n, D ** -0.5, *out, over)
    for a, b in zip(want[:3], out):
        assert a.shape == b.shape
    # a workspace that is too small is refused
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    if T == 1500:
        rc = ct.lib().ct_linear_attention_forward(
            q.data_ptr(), st, k.data_ptr(), st, v.data_ptr(), st, out[0].data_ptr(), st, ld.data_ptr(), None, None, None, ws.data_ptr(),
            256, B, T, H, D, D, 1.0, ct.dtype_code(q.dtype), torch.cuda.current_stream().cuda_stream)
        assert rc == ct.ct.CT_ERR_WORKSPACE


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,T,H,Dk,Dv", [(7, 500, 23, 24, 40), (1, 1100, 155, 64, 64), (2, 300, 111, 72, 128), (19, 400, 9, 128, 33)])
def test_more_walks_than_processors(dtype, B, T, H, Dk, Dv):
    """Walks shared between processors: one begins a walk, the next ends it."""
    run_all(B * T, B, T, H, Dk, Dv, dtype, states=T != 300)
    lengths = [(97 * i) % (T + 1) for i in range(B)]
    run_all(B * T + 1, B, T, H, Dk, Dv, dtype, lengths=lengths)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_shared_walks_in_a_graph(dtype):
    """The launch whose blocks wait for one another, captured and replayed on other values."""
    B, T, H, D = 4, 700, 60, 64
    q, k, v, do, ld, s, ds = inputs(5, B, T, H, D, D, dtype)
    held = [t.clone() for t in (q, k, v, do)]
    ct.linear_attention_backward(*held[:3], ld, held[3], s, ds)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, last = ct.linear_attention(*held[:3], ld, s)
        got = ct.linear_attention_backward(*held[:3], ld, held[3], s, ds)
    for seed in (6, 7):
        new = inputs(seed, B, T, H, D, D, dtype)
        for h, n in zip(held, new):
            h.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        eo, elast = ct.linear_attention(*new[:3], ld, s)
        eager = ct.linear_attention_backward(*new[:3], ld, new[3], s, ds)
        for a, b in zip((o, last, *got), (eo, elast, *eager)):
            assert torch.equal(a, b)
