"""What the sums of two 16-bit numbers in attention's products are for: the last state's digits, and outputs that are exact."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import DT, gen, need_gpu, randn, scan_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def off(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


# The rounding of a state's terms: bf16 keeps a decayed key as two numbers, the
# second good to 2^-9 of the first one's 2^-9, 2^-18 = 3.8e-6 at most; f16's
# two come to 2^-24, as do fp32's products, and what the sums of a few hundred
# such terms add stays below ten times that.
STATE = {"bf16": 4e-6 + 6e-7, "f16": 7e-7, "f32": 7e-7}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("B,T,H,Dk,Dv", [(2, 600, 2, 64, 64), (2, 600, 2, 128, 128), (1, 2500, 1, 128, 64), (1, 700, 160, 64, 128)])
def test_states_keep_their_digits(B, T, H, Dk, Dv, dtype):
    g = gen(T + Dk)
    q, k, v, do = (randn(g, B, T, H, D, dtype=dtype) for D in (Dk, Dk, Dv, Dv))
    ld = -torch.exp2(-1.0 - 7.0 * torch.rand(H, generator=g, device="cuda"))
    s, ds = randn(g, B, H, Dk, Dv), randn(g, B, H, Dk, Dv)
    _, last = ct.linear_attention(q, k, v, ld, s)
    first = ct.linear_attention_backward(q, k, v, ld, do, s, ds, need=("dstate",))[3]
    all_four = ct.linear_attention_backward(q, k, v, ld, do, s, ds)
    decay = torch.exp(ld.double())
    ref = scan_ref(q, k, v, s, decay, None, 1.0, 1.0, False)[1]
    assert off(last, ref) <= STATE[dtype]
    ref = scan_ref(k, q, do, ds, decay, None, Dk ** -0.5, 1.0, True)[1]
    assert off(first, ref) <= STATE[dtype] and off(all_four[3], ref) <= STATE[dtype]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("B,T,H,D", [(2, 300, 2, 64), (2, 300, 2, 128), (1, 1600, 1, 64), (1, 700, 160, 64), (3, 26, 2, 64)])
def test_outputs_that_are_whole_numbers(B, T, H, D, dtype):
    """No decay and whole numbers: keys in pairs that differ by one in their last place, with opposite values, and a state whose
    rows in pairs nearly cancel under q.  Scores and state need 11 bits and more; what is left of them after every second token
    is a small whole number, and any digit lost on the way shows in it."""
    g = gen(D + T)

    def whole(top, *shape):
        return torch.randint(-top, top + 1, shape, generator=g, device="cuda").float()

    q, k, v = whole(4, B, T, H, D), whole(64, B, T, H, D), whole(1, B, T, H, D)
    q[..., 1:D - 2:2] = -q[..., 0:D - 2:2]
    q[..., -2], q[..., -1] = 0, whole(1, B, T, H)
    k[:, 1::2], v[:, 1::2] = k[:, ::2], -v[:, ::2]
    k[..., -1] = torch.arange(T, device="cuda").view(1, T, 1) % 2
    s = whole(4000, B, H, D, D)
    s[:, :, 1:D - 2:2] = s[:, :, 0:D - 2:2] + whole(1, B, H, D // 2 - 1, D)
    s[:, :, -1] = whole(2, B, H, D)
    qd, kd, vd, sd = (t.double() for t in (q, k, v, s))
    o, last = ct.linear_attention(*(t.to(DT[dtype]) for t in (q, k, v)), torch.zeros(H, device="cuda"), s, scale=1.0)
    ref, refm = scan_ref(qd, kd, vd, sd, torch.ones(H, device="cuda").double(), None, 1.0, 1.0, False)
    assert ref[:, 1::2].abs().max() <= 256 and ref[:, ::2].abs().max() > 1024
    assert torch.equal(o[:, 1::2].double(), ref[:, 1::2])
    assert torch.equal(last.double(), refm)
