"""Linear attention on values at the ends: decays that are NaN."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import DT, gen, need_gpu, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def inputs(seed, B, T, H, Dk, Dv, dtype):
    g = gen(seed)
    q, k, v, do = (randn(g, B, T, H, D, dtype=dtype) for D in (Dk, Dk, Dv, Dv))
    ld = -torch.exp2(-torch.rand(H, generator=g, device="cuda") * 6)
    return q, k, v, do, ld, randn(g, B, H, Dk, Dv), randn(g, B, H, Dk, Dv)


def outputs(q, k, v, ld, do, s, ds, n=None, scale=None):
    return ct.linear_attention(q, k, v, ld, s, n, scale) + ct.linear_attention_backward(q, k, v, ld, do, s, ds, n, scale)


# ---- decays that are NaN -------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("B,T,H", [(2, 1, 3), (2, 20, 3), (2, 300, 3), (1, 1700, 2), (1, 700, 155)])
def test_a_decay_that_is_nan(dtype, B, T, H):
    """A NaN decay makes its own head NaN, and no other head differs."""
    D = 64
    q, k, v, do, ld, s, ds = inputs(T, B, T, H, D, D, dtype)
    bad = ld.clone()
    bad[1] = float("nan")
    clean, got = outputs(q, k, v, ld, do, s, ds), outputs(q, k, v, bad, do, s, ds)
    others = [h for h in range(H) if h != 1]
    for i, name in enumerate(("o", "state", "dq", "dk", "dv", "dstate")):
        a, b = (t if name.endswith("state") else t.transpose(1, 2) for t in (clean[i], got[i]))  # [B, H, ...]
        assert torch.equal(a[:, others], b[:, others]), name
        # the last token's own k and v gradients come before any decay
        mine = b[:, 1, :T - 1] if name in ("dk", "dv") else b[:, 1]
        assert torch.isnan(mine).all(), name
