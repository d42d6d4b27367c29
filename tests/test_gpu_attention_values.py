"""Linear attention on values at the ends: decays that are NaN, infinities and NaN among the values, small fp16 values."""
import pytest
import torch

import transposed_convolution_convtranspose1_gb300 as ct
from _block import DT, TINY, U, attention_k, gen, need_gpu, randn, scan_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    need_gpu()


def inputs(seed, B, T, H, Dk, Dv, dtype):
    g = gen(seed)
    q, k, v, do = (randn(g, B, T, H, D, dtype=dtype) for D in (Dk, Dk, Dv, Dv))
    ld = -torch.exp2(-torch.rand(H, generator=g, device="cuda") * 6)
    return q, k, v, do, ld, randn(g, B, H, Dk, Dv), randn(g, B, H, Dk, Dv)


def walks(q, k, v, ld, do, s, ds, n, scale):
    """(name, index of the call's output, index of its last matrix or None, the walk) of the four uses of the recurrence."""
    st, dst = (None if t is None else t.transpose(2, 3) for t in (s, ds))
    return (("o", 0, 1, (q, k, v, s, n, 1.0, scale, False)), ("dq", 2, None, (do, v, k, st, n, 1.0, scale, False)),
            ("dk", 3, None, (v, do, q, dst, n, scale, 1.0, True)), ("dv", 4, 5, (k, q, do, ds, n, scale, 1.0, True)))


def outputs(q, k, v, ld, do, s, ds, n=None, scale=None):
    return ct.linear_attention(q, k, v, ld, s, n, scale) + ct.linear_attention_backward(q, k, v, ld, do, s, ds, n, scale)


def reference(ld, walk):
    z, x, y, m, n, ms, os, rev = walk
    ref = scan_ref(z, x, y, m, torch.exp(ld.double()), n, ms, os, rev)
    mag = scan_ref(z.abs(), x.abs(), y.abs(), None if m is None else m.abs(), torch.exp(ld.double()), n, ms, os, rev)
    return ref, mag


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


# ---- values that are not finite ----------------------------------------------

GEOMETRY = {"walks": (2, 300, 2), "segments": (1, 1700, 1), "shared": (1, 1100, 155)}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("where", list(GEOMETRY))
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (40, 128)])
def test_what_is_not_finite_reaches_only_those_who_see_it(dtype, where, Dk, Dv):
    """Outputs are not finite exactly where the recurrence's are; all others keep their bounds, in the same chunk too."""
    B, T, H = GEOMETRY[where]
    q, k, v, do, ld, s, ds = inputs(Dk + Dv + T, B, T, H, Dk, Dv, dtype)
    inf, nan = float("inf"), float("nan")
    heads = range(0, H, 5)  # the others stay finite
    for i, h in enumerate(heads):
        kind = i % 3
        if kind == 0:  # v in two columns, one after the other
            v[-1, 70, h, 3] = inf
            v[-1, 200, h, 9] = nan
            do[-1, 211, h, 1] = -inf
        elif kind == 1:  # k: all columns from there on
            k[-1, 77, h, 5] = nan
            do[-1, T - 3, h, 2] = nan
        else:  # q: its own token forward in time
            q[-1, 130, h, 4] = inf
            v[-1, T - 1, h, 0] = inf
    if H == 1:
        q[-1, 60, 0, 4] = nan
    if where == "segments":  # heads before tokens
        q, k, v, do = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v, do))
    got = outputs(q, k, v, ld, do, s, ds)
    over = s.clone()
    o, _ = ct.linear_attention(q, k, v, ld, over, state_out=over)
    for a, b in ((o, got[0]), (over, got[1])):  # the last state in the first one's place
        assert torch.equal(a.nan_to_num(7, 8, 9), b.nan_to_num(7, 8, 9))
    for name, i, j, walk in walks(q, k, v, ld, do, s, ds, None, Dk ** -0.5):
        (ref, refm), (mag, magm) = reference(ld, walk)
        kk = attention_k(T, walk[1].shape[3], dtype)
        for what, g, r, m, u, tiny in ((name, got[i], ref, mag, U[dtype], TINY[dtype]),
                                       (name + " state", None if j is None else got[j], refm, magm, 0.0, 0.0)):
            if g is None:
                continue
            fine = torch.isfinite(r)
            assert 0 < fine.sum() < fine.numel()
            wrong = torch.isfinite(g) != fine
            assert not wrong.any(), f"{what}: {wrong.sum().item()} of {wrong.numel()} finite or not in the wrong place"
            off = ((g.double() - r).abs() - (r.abs() * u + m * kk + tiny))[fine]
            assert off.max().item() <= 0, f"{what}: {off.max().item():.3e} over its bound"


# ---- small fp16 values -----------------------------------------------------------

def off(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (64, 128)])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-5, 3e-6])
@pytest.mark.parametrize("small", ["do", "k and v", "state"])
def test_small_fp16_values_keep_their_digits(Dk, Dv, size, small):
    """Gradients of the sizes that a mean loss gives, small keys and values, a small state read by large queries: no output is
    further from 64 bits than rounding it to fp16 and 2^-17 of its terms come to."""
    B, T, H = 2, 300, 2
    q, k, v, do, ld, s, ds = inputs(Dk + Dv, B, T, H, Dk, Dv, "f16")
    ld = -torch.tensor([1.0 / 128, 1.0 / 16], device="cuda")
    if small == "do":
        do, s, ds = do * size, None, None
    elif small == "k and v":
        k, v, s, ds = k * size ** 0.5, v * size ** 0.5, s * size, None
    else:
        q, k, v, s, ds = q * 64, k * size, v * size, s * size, None
    got = outputs(q, k, v, ld, do, s, ds)
    for name, i, j, walk in walks(q, k, v, ld, do, s, ds, None, Dk ** -0.5):
        (ref, refm), (mag, magm) = reference(ld, walk)
        rounded = off(ref.half(), ref)
        limit = 1.05 * rounded + 2.0 ** -17 * (mag.norm() / ref.norm()).item()
        assert off(got[i], ref) <= limit, f"{name}: {off(got[i], ref):.2e}, rounding alone {rounded:.2e}, limit {limit:.2e}"
        if j is not None and got[j] is not None:
            limit = 2.0 ** -17 * (magm.norm() / refm.norm()).item()
            assert off(got[j], refm) <= limit, f"{name} state: {off(got[j], refm):.2e}, limit {limit:.2e}"
