"""Plain 64-bit forms of the norm, checkpoint and linear-attention operators,
and the bounds their fp32 kernels are held to.

U is the unit roundoff of an output type (one rounding to nearest: relative
error at most U).  E = 2^-24 is fp32's.  A sum of n terms added in fp32 in
chains of length m has an error of at most m * E times the sum of the terms'
magnitudes, so each bound below is U * |value| + (chain length + a few) * E *
(the same expression with every term's magnitude).
"""
import torch

import transposed_convolution_convtranspose1_gb300 as ct

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half a subnormal step
E = 2.0 ** -24
TOP = {"int8": 127.0, "e4m3": 448.0}


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape, std=1.0, dtype="f32"):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dtype])


def within(got, ref, bound, what=""):
    """|got - ref| <= bound everywhere; NaN exactly where ref has NaN."""
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    off = torch.where(nan, torch.zeros_like(ref), (got - ref).abs() - bound)
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} over its bound"


# ---- norm ------------------------------------------------------------------

def norm_ref(x, w, r, eps):
    s = x.double() if r is None else x.double() + r.double()
    rstd = ((s * s).mean(-1) + eps).rsqrt()
    y = s * rstd[..., None]
    return s, rstd, y if w is None else y * w.double()


def norm_chain(cols):
    # at most cols / 32 terms a lane, then 5 + 5 joining steps; the square
    # root halves it; s, eps, mean, reciprocal, two products
    return cols / 32 + 32


def check_norm(x, w, r, eps, dtype, y, h, rstd):
    s, rs, yr = norm_ref(x, w, r, eps)
    k = norm_chain(x.shape[-1]) * E
    if rstd is not None:
        within(rstd, rs, rs * k, "rstd")
    if r is not None:
        within(h, s, s.abs() * (U[dtype] + E) + TINY[dtype], "h")
    if y is not None:
        within(y, yr, yr.abs() * (U[dtype] + k) + TINY[dtype], "y")
    return yr


def norm_back_ref(dy, h, rstd, w, dres):
    dy, u, rs = dy.double(), h.double() * rstd.double()[..., None], rstd.double()[..., None]
    wdy = dy if w is None else dy * w.double()
    c = (wdy * u).mean(-1, keepdim=True)
    dx = rs * (wdy - u * c)
    ca = (wdy * u).abs().mean(-1, keepdim=True)
    dxa = rs * (wdy.abs() + u.abs() * ca)
    if dres is not None:
        dx, dxa = dx + dres.double(), dxa + dres.double().abs()
    flat = (dy * u).flatten(0, -2)
    return dx, dxa, flat.sum(0), flat.abs().sum(0)


# ---- 8 bits ----------------------------------------------------------------

def q8_ref(v, quant, group):
    """codes (as numbers) and fp32 scales of an fp32 matrix, by the format's rule."""
    rows, cols = v.shape
    n = -(-cols // group)
    p = torch.zeros(rows, n * group, device=v.device)
    p[:, :cols] = v
    p = p.view(rows, n, group)
    amax = p.abs().amax(2)
    scale = amax * (1.0 / TOP[quant])
    bad = ~torch.isfinite(p).all(2)
    zero = scale < torch.finfo(torch.float32).tiny
    codes = p * scale.reciprocal()[..., None]
    if quant == "int8":
        codes = codes.round().clamp(-127, 127)
    else:
        codes = codes.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    codes = torch.where((bad | zero)[..., None], torch.zeros_like(codes), codes)
    scale = torch.where(bad, torch.full_like(scale, float("nan")), torch.where(zero, torch.zeros_like(scale), scale))
    return codes.reshape(rows, -1)[:, :cols], scale


def decoded(c):
    """The values of a checkpoint in 64 bits."""
    cols = c.codes.shape[-1]
    s = c.scales.double().repeat_interleave(c.group, -1)[..., :cols]
    return c.codes.float().double() * s


def act_ref(x, act, alpha=0.01):
    import math
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "leaky_relu":
        return torch.where(x >= 0, x, alpha * x)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.erfc(-x / math.sqrt(2.0))
    if act == "tanh":
        return torch.tanh(x)
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    return x


# ---- linear attention ------------------------------------------------------

def scan_ref(z, x, y, m, decay, lengths, mscale, oscale, reverse):
    """out_t = oscale * M_t^T z_t, M_t = decay M + mscale x_t y_t^T token by
    token in 64 bits; inputs [B, T, H, D].  Returns out and the last M."""
    B, T, H, Da = x.shape
    Db = y.shape[3]
    out = torch.zeros(B, T, H, Db, dtype=torch.float64, device=x.device)
    m = torch.zeros(B, H, Da, Db, dtype=torch.float64, device=x.device) if m is None else m.double().clone()
    dec = decay.double().view(1, H, 1, 1)
    n = torch.full((B,), T, device=x.device) if lengths is None else lengths.long().clamp(0, T)
    z, x, y = z.double(), x.double(), y.double()
    for t in (range(T - 1, -1, -1) if reverse else range(T)):
        on = (t < n).view(B, 1, 1, 1)
        first = (t == n - 1).view(B, 1, 1, 1) if reverse else torch.zeros_like(on)
        g = torch.where(first, torch.ones_like(dec), dec)
        new = g * m + mscale * x[:, t, :, :, None] * y[:, t, :, None, :]
        m = torch.where(on, new, m)
        out[:, t] = torch.where(on[..., 0], (z[:, t, :, None, :] @ m).squeeze(2) * oscale, torch.zeros_like(out[:, t]))
    if reverse:
        m = torch.where((n > 0).view(B, 1, 1, 1), dec * m, m)
    return out, m


# Extra error of the kernels that multiply 16-bit operands on the tensor
# cores: matrices that are not 16-bit numbers themselves (masked scores, the
# state, decayed inputs) enter as a sum of two 16-bit numbers, which leaves
# U^2 of each value; three such operands, and the tensor core's own fp32
# sums (chunks of at most 128 terms, 2^-18 of the terms' magnitudes).
SPLIT = {"f32": 0.0, "f16": 2.0 ** -17, "bf16": 2.0 ** -14}


def attention_k(T, Da, dtype):
    # one rounding per product and sum of a dot of Da, two for each token that
    # has passed through the state
    return (Da + 2 * T + 32) * E + SPLIT[dtype]


def check_core(dtype, got, got_m, z, x, y, m, log_decay, lengths, mscale, oscale, reverse, what):
    decay = torch.exp(log_decay.double())
    T, Da = x.shape[1], x.shape[3]
    k = attention_k(T, Da, dtype)
    ref, refm = scan_ref(z, x, y, m, decay, lengths, mscale, oscale, reverse)
    mag, magm = scan_ref(z.abs(), x.abs(), y.abs(), None if m is None else m.abs(), decay, lengths, abs(mscale), abs(oscale),
                         reverse)
    if got is not None:
        within(got, ref, ref.abs() * U[dtype] + mag * k + TINY[dtype], what)
    if got_m is not None:
        within(got_m, refm, magm * k, what + " state")


def valid(t, lengths):
    """t with what lies after each sequence's length set to zero."""
    if lengths is None:
        return t
    at = torch.arange(t.shape[1], device=t.device)[None, :, None, None]
    return torch.where(at < lengths.view(-1, 1, 1, 1), t, torch.zeros_like(t))


def check_attention(dtype, q, k, v, ld, state, lengths, scale, o, last):
    q, k, v = (valid(t, lengths) for t in (q, k, v))
    check_core(dtype, o, last, q, k, v, state, ld, lengths, 1.0, scale, False, "o")


def check_attention_back(dtype, q, k, v, ld, do, state, dstate, lengths, scale, dq, dk, dv, dfirst):
    q, k, v, do = (valid(t, lengths) for t in (q, k, v, do))
    st = None if state is None else state.transpose(2, 3)
    dt = None if dstate is None else dstate.transpose(2, 3)
    if dq is not None:
        check_core(dtype, dq, None, do, v, k, st, ld, lengths, 1.0, scale, False, "dq")
    if dk is not None:
        check_core(dtype, dk, None, v, do, q, dt, ld, lengths, scale, 1.0, True, "dk")
    if dv is not None or dfirst is not None:
        check_core(dtype, dv, dfirst, k, q, do, dstate, ld, lengths, scale, 1.0, True, "dv")


def need_gpu():
    import pytest
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transposed_convolution_convtranspose1_gb300 import _build
    _build.build_library()
    ct.lib()
