"""The operators of a decoder block around the transposed convolution, for measurement.

Three operators and their gradients: a root-mean-square norm with the residual's addition and an optional 8-bit output, a (gated)
activation that keeps its inputs as 8-bit checkpoints and differentiates from them, and causal linear attention with a decay for each
head.  `run` computes one pass, either in plain torch operations in 32 bits or (own = True) by the package's calls; `exact` gives the
same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
QUANTS = {"int8": (1.0 / 127.0, 127.0), "e4m3": (1.0 / 448.0, 448.0)}
EPS = 1e-6


def listed():
    return [
        # one step of eight streamed utterances: 512 channels, the residual added, 8-bit output read back by the next layer
        dict(name="norm_token", op="norm_fwd", rows=8, cols=512, dtype="bf16", residual=True, quant="int8", group=128),
        # a batch of 8 x 2048 positions at a wide model, activations handed on in 8 bits
        dict(name="norm_prompt", op="norm_fwd", rows=16384, cols=2048, dtype="bf16", residual=True, quant="e4m3", group=128),
        # an odd number of channels in full precision, no residual
        dict(name="norm_ragged", op="norm_fwd", rows=5003, cols=999, dtype="f32", residual=False, quant="none", group=64),
        # training: the gradient at the wide model, with the gradient that comes along the residual
        dict(name="norm_back", op="norm_bwd", rows=32768, cols=2048, dtype="bf16", residual=True),
        # training: gated activation between two projections, both inputs kept in 8 bits
        dict(name="gate_prompt", op="act_fwd", rows=16384, cols=4096, dtype="bf16", gated=True, packed=True, act="silu", quant="int8", group=128),
        # and its gradient from the 8-bit inputs
        dict(name="gate_back", op="act_bwd", rows=16384, cols=4096, dtype="bf16", gated=True, packed=True, act="silu", quant="int8", group=128),
        # the activation after an upsampling layer with an odd output width: 8 x 256 rows of 2049 positions
        dict(name="act_odd", op="act_fwd", rows=2048, cols=2049, dtype="f16", gated=False, packed=False, act="gelu", quant="e4m3", group=32),
        # one new token for 64 streams from their states
        dict(name="attn_token", op="attn_fwd", B=64, T=1, H=8, Dk=128, Dv=128, dtype="bf16", state=True, ragged=False, layout="bthd"),
        # prompts of a batch of 8, 2048 positions of 2048 channels
        dict(name="attn_prompt", op="attn_fwd", B=8, T=2048, H=16, Dk=128, Dv=128, dtype="bf16", state=False, ragged=False, layout="bthd"),
        # one long sequence on few heads
        dict(name="attn_long", op="attn_fwd", B=1, T=32768, H=8, Dk=64, Dv=64, dtype="f16", state=True, ragged=False, layout="bhtd"),
        # training at the vocoder's 8 x 2048 positions of 512 channels
        dict(name="attn_back", op="attn_bwd", B=8, T=2048, H=8, Dk=64, Dv=64, dtype="bf16", state=False, ragged=False, layout="bthd"),
        # a batch of unequal lengths (an empty one among them), odd head sizes, full precision
        dict(name="attn_ragged", op="attn_fwd", B=5, T=333, H=3, Dk=40, Dv=72, dtype="f32", state=True, ragged=True, layout="bthd"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "act_fwd", "act_bwd", "attn_fwd", "attn_fwd", "attn_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if not op.startswith("attn"):
        cols = _log_int(rng, 64, 8192)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        rows = _log_int(rng, 1, max(2, 33_000_000 // cols))
        if op == "norm_fwd":
            return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7,
                        quant=rng.choice(["none", "int8", "e4m3"]), group=rng.choice([32, 64, 128]))
        if op == "norm_bwd":
            return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7)
        gated = rng.random() < 0.6
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, gated=gated, packed=gated and rng.random() < 0.5,
                    act=rng.choice(["silu", "silu", "gelu", "tanh", "relu"]), quant=rng.choice(["int8", "e4m3"]), group=rng.choice([32, 64, 128]))
    size = rng.choice([64, 64, 128, 128, 8 * rng.randint(2, 16), rng.randint(16, 128)])
    other = size if rng.random() < 0.6 else 8 * rng.randint(2, 16)
    H = rng.randint(1, 16)
    B = _log_int(rng, 1, 16)
    T = _log_int(rng, 1, max(2, min(32768, (1_500_000 if dtype == "f32" else 16_000_000) // (B * H * max(size, other)))))
    return dict(op=op, B=B, T=T, H=H, Dk=size, Dv=other, dtype=dtype, state=rng.random() < 0.5, ragged=B > 1 and rng.random() < 0.4,
                layout=rng.choice(["bthd", "bhtd"]))


def lengths_of(case):
    """Tokens of each sequence: all of them, or spread from none to all."""
    B, T = case["B"], case["T"]
    return [T * b // (B - 1) for b in range(B)] if case["ragged"] else [T] * B


def work(case):
    if case["op"].startswith("attn"):
        e, H, Dk, Dv = DTYPES[case["dtype"]].itemsize, case["H"], case["Dk"], case["Dv"]
        n, every = sum(lengths_of(case)) * H, case["B"] * case["T"] * H
        states = 4 * case["B"] * H * Dk * Dv
        if case["op"] == "attn_fwd":
            return {"bytes": n * e * (2 * Dk + Dv) + every * e * Dv + states * (2 if case["state"] else 1), "flops": 4 * n * Dk * Dv}
        return {"bytes": n * e * 2 * (Dk + Dv) + every * e * (2 * Dk + Dv) + (3 * states if case["state"] else 0), "flops": 10 * n * Dk * Dv}
    n, e, rows, cols = case["rows"] * case["cols"], DTYPES[case["dtype"]].itemsize, case["rows"], case["cols"]
    if case["op"] == "norm_fwd":
        r = case["residual"]
        b = n * e * (3 if r else 1) + 4 * rows + cols * e
        if case["quant"] == "none":
            return {"bytes": b + n * e, "flops": 6 * n}
        scales = 4 * rows * -(-cols // case["group"])
        if case["quant"] == "int8":  # written, read back
            return {"bytes": b + 2 * (n + scales) + n * e, "flops": 10 * n}
        return {"bytes": b + n + scales, "flops": 8 * n}
    if case["op"] == "norm_bwd":
        return {"bytes": n * e * (4 if case["residual"] else 3) + 4 * rows + 2 * cols * e, "flops": 10 * n}
    scales = 4 * rows * -(-cols // case["group"])
    k = 2 if case["gated"] else 1
    return {"bytes": k * (n * e + n + scales) + n * e, "flops": (10 + 5 * k) * n}


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)

    s = {"case": case}
    if case["op"].startswith("attn"):
        B, T, H, Dk, Dv = (case[k] for k in ("B", "T", "H", "Dk", "Dv"))

        def heads(D):
            t = normal(B, H, T, D).to(dt) if case["layout"] == "bhtd" else normal(B, T, H, D).to(dt)
            return t.transpose(1, 2) if case["layout"] == "bhtd" else t

        s["q"], s["k"], s["v"] = heads(Dk), heads(Dk), heads(Dv)
        # a geometric ladder of memory lengths over the heads, from a few tokens to a few hundred
        s["log_decay"] = -torch.exp2(-1.0 - 7.0 * torch.arange(H, device="cuda", dtype=torch.float32) / max(1, H - 1))
        s["state"] = normal(B, H, Dk, Dv, std=2.0) if case["state"] else None
        s["lengths"] = torch.tensor(lengths_of(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        s["scale"] = Dk ** -0.5
        if case["op"] == "attn_bwd":
            s["do"] = heads(Dv)
            s["dstate"] = normal(B, H, Dk, Dv, std=0.1) if case["state"] else None
        return s
    rows, cols = case["rows"], case["cols"]
    if case["op"].startswith("norm"):
        s["weight"] = (1.0 + normal(cols, std=0.1)).to(dt)
        wide = 1.0 + 20.0 * (torch.rand(cols, generator=g, device="cuda") < 0.004)  # a few channels are far larger than the others
        if case["op"] == "norm_fwd":
            s["x"] = normal(rows, cols).to(dt)
            s["residual"] = (normal(rows, cols) * wide).to(dt) if case["residual"] else None
        else:
            s["h"] = (normal(rows, cols) * wide).to(dt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
            s["dy"] = normal(rows, cols, std=0.01).to(dt)
            s["dresidual"] = normal(rows, cols, std=0.01).to(dt) if case["residual"] else None
        return s
    groups = -(-cols // case["group"])

    def inputs():
        if not case["gated"]:
            return [normal(rows, cols, std=1.5).to(dt)]
        if case["packed"]:  # the two halves of one projection's output
            both = normal(rows, 2 * cols, std=1.5).to(dt)
            return [both[:, :cols], both[:, cols:]]
        return [normal(rows, cols, std=1.5).to(dt) for _ in range(2)]

    if case["op"] == "act_fwd":
        s["inputs"] = inputs()
        return s
    s["dy"] = normal(rows, cols, std=0.01).to(dt)
    s["kept"] = []
    for _ in range(2 if case["gated"] else 1):
        top = QUANTS[case["quant"]][1]
        codes = normal(rows, cols, std=top / 3).clamp_(-top, top)
        codes = codes.round_().to(torch.int8) if case["quant"] == "int8" else codes.to(torch.float8_e4m3fn)
        s["kept"].append((codes, (torch.rand(rows, groups, generator=g, device="cuda") * 2 + 3) / top))
    return s


# ---- plain forms -------------------------------------------------------------------------------------------------------------------

def _grouped(v, group):
    rows, cols = v.shape
    n = -(-cols // group)
    out = v.new_zeros(rows, n * group)
    out[:, :cols] = v
    return out.view(rows, n, group)


def _to_8_bits(v, quant, group):
    """Codes and scales of an fp32 matrix: a scale for each `group` consecutive values of a row."""
    rows, cols = v.shape
    inverse, top = QUANTS[quant]
    v = _grouped(v, group)
    scales = v.abs().amax(2) * inverse
    codes = v * scales.reciprocal().unsqueeze(2)
    codes = codes.round().clamp(-top, top).to(torch.int8) if quant == "int8" else codes.clamp(-top, top).to(torch.float8_e4m3fn)
    return codes.view(rows, -1)[:, :cols].contiguous(), scales


def _from_8_bits(codes, scales, group):
    rows, cols = codes.shape
    return (_grouped(codes.float(), group) * scales.unsqueeze(2)).view(rows, -1)[:, :cols]


def _norm_forward(s):
    c = s["case"]
    total = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    rstd = torch.rsqrt(total.square().mean(1, keepdim=True) + EPS)
    y = total * rstd * s["weight"].float()
    out = {"rstd": rstd.squeeze(1)}
    if s["residual"] is not None:
        out["h"] = total.to(s["x"].dtype)
    if c["quant"] == "none":
        out["y"] = y.to(s["x"].dtype)
    else:
        codes, scales = _to_8_bits(y, c["quant"], c["group"])
        if c["quant"] == "int8":
            out["y"] = _from_8_bits(codes, scales, c["group"]).to(s["x"].dtype)
        else:
            out["codes"], out["scales"] = codes, scales
    return out


def _norm_backward(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
    unit = h * rstd
    wdy = dy * s["weight"].float()
    dx = rstd * (wdy - unit * (wdy * unit).mean(1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * unit).sum(0).to(s["h"].dtype)}


def _act(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return torch.tanh(x) if act == "tanh" else torch.clamp(x, min=0.0)


def _act_slope(x, act):
    if act == "silu":
        g = torch.sigmoid(x)
        return g * (1.0 + x * (1.0 - g))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    return 1.0 - torch.tanh(x).square() if act == "tanh" else (x > 0).float()


def _act_forward(s):
    c = s["case"]
    wide = [t.float() for t in s["inputs"]]
    y = _act(wide[0], c["act"])
    if c["gated"]:
        y = y * wide[1]
    return {"y": y.to(s["inputs"][0].dtype), "kept": [_to_8_bits(t, c["quant"], c["group"]) for t in wide]}


def _act_backward(s):
    c = s["case"]
    wide = [_from_8_bits(codes, scales, c["group"]) for codes, scales in s["kept"]]
    dy = s["dy"].float()
    slope = dy * _act_slope(wide[0], c["act"])
    if not c["gated"]:
        return [slope.to(s["dy"].dtype)]
    return [(slope * wide[1]).to(s["dy"].dtype), (dy * _act(wide[0], c["act"])).to(s["dy"].dtype)]


CHUNK = 64


def _decayed(z, x, y, log_decay):
    """out_t = sum over s <= t of decay^(t-s) (z_t . x_s) y_s for [B, H, T, D] inputs, in chunks: within a chunk by the masked product,
    across chunks by the chunks' own states and the decays between them."""
    B, H, T, Da = x.shape
    n = -(-T // CHUNK)

    def cut(t):
        out = t.new_zeros(B, H, n * CHUNK, t.shape[3])
        out[:, :, :T] = t
        return out.view(B, H, n, CHUNK, t.shape[3])

    z, x, y = cut(z), cut(x), cut(y)
    g = log_decay.view(H, 1, 1)
    i = torch.arange(CHUNK, device=x.device)
    gap = i[:, None] - i[None, :]
    mask = torch.where(gap >= 0, torch.exp(g * gap.clamp(min=0)), 0.0)
    out = (z @ x.transpose(3, 4) * mask[None, :, None]) @ y
    if n > 1:
        tail = torch.exp(log_decay[:, None] * (CHUNK - 1 - i))[None, :, None, :, None]
        local = ((x * tail).transpose(3, 4) @ y).view(B, H, n, -1)
        c = torch.arange(n, device=x.device)
        between = c[:, None] - 1 - c[None, :]
        start = torch.where(between >= 0, torch.exp(g * CHUNK * between.clamp(min=0)), 0.0) @ local
        out = out + (z * torch.exp(log_decay[:, None] * (i + 1))[None, :, None, :, None]) @ start.view(B, H, n, Da, -1)
    return out.view(B, H, n * CHUNK, -1)[:, :, :T]


def _attention_inputs(s):
    """fp32 [B, H, T, D] inputs with what lies past a sequence's length set to zero, the token's place and the lengths."""
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    lengths = s["lengths"] if s["lengths"] is not None else torch.full((c["B"],), c["T"], dtype=torch.int32, device="cuda")
    valid = (t[None] < lengths[:, None])[:, None, :, None]
    wide = [torch.where(valid, s[name].transpose(1, 2).float(), 0.0) for name in ("q", "k", "v", "do") if name in s]
    wide[0] = wide[0] * s["scale"]
    n = lengths[:, None, None]
    return wide, t, n, valid


def _attention_forward(s):
    (q, k, v), t, n, _ = _attention_inputs(s)
    g = s["log_decay"][:, None]
    out = _decayed(q, k, v, s["log_decay"])
    left = torch.exp(g * (n - 1 - t).clamp(min=0))  # past the length there are zeros
    state = (k * left.unsqueeze(3)).transpose(2, 3) @ v
    if s["state"] is not None:
        out = out + (q * torch.exp(g * (t + 1))[None, :, :, None]) @ s["state"]
        state = state + torch.exp(g[None] * n).view(-1, g.shape[0], 1, 1) * s["state"]
    return {"o": out.transpose(1, 2).contiguous().to(s["q"].dtype), "state": state}


def _attention_backward(s):
    (qs, k, v, do), t, n, valid = _attention_inputs(s)
    ld, dt = s["log_decay"], s["q"].dtype
    g = ld[:, None]
    dq = _decayed(do, v, k, ld)
    dv = _decayed(k.flip(2), qs.flip(2), do.flip(2), ld).flip(2)
    dk = _decayed(v.flip(2), do.flip(2), qs.flip(2), ld).flip(2)
    into = torch.exp(g * (t + 1))[None, :, :, None]
    dstate = (qs * into).transpose(2, 3) @ do
    if s["state"] is not None:
        dq = dq + (do * into) @ s["state"].transpose(2, 3)
        left = torch.where(valid, torch.exp(g * (n - 1 - t).clamp(min=0)).unsqueeze(3), 0.0)
        dk = dk + (v * left) @ s["dstate"].transpose(2, 3)
        dv = dv + (k * left) @ s["dstate"]
        dstate = dstate + torch.exp(g[None] * n).view(-1, g.shape[0], 1, 1) * s["dstate"]
    out = {"dq": dq * s["scale"], "dk": dk, "dv": dv}
    out = {name: u.transpose(1, 2).contiguous().to(dt) for name, u in out.items()}
    if s["state"] is not None:
        out["dstate"] = dstate
    return out


PLAIN = {"norm_fwd": _norm_forward, "norm_bwd": _norm_backward, "act_fwd": _act_forward, "act_bwd": _act_backward,
         "attn_fwd": _attention_forward, "attn_bwd": _attention_backward}


# ---- the package's calls -----------------------------------------------------------------------------------------------------------

def _own(s):
    import transposed_convolution_convtranspose1_gb300 as ct
    c = s["case"]
    if c["op"] == "norm_fwd":
        quant = None if c["quant"] == "none" else c["quant"]
        y, h, rstd, kept = ct.rms_norm(s["x"], s["weight"], s["residual"], eps=EPS, quant=quant, group=c["group"],
                                       need=("y", "rstd") if quant is None else ("rstd",))
        out = {"rstd": rstd}
        if s["residual"] is not None:
            out["h"] = h
        if c["quant"] == "none":
            out["y"] = y
        elif c["quant"] == "int8":
            out["y"] = ct.checkpoint_load(kept)
        else:
            out["codes"], out["scales"] = kept.codes, kept.scales
        return out
    if c["op"] == "norm_bwd":
        dx, dw = ct.rms_norm_backward(s["dy"], s["h"], s["rstd"], s["weight"], s["dresidual"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "act_fwd":
        up = s["inputs"][1] if c["gated"] else None
        y, *kept = ct.checkpointed_activation(s["inputs"][0], up, activation=c["act"], quant=c["quant"], group=c["group"])
        return {"y": y, "kept": [(k.codes, k.scales) for k in kept if k is not None]}
    if c["op"] == "act_bwd":
        kept = [ct.Checkpoint(codes, scales, c["group"], s["dy"].dtype) for codes, scales in s["kept"]]
        grads = ct.checkpointed_activation_backward(s["dy"], kept[0], kept[1] if c["gated"] else None, activation=c["act"])
        return [t for t in grads if t is not None]
    if c["op"] == "attn_fwd":
        o, state = ct.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], state=s["state"], lengths=s["lengths"], scale=s["scale"])
        return {"o": o, "state": state}
    dq, dk, dv, dstate = ct.linear_attention_backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"], state=s["state"], dstate=s["dstate"],
                                                      lengths=s["lengths"], scale=s["scale"])
    out = {"dq": dq, "dk": dk, "dv": dv}
    if s["state"] is not None:
        out["dstate"] = dstate
    return out


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------------------------

def _exact_8_bits(v, quant, group):
    """(values, scales): what each group's codes stand for, by loops over the groups."""
    inverse, top = QUANTS[quant]
    values, scales = [], []
    for part in v.split(group, dim=1):
        scale = part.abs().max(1, keepdim=True).values / top
        code = part / scale
        code = torch.round(code) if quant == "int8" else code.float().to(torch.float8_e4m3fn).double()
        values.append(code)
        scales.append(scale)
    return torch.cat(values, 1), torch.cat(scales, 1)


def _exact_act(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.erfc(-x / math.sqrt(2.0))
    return 1.0 - 2.0 / (torch.exp(2.0 * x) + 1.0) if act == "tanh" else torch.where(x > 0, x, 0.0)


def _exact_scan(z, x, y, m, decay, lengths, order):
    """out_t = m_t^T z_t with m_t = decay m + x_t y_t^T, token by token in `order`; the last m."""
    out = torch.zeros(z.shape[0], z.shape[1], z.shape[2], y.shape[3], dtype=torch.float64, device="cuda")
    for t in order:
        new = decay * m + x[:, :, t, :, None] * y[:, :, t, None, :]
        here = (lengths > t).view(-1, 1, 1, 1)
        m = torch.where(here, new, m)
        out[:, :, t] = torch.where(here.squeeze(3), (z[:, :, t, None, :] @ m).squeeze(2), 0.0)
    return out, m


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op == "norm_fwd":
        total = d["x"] + d["residual"] if case["residual"] else d["x"]
        rstd = 1.0 / torch.sqrt((total * total).sum(1) / case["cols"] + EPS)
        y = total * rstd[:, None] * d["weight"]
        out = {"rstd": rstd}
        if case["residual"]:
            out["h"] = total
        if case["quant"] == "none":
            out["y"] = y
        else:
            codes, scales = _exact_8_bits(y, case["quant"], case["group"])
            if case["quant"] == "int8":
                out["y"] = codes * scales.repeat_interleave(case["group"], 1)[:, :case["cols"]]
            else:
                out["codes"], out["scales"] = codes, scales
        return out
    if op == "norm_bwd":
        # y_i = w_i h_i r with r = (mean h^2 + eps)^(-1/2): dy_i/dh_j = w_i r (i = j) - w_i h_i h_j r^3 / n
        r, n = d["rstd"][:, None], case["cols"]
        a = (d["weight"] * d["dy"] * d["h"]).sum(1, keepdim=True)
        dx = d["weight"] * d["dy"] * r - d["h"] * r ** 3 * a / n
        return {"dx": dx + d["dresidual"] if case["residual"] else dx, "dw": (d["dy"] * d["h"] * r).sum(0)}
    if op == "act_fwd":
        x = [t.double() for t in s["inputs"]]
        y = _exact_act(x[0], case["act"]) * (x[1] if case["gated"] else 1.0)
        kept = []
        for t in x:
            codes, scales = _exact_8_bits(t, case["quant"], case["group"])
            kept.append((None if case["quant"] == "int8" else codes, scales))
        return {"y": y, "kept": kept}
    if op == "act_bwd":
        x = [codes.double() * scales.double().repeat_interleave(case["group"], 1)[:, :case["cols"]] for codes, scales in s["kept"]]
        one = x[0].clone().requires_grad_()
        y = _exact_act(one, case["act"])
        da = torch.autograd.grad(y, one, d["dy"] * (x[1] if case["gated"] else 1.0))[0]
        return [da, d["dy"] * y.detach()] if case["gated"] else [da]
    if case["T"] * case["B"] * case["H"] * case["Dk"] * case["Dv"] > 6e9:
        return None
    B, T, H, Dk, Dv = (case[k] for k in ("B", "T", "H", "Dk", "Dv"))
    q, k, v = (d[name].transpose(1, 2) for name in ("q", "k", "v"))
    q = q * s["scale"]
    decay = torch.exp(d["log_decay"]).view(1, H, 1, 1)
    lengths = torch.tensor(lengths_of(case), device="cuda")
    zero = torch.zeros(B, H, Dk, Dv, dtype=torch.float64, device="cuda")
    first = d["state"] if case["state"] else zero
    if op == "attn_fwd":
        o, last = _exact_scan(q, k, v, first, decay, lengths, range(T))
        return {"o": o.transpose(1, 2), "state": last}
    do = d["do"].transpose(1, 2)
    end = d["dstate"] if case["state"] else zero
    dq, _ = _exact_scan(do, v, k, first.transpose(2, 3), decay, lengths, range(T))
    # backwards in time the gradient of the last state enters undecayed; 1/decay makes up for the scan's first step
    dv, dfirst = _exact_scan(k, q, do, end / decay, decay, lengths, range(T - 1, -1, -1))
    dk, _ = _exact_scan(v, do, q, (end / decay).transpose(2, 3), decay, lengths, range(T - 1, -1, -1))
    out = {"dq": dq.transpose(1, 2) * s["scale"], "dk": dk.transpose(1, 2), "dv": dv.transpose(1, 2)}
    if case["state"]:
        out["dstate"] = dfirst * decay
    return out
