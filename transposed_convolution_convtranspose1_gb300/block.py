"""Binding of the layers around a transposed convolution in a decoder block:
RMS norm, 8-bit activation checkpoints with the (gated) activation that uses
them, and linear attention with a decay for each head (include/ct.h).

Argument marshalling only, as in ct.py: every step of the computation runs in
libct.so on the current stream of the tensors' device.  A call given `stream`
runs as if that were the current one, outputs included: as after any work on a
side stream, the caller orders the streams around it.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from .ct import (ACTIVATIONS, CT_ERR_DTYPE, CT_ERR_PARAM, CT_ERR_SHAPE, CtError, _check, _stream_handle,
                 dtype_code, lib)

CT_Q_NONE, CT_Q_INT8, CT_Q_E4M3 = 0, 1, 2
QUANTS = {None: CT_Q_NONE, "none": CT_Q_NONE, "int8": CT_Q_INT8, "e4m3": CT_Q_E4M3}
_CODE_DTYPE = {CT_Q_INT8: torch.int8, CT_Q_E4M3: torch.float8_e4m3fn}
_QUANT_OF = {torch.int8: CT_Q_INT8, torch.float8_e4m3fn: CT_Q_E4M3}


class Checkpoint(NamedTuple):
    """A tensor kept in 8 bits: codes (int8 or float8_e4m3fn, the tensor's
    shape), one fp32 scale for each `group` consecutive values of the last
    axis, and the dtype it is read back in."""
    codes: torch.Tensor
    scales: torch.Tensor
    group: int
    dtype: torch.dtype


# What follows runs on the host for every call, on tensors of any size: small
# calls take as long as it does, so it stays short.

def _index_of(first, *others) -> int:
    """The index of the one CUDA device of all given tensors (None skipped)."""
    index = first.get_device()
    if index < 0:
        raise CtError(CT_ERR_PARAM, f"device tensors expected, got {first.device}")
    for t in others:
        if t is not None and t.get_device() != index:
            raise CtError(CT_ERR_PARAM, f"tensors must share one device, got {first.device} and {t.device}")
    return index


# The current stream's handle without building a Stream object (6 us a call on
# the GPU's host, a quarter of a small call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _call(fn, index, *args):
    """fn(*args, stream) on the current stream of the tensors' device, which is made current."""
    s = _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream
    if index == (_get_device() if _get_device is not None else torch.cuda.current_device()):
        rc = fn(*args, s)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, s)
    if rc:
        _check(rc)


def _on(stream, first):
    """`stream` (a torch stream or a raw handle) as the current one.  A call's
    outputs and workspace come from the allocator's pool of the current stream
    and are free for reuse in that stream's order: taken from another stream's
    pool, a workspace would be handed out again while kernels still use it."""
    index = _index_of(first)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_handle(stream, None)
        stream = torch.cuda.ExternalStream(handle, index) if handle else torch.cuda.default_stream(index)
    if stream.device.index != index:
        raise CtError(CT_ERR_PARAM, f"the stream is of {stream.device}, the tensors are on cuda:{index}")
    return torch.cuda.stream(stream)


def _rows(t: Optional[torch.Tensor], like: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None):
    """(pointer, row stride) of a tensor read as a matrix of its last axis."""
    if t is None:
        return None, 0
    shape = t.shape
    if like is not None and shape != like.shape:
        raise CtError(CT_ERR_SHAPE, f"expected shape {tuple(like.shape)}, got {tuple(shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise CtError(CT_ERR_DTYPE, f"expected {dtype}, got {t.dtype}")
    if shape and t.is_contiguous():
        return t.data_ptr(), shape[-1]
    strides = t.stride()
    if not shape:
        raise CtError(CT_ERR_SHAPE, "a tensor of at least one axis is expected")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError("the last axis must be dense")
    stride, below = shape[-1], None
    for n, st in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if below is None:
            stride = st
        elif st != below:
            raise ValueError("the leading axes must be evenly spaced rows")
        below = st * n
    return t.data_ptr(), stride


def _dense(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("this tensor must be contiguous")
    return t.data_ptr()  # 0, NULL, for a tensor without elements


def _extent(t: torch.Tensor):
    shape = t.shape
    if len(shape) == 2:
        return shape
    cols = shape[-1]
    return (t.numel() // cols if cols else 0), cols


def _like(t: torch.Tensor) -> torch.Tensor:
    """A new dense tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(t, memory_format=torch.contiguous_format)


def _groups(cols: int, group: int) -> int:
    return -(-cols // group) if group > 0 else 0


def _quant(quant) -> int:
    if quant not in QUANTS:
        raise CtError(CT_ERR_PARAM, f"quant must be None, 'int8' or 'e4m3', got {quant!r}")
    return QUANTS[quant]


def _checkpoint_quant(quant) -> int:
    q = _quant(quant)
    if q == CT_Q_NONE:
        raise CtError(CT_ERR_PARAM, "a checkpoint is 'int8' or 'e4m3'")
    return q


def _activation(a) -> int:
    if isinstance(a, str):
        if a not in ACTIVATIONS:
            raise CtError(CT_ERR_PARAM, f"activation {a!r} is not one of {sorted(ACTIVATIONS)}")
        return ACTIVATIONS[a]
    return int(a)


def _new_checkpoint(x, quant, group) -> Checkpoint:
    shape = x.shape
    codes = torch.empty(shape, dtype=_CODE_DTYPE[quant], device=x.device)
    n = _groups(shape[-1], group)
    scales = torch.empty((shape[0], n) if len(shape) == 2 else (*shape[:-1], n), dtype=torch.float32, device=x.device)
    return Checkpoint(codes, scales, group, x.dtype)


def _kept(c: Optional[Checkpoint], like: Optional[torch.Tensor] = None):
    """(codes pointer, scales pointer) of a checkpoint, checked."""
    if c is None:
        return None, None
    if c.codes.dtype not in _QUANT_OF or c.scales.dtype != torch.float32:
        raise CtError(CT_ERR_DTYPE, "a checkpoint has int8 or float8_e4m3fn codes and float32 scales")
    if like is not None and c.codes.shape != like.shape:
        raise CtError(CT_ERR_SHAPE, f"expected codes of shape {tuple(like.shape)}, got {tuple(c.codes.shape)}")
    shape = c.codes.shape
    if c.scales.shape != (*shape[:-1], _groups(shape[-1], c.group)):
        raise CtError(CT_ERR_SHAPE, f"{tuple(c.scales.shape)} scales do not fit codes of shape {tuple(c.codes.shape)} "
                                    f"in groups of {c.group}")
    return _dense(c.codes), _dense(c.scales)


# ---- norm ------------------------------------------------------------------

def _check_weight(weight, x):
    if weight is None:
        return
    if weight.shape != x.shape[-1:]:
        raise CtError(CT_ERR_SHAPE, f"weight must be [{x.size(-1)}], got {tuple(weight.shape)}")
    if weight.dtype is not x.dtype:
        raise CtError(CT_ERR_DTYPE, f"weight must be {x.dtype}, got {weight.dtype}")


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6, quant: Optional[str] = None, group: int = 128, need=("y", "rstd"), stream=None):
    """Root-mean-square norm over the last axis, the residual added first.

    Returns (y, h, rstd, checkpoint): y the normalised tensor, h = x + residual
    (x itself without a residual), rstd fp32 of the leading shape, checkpoint y
    in 8 bits where `quant` is "int8" or "e4m3".  y and rstd are None unless
    named in `need`.
    """
    if stream is not None:
        with _on(stream, x):
            return rms_norm(x, weight, residual, eps, quant, group, need)
    q = _quant(quant)
    px, sx = _rows(x)
    pr, sr = _rows(residual, x, x.dtype)
    _check_weight(weight, x)
    index = _index_of(x, residual, weight)
    rows, cols = _extent(x)
    y = _like(x) if "y" in need else None
    h = _like(x) if residual is not None else None
    rstd = torch.empty(rows if x.dim() == 2 else x.shape[:-1], dtype=torch.float32, device=x.device) if "rstd" in need else None
    kept = _new_checkpoint(x, q, group) if q != CT_Q_NONE else None
    _call(lib().ct_rms_norm_forward, index, px, sx, pr, sr, _dense(weight), y.data_ptr() if y is not None else None, cols,
          h.data_ptr() if h is not None else None, cols, rstd.data_ptr() if rstd is not None else None,
          kept.codes.data_ptr() if kept is not None else None, kept.scales.data_ptr() if kept is not None else None, rows, cols,
          eps, dtype_code(x.dtype), q, group)
    return y, x if residual is None else h, rstd, kept


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                      dresidual: Optional[torch.Tensor] = None, need=("dx", "dw"), stream=None):
    """(dx, dw) of rms_norm from its h and rstd; dresidual is the gradient that
    arrives along h and is added to dx.  Entries not in `need` are None, and dw
    where there is no weight."""
    if stream is not None:
        with _on(stream, h):
            return rms_norm_backward(dy, h, rstd, weight, dresidual, need)
    pd, sd = _rows(dy, h, h.dtype)
    ph, sh = _rows(h)
    pr, sr = _rows(dresidual, h, h.dtype)
    if rstd.shape != h.shape[:-1] or rstd.dtype != torch.float32:
        raise CtError(CT_ERR_SHAPE, f"rstd must be float32 {tuple(h.shape[:-1])}")
    _check_weight(weight, h)
    index = _index_of(h, dy, rstd, weight, dresidual)
    rows, cols = _extent(h)
    code = dtype_code(h.dtype)
    dx = _like(h) if "dx" in need else None
    dw = ws = None
    nws = 0
    if "dw" in need and weight is not None:
        dw = torch.empty((cols,), dtype=h.dtype, device=h.device)
        n = ctypes.c_size_t(0)
        _check(lib().ct_rms_norm_backward_workspace_bytes(rows, cols, code, ctypes.byref(n)))
        nws = n.value
        ws = torch.empty((nws,), dtype=torch.uint8, device=h.device)
    _call(lib().ct_rms_norm_backward, index, pd, sd, ph, sh, _dense(rstd), _dense(weight), pr, sr, _dense(dx),
          cols, _dense(dw), _dense(ws), nws, rows, cols, code)
    return dx, dw


class RmsNormFunction(torch.autograd.Function):
    """torch.autograd binding of rms_norm."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd, _ = rms_norm(x, weight, residual, eps)
        ctx.save_for_backward(h, rstd, weight)
        ctx.has_residual = residual is not None
        return (y, h) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, rstd, weight = ctx.saved_tensors
        need = tuple(n for n, flag in (("dx", ctx.needs_input_grad[0] or ctx.needs_input_grad[2]),
                                       ("dw", ctx.needs_input_grad[1])) if flag)
        dx, dw = rms_norm_backward(dy.contiguous(), h, rstd, weight, None if dh is None else dh.contiguous(), need)
        return dx, dw, dx if ctx.has_residual else None, None


def rms_norm_autograd(x, weight=None, residual=None, eps: float = 1e-6):
    """rms_norm that records itself for torch.autograd: y, or (y, h) with a residual."""
    return RmsNormFunction.apply(x, weight, residual, eps)


# ---- 8-bit checkpoints -----------------------------------------------------

def checkpoint_store(x: torch.Tensor, quant: str = "int8", group: int = 128, stream=None) -> Checkpoint:
    """x kept in 8 bits, one scale for each `group` values of the last axis."""
    if stream is not None:
        with _on(stream, x):
            return checkpoint_store(x, quant, group)
    q = _checkpoint_quant(quant)
    px, sx = _rows(x)
    index = _index_of(x)
    rows, cols = _extent(x)
    c = _new_checkpoint(x, q, group)
    _call(lib().ct_checkpoint_store, index, px, sx, _dense(c.codes), _dense(c.scales), rows, cols,
          dtype_code(x.dtype), q, group)
    return c


def checkpoint_load(c: Checkpoint, dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """The values a checkpoint stands for, in its own dtype or another."""
    if stream is not None:
        with _on(stream, c.codes):
            return checkpoint_load(c, dtype)
    pc, ps = _kept(c)
    index = _index_of(c.codes, c.scales)
    rows, cols = _extent(c.codes)
    y = torch.empty_like(c.codes, dtype=dtype or c.dtype)
    _call(lib().ct_checkpoint_load, index, pc, ps, y.data_ptr(), cols, rows, cols, dtype_code(y.dtype),
          _QUANT_OF[c.codes.dtype], c.group)
    return y


def checkpointed_activation(gate: torch.Tensor, up: Optional[torch.Tensor] = None, activation="silu",
                            alpha: float = 0.01, quant: str = "int8", group: int = 128, stream=None):
    """(y, gate checkpoint, up checkpoint): y = act(gate) * up, or act(gate)
    without `up` (whose checkpoint is then None)."""
    if stream is not None:
        with _on(stream, gate):
            return checkpointed_activation(gate, up, activation, alpha, quant, group)
    q, act = _checkpoint_quant(quant), _activation(activation)
    pg, sg = _rows(gate)
    pu, su = _rows(up, gate, gate.dtype)
    index = _index_of(gate, up)
    rows, cols = _extent(gate)
    y = _like(gate)
    cg = _new_checkpoint(gate, q, group)
    cu = _new_checkpoint(up, q, group) if up is not None else None
    _call(lib().ct_checkpointed_activation_forward, index, pg, sg, pu, su, y.data_ptr(), cols, cg.codes.data_ptr(),
          cg.scales.data_ptr(), cu.codes.data_ptr() if cu else None, cu.scales.data_ptr() if cu else None, rows, cols, act, alpha,
          dtype_code(gate.dtype), q, group)
    return y, cg, cu


def checkpointed_activation_backward(dy: Optional[torch.Tensor], gate: Checkpoint, up: Optional[Checkpoint] = None,
                                     activation="silu", alpha: float = 0.01, need=("dgate", "dup"), stream=None):
    """(dgate, dup) from the checkpoints; with "y" in `need`, (dgate, dup, y),
    y recomputed from them (a following layer's weight gradient reads it).
    Entries not in `need` are None, and dup without `up`."""
    if stream is not None:
        with _on(stream, gate.codes):
            return checkpointed_activation_backward(dy, gate, up, activation, alpha, need)
    act = _activation(activation)
    pg, sg = _kept(gate)
    pu, su = _kept(up, gate.codes)
    if up is not None and (up.codes.dtype != gate.codes.dtype or up.group != gate.group):
        raise CtError(CT_ERR_PARAM, "gate and up must be kept in one format")
    dtype = dy.dtype if dy is not None else gate.dtype
    pd, sd = _rows(dy, gate.codes)
    index = _index_of(gate.codes, gate.scales, dy, *((up.codes, up.scales) if up is not None else ()))
    rows, cols = _extent(gate.codes)

    def new(name):
        return torch.empty_like(gate.codes, dtype=dtype) if name in need else None

    dgate, dup, y = new("dgate"), new("dup") if up is not None else None, new("y")
    _call(lib().ct_checkpointed_activation_backward, index, pd, sd, pg, sg, pu, su, _dense(dgate), cols,
          _dense(dup), cols, _dense(y), cols, rows, cols, act, alpha, dtype_code(dtype), _QUANT_OF[gate.codes.dtype],
          gate.group)
    return (dgate, dup, y) if "y" in need else (dgate, dup)


class CheckpointedActivationFunction(torch.autograd.Function):
    """torch.autograd binding: only the 8-bit checkpoints are kept."""

    @staticmethod
    def forward(ctx, gate, up, activation, alpha, quant, group):
        y, cg, cu = checkpointed_activation(gate, up, activation, alpha, quant, group)
        ctx.save_for_backward(cg.codes, cg.scales, *((cu.codes, cu.scales) if cu is not None else ()))
        ctx.args = (activation, alpha, group, gate.dtype)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        activation, alpha, group, dtype = ctx.args
        t = ctx.saved_tensors
        cg = Checkpoint(t[0], t[1], group, dtype)
        cu = Checkpoint(t[2], t[3], group, dtype) if len(t) > 2 else None
        need = tuple(n for n, flag in (("dgate", ctx.needs_input_grad[0]), ("dup", ctx.needs_input_grad[1])) if flag)
        dgate, dup = checkpointed_activation_backward(dy.contiguous(), cg, cu, activation, alpha, need)
        return dgate, dup, None, None, None, None


def checkpointed_activation_autograd(gate, up=None, activation="silu", alpha: float = 0.01, quant: str = "int8",
                                     group: int = 128):
    """checkpointed_activation that records itself for torch.autograd; returns y."""
    return CheckpointedActivationFunction.apply(gate, up, activation, alpha, quant, group)


# ---- linear attention ------------------------------------------------------

_I64x3 = ctypes.c_int64 * 3


def _heads(t: Optional[torch.Tensor], shape, dtype):
    """(pointer, strides of batch, token and head) of a [B, T, H, D] tensor."""
    if t is None:
        return None, None
    if t.shape != shape:
        raise CtError(CT_ERR_SHAPE, f"expected shape {shape}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise CtError(CT_ERR_DTYPE, f"expected {dtype}, got {t.dtype}")
    b, s, h, d = t.stride()
    if d != 1 and shape[3] > 1:
        raise ValueError("the last axis must be dense")
    return t.data_ptr(), _strides(b, s, h)


@functools.lru_cache(maxsize=256)
def _strides(b: int, t: int, h: int):
    return _I64x3(b, t, h)


def _attention_problem(q, v, log_decay, lengths, *states):
    if q.dim() != 4 or v.dim() != 4:
        raise CtError(CT_ERR_SHAPE, "q and k are [B, T, H, Dk], v is [B, T, H, Dv]")
    B, T, H, Dk = q.shape
    Dv = v.shape[3]
    if log_decay.shape != (H,) or log_decay.dtype != torch.float32:
        raise CtError(CT_ERR_SHAPE, f"log_decay must be float32 [{H}]")
    if lengths is not None and (lengths.shape != (B,) or lengths.dtype != torch.int32):
        raise CtError(CT_ERR_SHAPE, f"lengths must be int32 [{B}]")
    for s in states:
        if s is not None and (s.shape != (B, H, Dk, Dv) or s.dtype != torch.float32):
            raise CtError(CT_ERR_SHAPE, f"a state must be float32 [{B}, {H}, {Dk}, {Dv}]")
    return B, T, H, Dk, Dv


@functools.lru_cache(maxsize=256)
def _attention_workspace_bytes(B, T, H, Dk, Dv, code, backward, index):
    n = ctypes.c_size_t(0)
    with torch.cuda.device(index):
        _check(lib().ct_linear_attention_workspace_bytes(B, T, H, Dk, Dv, code, backward, ctypes.byref(n)))
    return n.value


def linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                     state: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                     scale: Optional[float] = None, state_out: Optional[torch.Tensor] = None, need=("state",),
                     stream=None):
    """Causal linear attention with a decay exp(log_decay[h]) for each head.

    q, k [B, T, H, Dk], v [B, T, H, Dv] (any strides, last axis dense),
    log_decay [H] float32, state [B, H, Dk, Dv] float32 before the first token,
    lengths [B] int32 tokens of each sequence, scale Dk**-0.5 unless given.
    Returns (o, state after the last token); the state is written to state_out
    where given (it may be `state` itself), and is None without "state" in
    `need`.  T = 1 is a streaming step.
    """
    if stream is not None:
        with _on(stream, q):
            return linear_attention(q, k, v, log_decay, state, lengths, scale, state_out, need)
    B, T, H, Dk, Dv = _attention_problem(q, v, log_decay, lengths, state, state_out)
    dt = q.dtype
    pq, sq = _heads(q, (B, T, H, Dk), dt)
    pk, sk = _heads(k, (B, T, H, Dk), dt)
    pv, sv = _heads(v, (B, T, H, Dv), dt)
    index = _index_of(q, k, v, log_decay, state, lengths, state_out)
    o = _like(v)
    if state_out is None and "state" in need:
        state_out = _like(state) if state is not None else torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device)
    code = dtype_code(dt)
    nws = _attention_workspace_bytes(B, T, H, Dk, Dv, code, 0, index)
    ws = torch.empty((nws,), dtype=torch.uint8, device=q.device) if nws else None
    _call(lib().ct_linear_attention_forward, index, pq, sq, pk, sk, pv, sv, o.data_ptr(),
          _strides(T * H * Dv, H * Dv, Dv), _dense(log_decay), _dense(state), _dense(state_out), _dense(lengths),
          _dense(ws), nws, B, T, H, Dk, Dv, Dk ** -0.5 if scale is None else scale, code)
    return o, state_out


def linear_attention_backward(q, k, v, log_decay, do, state=None, dstate=None, lengths=None,
                              scale: Optional[float] = None, need=("dq", "dk", "dv", "dstate"), stream=None):
    """(dq, dk, dv, dstate) of linear_attention for the gradients `do` of o and
    `dstate` of the last state; the returned dstate is the first state's.
    Entries not in `need` are None, and dstate without `state`."""
    if stream is not None:
        with _on(stream, q):
            return linear_attention_backward(q, k, v, log_decay, do, state, dstate, lengths, scale, need)
    B, T, H, Dk, Dv = _attention_problem(q, v, log_decay, lengths, state, dstate)
    dt = q.dtype
    pq, sq = _heads(q, (B, T, H, Dk), dt)
    pk, sk = _heads(k, (B, T, H, Dk), dt)
    pv, sv = _heads(v, (B, T, H, Dv), dt)
    po, so = _heads(do, (B, T, H, Dv), dt)
    index = _index_of(q, k, v, log_decay, do, state, dstate, lengths)
    dev = q.device

    def new(name, D):
        return torch.empty((B, T, H, D), dtype=dt, device=dev) if name in need else None

    dq, dk, dv = new("dq", Dk), new("dk", Dk), new("dv", Dv)
    dfirst = None
    if "dstate" in need and state is not None:
        dfirst = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev)
    sqk, svv = _strides(T * H * Dk, H * Dk, Dk), _strides(T * H * Dv, H * Dv, Dv)
    code = dtype_code(dt)
    nws = _attention_workspace_bytes(B, T, H, Dk, Dv, code, 1, index)
    ws = torch.empty((nws,), dtype=torch.uint8, device=dev) if nws else None
    _call(lib().ct_linear_attention_backward, index, pq, sq, pk, sk, pv, sv, po, so, _dense(log_decay),
          _dense(state), _dense(dstate), _dense(lengths), _dense(dq), sqk, _dense(dk), sqk, _dense(dv), svv,
          _dense(dfirst), _dense(ws), nws, B, T, H, Dk, Dv, Dk ** -0.5 if scale is None else scale, code)
    return dq, dk, dv, dfirst


class LinearAttentionFunction(torch.autograd.Function):
    """torch.autograd binding of linear_attention (the decays are constants)."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, state, lengths, scale):
        ctx.save_for_backward(q, k, v, log_decay, state, lengths)
        ctx.scale = scale
        return linear_attention(q, k, v, log_decay, state, lengths, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dstate):
        q, k, v, log_decay, state, lengths = ctx.saved_tensors
        need = tuple(n for n, i in (("dq", 0), ("dk", 1), ("dv", 2), ("dstate", 4)) if ctx.needs_input_grad[i])
        dq, dk, dv, dfirst = linear_attention_backward(q, k, v, log_decay, do.contiguous(), state, dstate.contiguous(),
                                                       lengths, ctx.scale, need)
        return dq, dk, dv, None, dfirst, None, None


def linear_attention_autograd(q, k, v, log_decay, state=None, lengths=None, scale: Optional[float] = None):
    """linear_attention that records itself for torch.autograd; returns (o, state).

    The decays are constants: a log_decay that asks for a gradient is refused
    (it would get none); pass log_decay.detach()."""
    if log_decay.requires_grad and torch.is_grad_enabled():
        raise CtError(CT_ERR_PARAM, "log_decay gets no gradient: pass log_decay.detach()")
    return LinearAttentionFunction.apply(q, k, v, log_decay, state, lengths, scale)
