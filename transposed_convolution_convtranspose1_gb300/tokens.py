"""Binding of the layers of an image or video decoder on channels-last tokens:
group norm with its activation, rotary positions with several axes, and the
gated projection of a feed-forward layer (include/ct.h).

Argument marshalling only, as in block.py: every step of the computation runs
in libct.so on the current stream of the tensors' device.  A call given
`stream` runs as if that were the current one, outputs included.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple, Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from .block import (_activation, _call, _check_weight, _dense, _extent, _heads, _index_of, _like, _on, _rows, _strides)
from .ct import CT_ERR_DTYPE, CT_ERR_GROUPS, CT_ERR_PARAM, CT_ERR_SHAPE, CtError, _check, dtype_code, lib

CT_POS_I32, CT_POS_I64, CT_POS_F32 = 0, 1, 2
_POSITION_DTYPE = {torch.int32: CT_POS_I32, torch.int64: CT_POS_I64, torch.float32: CT_POS_F32}
_I64x2 = ctypes.c_int64 * 2


def _act(activation) -> int:
    return 0 if activation is None else _activation(activation)


@functools.lru_cache(maxsize=256)
def _two(a: int, b: int):
    return _I64x2(a, b)


# ---- group norm ------------------------------------------------------------

def _samples(t: Optional[torch.Tensor], like: Optional[torch.Tensor] = None):
    """(pointer, strides of batch and position) of a [B, ..., C] tensor."""
    if t is None:
        return None, None
    shape = t.shape
    if like is not None:
        if shape != like.shape:
            raise CtError(CT_ERR_SHAPE, f"expected shape {tuple(like.shape)}, got {tuple(shape)}")
        if t.dtype is not like.dtype:
            raise CtError(CT_ERR_DTYPE, f"expected {like.dtype}, got {t.dtype}")
    if len(shape) < 2:
        raise CtError(CT_ERR_SHAPE, "x is [B, ..., C]")
    if t.is_contiguous():
        C = shape[-1]
        return t.data_ptr(), _two(t.numel() // shape[0] if shape[0] else 0, C)
    strides = t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError("the last axis must be dense")
    row, below = shape[-1], None
    for n, st in zip(reversed(shape[1:-1]), reversed(strides[1:-1])):
        if n == 1:
            continue
        if below is None:
            row = st
        elif st != below:
            raise ValueError("the positions of a sample must be evenly spaced rows")
        below = st * n
    return t.data_ptr(), _two(strides[0], row)


def _norm_sizes(x, groups):
    shape = x.shape
    B, C = shape[0], shape[-1]
    if C < 1:
        raise CtError(CT_ERR_SHAPE, "at least one channel is expected")
    groups = int(groups)
    if groups < 1 or C % groups:
        raise CtError(CT_ERR_GROUPS, f"groups must divide the {C} channels (got {groups})")
    return B, x.numel() // (B * C) if B else math.prod(shape[1:-1]), C, groups


@functools.lru_cache(maxsize=256)
def _norm_workspace_bytes(B, S, C, groups, code, backward, index):
    n = ctypes.c_size_t(0)
    with torch.cuda.device(index):
        _check(lib().ct_group_norm_workspace_bytes(B, S, C, groups, code, backward, ctypes.byref(n)))
    return n.value


def group_norm(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, activation=None, alpha: float = 0.01, stream=None):
    """Group norm over [B, ..., C] with the channels last, the activation after it.

    A group is C / groups neighbouring channels at all positions of a sample.
    Returns (y, mean, rstd), mean and rstd float32 [B, groups] (the gradient
    needs them).  x may have any strides with dense channels and evenly spaced
    positions: an image in torch.channels_last is passed as
    x.permute(0, 2, 3, 1), without a copy.
    """
    if stream is not None:
        with _on(stream, x):
            return group_norm(x, groups, weight, bias, eps, activation, alpha)
    px, sx = _samples(x)
    B, S, C, groups = _norm_sizes(x, groups)
    _check_weight(weight, x)
    _check_weight(bias, x)
    act = _act(activation)
    index = _index_of(x, weight, bias)
    code = dtype_code(x.dtype)
    nws = _norm_workspace_bytes(B, S, C, groups, code, 0, index)
    y = _like(x)
    mean = torch.empty((B, groups), dtype=torch.float32, device=x.device)
    rstd = torch.empty((B, groups), dtype=torch.float32, device=x.device)
    ws = torch.empty((nws,), dtype=torch.uint8, device=x.device) if nws else None
    _call(lib().ct_group_norm_forward, index, px, sx, _dense(weight), _dense(bias), y.data_ptr(), _two(S * C, C),
          mean.data_ptr(), rstd.data_ptr(), _dense(ws), nws, B, S, C, groups, eps, act, alpha, code)
    return y, mean, rstd


def group_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, activation=None,
                        alpha: float = 0.01, need=("dx", "dweight", "dbias"), stream=None):
    """(dx, dweight, dbias) of group_norm from its x, mean and rstd [B, groups].
    Entries not in `need` are None, and dweight and dbias where there is no
    weight or bias."""
    if stream is not None:
        with _on(stream, x):
            return group_norm_backward(dy, x, mean, rstd, weight, bias, activation, alpha, need)
    px, sx = _samples(x)
    pd, sd = _samples(dy, x)
    if mean.dim() != 2 or mean.shape[0] != x.shape[0] or mean.dtype != torch.float32:
        raise CtError(CT_ERR_SHAPE, f"mean and rstd are float32 [{x.shape[0]}, groups]")
    if rstd.shape != mean.shape or rstd.dtype != torch.float32:
        raise CtError(CT_ERR_SHAPE, f"rstd must be float32 {tuple(mean.shape)}")
    B, S, C, groups = _norm_sizes(x, mean.shape[1])
    _check_weight(weight, x)
    _check_weight(bias, x)
    act = _act(activation)
    index = _index_of(x, dy, mean, rstd, weight, bias)
    code = dtype_code(x.dtype)
    nws = _norm_workspace_bytes(B, S, C, groups, code, 1, index)
    dx = _like(x) if "dx" in need else None
    dw = torch.empty((C,), dtype=x.dtype, device=x.device) if "dweight" in need and weight is not None else None
    db = torch.empty((C,), dtype=x.dtype, device=x.device) if "dbias" in need and bias is not None else None
    ws = torch.empty((nws,), dtype=torch.uint8, device=x.device) if nws else None
    _call(lib().ct_group_norm_backward, index, pd, sd, px, sx, _dense(mean), _dense(rstd), _dense(weight), _dense(bias),
          _dense(dx), _two(S * C, C), _dense(dw), _dense(db), _dense(ws), nws, B, S, C, groups, act, alpha, code)
    return dx, dw, db


class GroupNormFunction(torch.autograd.Function):
    """torch.autograd binding of group_norm."""

    @staticmethod
    def forward(ctx, x, groups, weight, bias, eps, activation, alpha):
        y, mean, rstd = group_norm(x, groups, weight, bias, eps, activation, alpha)
        ctx.save_for_backward(x, mean, rstd, weight, bias)
        ctx.args = (activation, alpha)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight, bias = ctx.saved_tensors
        need = tuple(n for n, i in (("dx", 0), ("dweight", 2), ("dbias", 3)) if ctx.needs_input_grad[i])
        dx, dw, db = group_norm_backward(dy.contiguous(), x, mean, rstd, weight, bias, *ctx.args, need=need)
        return dx, None, dw, db, None, None, None


def group_norm_autograd(x, groups: int, weight=None, bias=None, eps: float = 1e-5, activation=None, alpha: float = 0.01):
    """group_norm that records itself for torch.autograd; returns y."""
    return GroupNormFunction.apply(x, groups, weight, bias, eps, activation, alpha)


# ---- rotary positions ------------------------------------------------------

class RotaryTable(NamedTuple):
    """How far each pair of a head turns for a step along its axis: turns
    (int64, the bits of an unsigned fraction of a turn in units of 2^-64), and
    the number of pairs of each axis."""
    turns: torch.Tensor
    sections: Tuple[int, ...]


def rotary_table(sections: Sequence[int], base: float = 10000.0, shared: bool = False, frequencies=None,
                 device="cuda") -> RotaryTable:
    """The table of `rotary` for sections[a] pairs on axis a.

    Pair i of an axis with n pairs turns base**(-i / n) radians a step; with
    `shared` the ladder runs over the pairs of all axes instead.  `frequencies`
    gives the radians of every pair instead (at least 0, below 2 pi).
    """
    sections = tuple(int(n) for n in sections)
    if not 1 <= len(sections) <= 4 or min(sections) < 0:
        raise CtError(CT_ERR_PARAM, f"1 to 4 axes of at least 0 pairs, got {sections}")
    if frequencies is None:
        if not base > 0:
            raise CtError(CT_ERR_PARAM, f"base must be above 0, got {base}")
        ladders = (sum(sections),) if shared else sections
        frequencies = [float(base) ** (-i / n) for n in ladders for i in range(n)]
    else:
        frequencies = [float(f) for f in frequencies]
    if len(frequencies) != sum(sections):
        raise CtError(CT_ERR_SHAPE, f"{len(frequencies)} frequencies for {sum(sections)} pairs")
    if not all(0 <= f < 2 * math.pi for f in frequencies):
        raise CtError(CT_ERR_PARAM, "frequencies are radians a step, at least 0 and below 2 pi")
    turns = [min(int(f / (2 * math.pi) * 2.0 ** 64), 2 ** 64 - 1) for f in frequencies]
    return RotaryTable(torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64).to(device), sections)


@functools.lru_cache(maxsize=64)
def _sections(sections):
    return (ctypes.c_int64 * max(len(sections), 1))(*sections)


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, table: RotaryTable, interleaved: bool = False,
           inverse: bool = False, out=None, stream=None):
    """Queries and keys turned by their positions along several axes.

    q [B, T, Hq, D], k [B, T, Hk, D] (or None; any strides, last axis dense),
    positions [B, T, axes] or [T, axes] (int32, int64, or float32 between grid
    points).  Pair i is (i, i + pairs), or (2i, 2i + 1) with `interleaved`; what
    follows the pairs is copied.  `inverse` turns back (the gradient).  Returns
    (q, k) turned, in `out` (a pair, which may be q and k themselves) if given;
    autograd does not see that, so `out` may not ask for a gradient where
    gradients are recorded.
    """
    if stream is not None:
        with _on(stream, q):
            return rotary(q, k, positions, table, interleaved, inverse, out)
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise CtError(CT_ERR_SHAPE, "q and k are [B, T, heads, D]")
    B, T, Hq, D = q.shape
    Hk = k.shape[2] if k is not None else 0
    dt = q.dtype
    axes = len(table.sections)
    if positions.dtype not in _POSITION_DTYPE:
        raise CtError(CT_ERR_DTYPE, f"positions are int32, int64 or float32, got {positions.dtype}")
    if positions.shape == (B, T, axes):
        sp = _strides(*positions.stride())
    elif positions.shape == (T, axes):
        sp = _strides(0, *positions.stride())
    else:
        raise CtError(CT_ERR_SHAPE, f"positions must be [{B}, {T}, {axes}] or [{T}, {axes}], got {tuple(positions.shape)}")
    if table.turns.dtype != torch.int64 or table.turns.shape != (sum(table.sections),):
        raise CtError(CT_ERR_SHAPE, "the table is not one of rotary_table's")
    pq, sq = _heads(q, (B, T, Hq, D), dt)
    pk, sk = _heads(k, (B, T, Hk, D), dt)
    if out is None:
        index = _index_of(q, k, positions, table.turns)
        qo = torch.empty((B, T, Hq, D), dtype=dt, device=q.device)
        pqo, sqo = qo.data_ptr(), _strides(T * Hq * D, Hq * D, D)
        ko = pko = sko = None
        if k is not None:
            ko = torch.empty((B, T, Hk, D), dtype=dt, device=q.device)
            pko, sko = ko.data_ptr(), _strides(T * Hk * D, Hk * D, D)
    else:
        qo, ko = out
        if (ko is None) != (k is None):
            raise CtError(CT_ERR_SHAPE, "out has a second entry exactly where there is k")
        if torch.is_grad_enabled() and (qo.requires_grad or (ko is not None and ko.requires_grad)):
            raise CtError(CT_ERR_PARAM, "out may not ask for a gradient: call rotary_autograd, or under torch.no_grad()")
        pqo, sqo = _heads(qo, (B, T, Hq, D), dt)
        pko, sko = _heads(ko, (B, T, Hk, D), dt)
        index = _index_of(q, k, positions, table.turns, qo, ko)
    _call(lib().ct_rotary, index, pq, sq, pk, sk, pqo, sqo, pko, sko, positions.data_ptr(), sp,
          _POSITION_DTYPE[positions.dtype], _dense(table.turns), _sections(table.sections), axes, B, T, Hq, Hk, D,
          int(interleaved), int(inverse), dtype_code(dt))
    if out is not None:  # a backward pass that kept them finds out
        increment_version(qo if ko is None else (qo, ko))
    return qo, ko


class RotaryFunction(torch.autograd.Function):
    """torch.autograd binding of rotary: the gradient turns back."""

    @staticmethod
    def forward(ctx, q, k, positions, turns, sections, interleaved):
        ctx.save_for_backward(positions, turns)
        ctx.args = (sections, interleaved)
        qo, ko = rotary(q, k, positions, RotaryTable(turns, sections), interleaved)
        return (qo, ko) if k is not None else qo

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk=None):
        positions, turns = ctx.saved_tensors
        sections, interleaved = ctx.args
        dq, dk = rotary(dq.contiguous(), dk.contiguous() if dk is not None else None, positions, RotaryTable(turns, sections),
                        interleaved, inverse=True)
        return dq, dk, None, None, None, None


def rotary_autograd(q, k, positions, table: RotaryTable, interleaved: bool = False):
    """rotary that records itself for torch.autograd; returns (q, k), or q where
    k is None.  Positions are constants."""
    if positions.requires_grad and torch.is_grad_enabled():
        raise CtError(CT_ERR_PARAM, "positions get no gradient: pass positions.detach()")
    return RotaryFunction.apply(q, k, positions, table.turns, table.sections, interleaved)


# ---- gated projection ------------------------------------------------------

_ALIGNED, _WEIGHTS_F, _WEIGHTS_C = 1, 2, 4  # CT_GATED_*: what the workspace query is told


def _weights(x, w_gate, w_up):
    """(gate, up) as [C, F] matrices; w_up None: w_gate holds both, [C, 2F]."""
    if w_up is None:
        if w_gate.dim() != 2 or w_gate.shape[1] % 2:
            raise CtError(CT_ERR_SHAPE, f"a weight for both is [C, 2F], got {tuple(w_gate.shape)}")
        F = w_gate.shape[1] // 2
        w_gate, w_up = w_gate[:, :F], w_gate[:, F:]
    if w_gate.dim() != 2 or w_gate.shape != w_up.shape or w_gate.shape[0] != x.shape[-1]:
        raise CtError(CT_ERR_SHAPE, f"the weights must be [{x.shape[-1]}, F], got {tuple(w_gate.shape)} and {tuple(w_up.shape)}")
    if w_gate.dtype is not x.dtype or w_up.dtype is not x.dtype:
        raise CtError(CT_ERR_DTYPE, f"the weights must be {x.dtype}, got {w_gate.dtype} and {w_up.dtype}")
    return w_gate, w_up


def _in_place(p, rows, cols, stride, e) -> bool:
    """Whether rows of `cols` elements of e bytes can be read as they lie:
    multiples of 16 bytes, rows that do not overlap."""
    return not p & 15 and (rows <= 1 or (stride >= cols and not stride * e & 15))


def _weights_in_place(pg, sg, pu, su, C, F, f_dense, e) -> bool:
    """The same of both weights, read along the axis that is dense in all of them and their gradients."""
    if f_dense:
        return _in_place(pg, C, F, sg[0], e) and _in_place(pu, C, F, su[0], e)
    return _in_place(pg, F, C, sg[1], e) and _in_place(pu, F, C, su[1], e)


@functools.lru_cache(maxsize=256)
def _projection_workspace_bytes(rows, C, F, code, backward, aligned, index):
    n = ctypes.c_size_t(0)
    with torch.cuda.device(index):
        _check(lib().ct_gated_projection_workspace_bytes(rows, C, F, code, backward, aligned, ctypes.byref(n)))
    return n.value


def gated_projection(x: torch.Tensor, w_gate: torch.Tensor, w_up: Optional[torch.Tensor] = None, activation="silu",
                     alpha: float = 0.01, stream=None) -> torch.Tensor:
    """act(x @ w_gate) * (x @ w_up) in one pass, x [..., C], weights [C, F].

    The weights may be halves of one tensor or transposed [F, C] ones: one axis
    dense, the same for both.  With w_up None, w_gate is [C, 2F] and holds both.
    """
    if stream is not None:
        with _on(stream, x):
            return gated_projection(x, w_gate, w_up, activation, alpha)
    act = _act(activation)
    px, sx = _rows(x)
    rows, C = _extent(x)
    gate, up = _weights(x, w_gate, w_up)
    F = gate.shape[1]
    index = _index_of(x, gate, up)
    code, e = dtype_code(x.dtype), x.element_size()
    y = torch.empty((*x.shape[:-1], F), dtype=x.dtype, device=x.device)
    sg, su, pg, pu = gate.stride(), up.stride(), gate.data_ptr(), up.data_ptr()
    f_dense = F <= 1 or sg[1] == su[1] == 1
    aligned = 0
    if _weights_in_place(pg, sg, pu, su, C, F, f_dense, e):
        aligned = (_WEIGHTS_F if f_dense else _WEIGHTS_C) | (_ALIGNED if _in_place(px, rows, C, sx, e) else 0)
    nws = _projection_workspace_bytes(rows, C, F, code, 0, aligned, index)
    ws = torch.empty((nws,), dtype=torch.uint8, device=x.device) if nws else None
    _call(lib().ct_gated_projection_forward, index, px, sx, pg, _two(*sg), pu, _two(*su),
          y.data_ptr(), F, _dense(ws), nws, rows, C, F, act, alpha, code)
    return y


def gated_projection_backward(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: Optional[torch.Tensor] = None,
                              activation="silu", alpha: float = 0.01, need=("dx", "dw_gate", "dw_up"), stream=None):
    """(dx, dw_gate, dw_up) of gated_projection; the projections are formed
    again from x.  Weight gradients are laid out as the weights are; with w_up
    None the one of both halves is dw_gate.  Entries not in `need` are None."""
    if stream is not None:
        with _on(stream, x):
            return gated_projection_backward(dy, x, w_gate, w_up, activation, alpha, need)
    act = _act(activation)
    px, sx = _rows(x)
    rows, C = _extent(x)
    gate, up = _weights(x, w_gate, w_up)
    F = gate.shape[1]
    if dy.shape != (*x.shape[:-1], F):
        raise CtError(CT_ERR_SHAPE, f"dy must be {(*x.shape[:-1], F)}, got {tuple(dy.shape)}")
    pd, sd = _rows(dy, None, x.dtype)
    index = _index_of(x, dy, gate, up)
    code, e, dev = dtype_code(x.dtype), x.element_size(), x.device
    sg, su = gate.stride(), up.stride()
    in_dense = sg[0] == 1 and not (sg[1] == 1 and C == 1)

    def like_weight(f):  # [C, f], the weights' dense axis dense
        return torch.empty((f, C), dtype=x.dtype, device=dev).t() if in_dense else torch.empty((C, f), dtype=x.dtype, device=dev)

    dx = _like(x) if "dx" in need else None
    if w_up is None:
        both = like_weight(2 * F) if "dw_gate" in need or "dw_up" in need else None
        dg, du = (both[:, :F], both[:, F:]) if both is not None else (None, None)
    else:
        both = None
        dg = like_weight(F) if "dw_gate" in need else None
        du = like_weight(F) if "dw_up" in need else None
    sdg, sdu = dg.stride() if dg is not None else (0, 0), du.stride() if du is not None else (0, 0)
    f_dense = F <= 1 or (sg[1] == su[1] == 1 and (dg is None or sdg[1] == 1) and (du is None or sdu[1] == 1))
    aligned = _ALIGNED if (_in_place(px, rows, C, sx, e) and _in_place(pd, rows, F, sd, e)
                           and _weights_in_place(gate.data_ptr(), sg, up.data_ptr(), su, C, F, f_dense, e)) else 0
    nws = _projection_workspace_bytes(rows, C, F, code, 1, aligned, index)
    ws = torch.empty((nws,), dtype=torch.uint8, device=dev) if nws else None
    _call(lib().ct_gated_projection_backward, index, pd, sd, px, sx, gate.data_ptr(), _two(*sg), up.data_ptr(), _two(*su),
          _dense(dx), C, dg.data_ptr() if dg is not None else None, _two(*sdg), du.data_ptr() if du is not None else None,
          _two(*sdu), _dense(ws), nws, rows, C, F, act, alpha, code)
    return dx, both if w_up is None else dg, du if w_up is not None else None


class GatedProjectionFunction(torch.autograd.Function):
    """torch.autograd binding of gated_projection: only its inputs are kept."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation, alpha):
        ctx.save_for_backward(x, w_gate, w_up)
        ctx.args = (activation, alpha)
        return gated_projection(x, w_gate, w_up, activation, alpha)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w_gate, w_up = ctx.saved_tensors
        need = tuple(n for n, i in (("dx", 0), ("dw_gate", 1), ("dw_up", 2)) if ctx.needs_input_grad[i])
        dx, dg, du = gated_projection_backward(dy.contiguous(), x, w_gate, w_up, *ctx.args, need=need)
        return dx, dg, du, None, None


def gated_projection_autograd(x, w_gate, w_up=None, activation="silu", alpha: float = 0.01):
    """gated_projection that records itself for torch.autograd."""
    return GatedProjectionFunction.apply(x, w_gate, w_up, activation, alpha)
