"""Torch-tensor front end of the products of rows by expert with each expert's
matrix, in the dtype or in 4 bits (include/topmoe.h).  As in block.py: shape /
dtype checks, output and workspace allocation on the kernels' stream, the
caller's stream (the current one by default).  Nothing here computes any part of
an operator."""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Union

import torch

from . import _binding as B
from .block import (Act8, _call, _code, _empty, _is, _matrix, _need_act8, _on_kernel_stream,
                    _pitched, _scratch)
from .ops import _ptr


class Mx4(NamedTuple):
    """Values [..., C] in 4 bits: q uint8 [..., C / 2], two e2m1 values a byte
    (the first in the low half), and scale uint8 [..., ceil(C / 32)]; value =
    e2m1 * 2^(scale - 127), a scale of 255 NaN."""
    q: torch.Tensor
    scale: torch.Tensor


class MoeLinearGrads(NamedTuple):
    dx: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]


def _experts(shape, expert_offsets: Optional[torch.Tensor], dev, what: str):
    """(E, O, last) of a matrix [E, O, last], or [O, last] without offsets."""
    if len(shape) == 2 and expert_offsets is None:
        return (1, *shape)
    if len(shape) != 3:
        raise ValueError(f"{what} must be [E, out, in], or [out, in] without expert_offsets; got "
                         f"shape {tuple(shape)}")
    E = shape[0]
    if expert_offsets is not None:
        _is(expert_offsets, "expert_offsets", (E + 1,), torch.int32, dev)
    elif E != 1:
        raise ValueError(f"{what} has {E} experts: expert_offsets are needed")
    if not 1 <= E <= B.LINEAR_MAX_EXPERTS:
        B.check(B.ERR_BAD_SHAPE, what)
    return tuple(shape)


def _output(t: Optional[torch.Tensor], name: str, R: int, C: int, dt, dev):
    """(tensor, row pitch) of an output [R, C], the caller's or a new one."""
    if t is None:
        return _empty(R, C, dtype=dt, device=dev), C
    return t, _pitched(t, name, (R, C), dt, dev)


@_on_kernel_stream
def moe_linear_fwd(x: torch.Tensor, w: torch.Tensor,
                   expert_offsets: Optional[torch.Tensor] = None, *,
                   y: Optional[torch.Tensor] = None, stream=None,
                   stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """A linear layer per expert: y[r] = w[e] x[r] for the rows r in
    [expert_offsets[e], expert_offsets[e + 1]).  x [R, K] as moe_dispatch_fwd
    lays rows out (a row pitch is fine), w [E, O, K], expert_offsets [E + 1]
    int32; without them w [O, K] or [1, O, K] takes all rows.  y [R, O], which must
    not overlap x or w; rows of no expert, behind expert_offsets[E], are zeros."""
    R, K = _matrix(x, "x")
    dev, dt = x.device, x.dtype
    code = _code(dt)
    E, O, _ = _experts(w.shape, expert_offsets, dev, "w")
    _is(w, "w", (*w.shape[:-1], K), dt, dev)
    ldx = _pitched(x, "x", (R, K), dt, dev)
    y, ldy = _output(y, "y", R, O, dt, dev)
    _call("moe_linear_fwd", dev, stage_events, x.data_ptr(), ldx, w.data_ptr(),
          _ptr(expert_offsets), R, K, O, E, code, y.data_ptr(), ldy)
    return y


@functools.lru_cache(maxsize=256)
def moe_linear_bwd_workspace_bytes(R: int, K: int, O: int, E: int = 1,
                                   dtype: Optional[torch.dtype] = None) -> int:
    """What moe_linear_bwd needs for gradients in ``dtype``; without it, enough for any."""
    if dtype is None:
        return int(B.lib().moe_linear_bwd_workspace_bytes(R, K, O, E))
    return int(B.lib().moe_linear_bwd_dtype_workspace_bytes(R, K, O, E, _code(dtype)))


@_on_kernel_stream
def moe_linear_bwd(dy: torch.Tensor, x: Optional[torch.Tensor], w: Optional[torch.Tensor],
                   expert_offsets: Optional[torch.Tensor] = None, *,
                   need_dx: bool = True, need_dw: bool = True,
                   dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None,
                   stage_events: Optional[B.StageEvents] = None) -> MoeLinearGrads:
    """Gradients of moe_linear_fwd for dy [R, O]: dx[r] = w[e]^T dy[r] (zeros in
    rows of no expert) and dw[e], the sum over e's rows of dy[r] x[r]^T (zeros
    for an expert without rows).  ``need_dx`` / ``need_dw``: what is not needed is
    None.  x may be None where dw is not needed; w is needed for its shape, its
    values only for dx."""
    R, O = _matrix(dy, "dy")
    dev, dt = dy.device, dy.dtype
    code = _code(dt)
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor")
    E, _, K = _experts(w.shape, expert_offsets, dev, "w")
    _is(w, "w", (*w.shape[:-2], O, K), dt, dev)
    lddy = _pitched(dy, "dy", (R, O), dt, dev)
    ldx = lddx = K
    if need_dw:
        ldx = _pitched(x, "x", (R, K), dt, dev)
        if dw is None:
            dw = _empty(w.shape, dtype=dt, device=dev)
        else:
            _is(dw, "dw", w.shape, dt, dev)
    else:
        dw = None
    if need_dx:
        dx, lddx = _output(dx, "dx", R, K, dt, dev)
    else:
        dx = None
    if dx is None and dw is None:
        return MoeLinearGrads(None, None)
    wp, wn, ws = _scratch(moe_linear_bwd_workspace_bytes(R, K, O, E, dt), "moe_linear_bwd", dev,
                          workspace)
    _call("moe_linear_bwd", dev, stage_events, dy.data_ptr(), lddy, _ptr(x) if need_dw else 0, ldx,
          w.data_ptr(), _ptr(expert_offsets), R, K, O, E, code, _ptr(dx), lddx, _ptr(dw),
          wp, wn)
    return MoeLinearGrads(dx, dw)


# ------------------------------------------------------------ 4 bits
def _flat(t: torch.Tensor, name: str):
    """(rows, C, pitch) of a contiguous [..., C] tensor or a [R, C] one with a row pitch."""
    if t.dim() == 2:
        R, C = t.shape
        return R, C, _pitched(t, name, (R, C), t.dtype, t.device)
    if t.dim() < 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a [R, C] tensor with contiguous rows or a contiguous "
                         f"one of more dimensions")
    C = t.shape[-1]
    return (t.numel() // C if C else 0), C, C


@_on_kernel_stream
def mx4_pack(x: torch.Tensor, *, stream=None,
             stage_events: Optional[B.StageEvents] = None) -> Mx4:
    """x [R, C] (a row pitch is fine) or contiguous [..., C], as the matrices
    [E, O, K] of the experts are, in 4 bits."""
    R, C, ld = _flat(x, "x")
    dev, code = x.device, _code(x.dtype)
    if C <= 0 or C % 8:
        B.check(B.ERR_BAD_SHAPE, "mx4_pack")
    lead = x.shape[:-1]
    p = Mx4(_empty(*lead, C // 2, dtype=torch.uint8, device=dev),
            _empty(*lead, -(-C // B.MX4_GROUP), dtype=torch.uint8, device=dev))
    _call("mx4_pack", dev, stage_events, x.data_ptr(), ld, R, C, code, p.q.data_ptr(),
          p.scale.data_ptr())
    return p


def _need_mx4(p: Mx4, name: str, dev):
    """(leading dimensions, C) of a packed tensor on ``dev``."""
    if not isinstance(p, Mx4) or not isinstance(p.q, torch.Tensor) or p.q.dim() < 2:
        raise TypeError(f"{name} must be an Mx4 of at least two dimensions")
    lead, C = tuple(p.q.shape[:-1]), 2 * p.q.shape[-1]
    _is(p.q, f"{name}.q", p.q.shape, torch.uint8, dev)
    _is(p.scale, f"{name}.scale", (*lead, -(-C // B.MX4_GROUP)), torch.uint8, dev)
    return lead, C


def mx4_unpack(p: Mx4, *, dtype: torch.dtype = torch.bfloat16, x: Optional[torch.Tensor] = None,
               stream=None, stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """The values that mx4_pack kept, [..., C] in ``dtype`` (or into ``x``; the
    rows of a [R, C] one may be pitched)."""
    if not isinstance(p, Mx4):
        raise TypeError("p must be an Mx4")
    return _unpack(p.q, p, dtype, x, stage_events, stream=stream)


@_on_kernel_stream
def _unpack(q, p, dtype, x, stage_events):
    dev = q.device
    lead, C = _need_mx4(p, "p", dev)
    if x is None:
        x = _empty(*lead, C, dtype=dtype, device=dev)
    elif not isinstance(x, torch.Tensor) or tuple(x.shape) != (*lead, C) or x.device != dev:
        raise ValueError(f"x must be a {(*lead, C)} tensor on {dev}")
    R, _, ld = _flat(x, "x")
    _call("mx4_unpack", dev, stage_events, q.data_ptr(), p.scale.data_ptr(), R, C, _code(x.dtype),
          x.data_ptr(), ld)
    return x


def mx4_linear_fwd(x: Union[torch.Tensor, Act8, Mx4], w: Mx4,
                   expert_offsets: Optional[torch.Tensor] = None, *,
                   dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
                   stream=None, stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """moe_linear_fwd with matrices in 4 bits: w an Mx4 of [E, O, K], or of
    [O, K] without expert_offsets.  x [R, K]: a bfloat16 or float32 tensor (a row
    pitch is fine), which is taken as it is; or act8_pack's or mx4_pack's rows,
    which run on the 8- and 4-bit matrix instructions.  y [R, O] in ``dtype``: x's
    own, which is all a plain x can have, and by default bfloat16 for packed
    rows.  K is a multiple of 32.  Of each eight consecutive products of 8-bit rows
    a bfloat16 y misses up to 2^-12 of the largest, which shows where large ones
    cancel; dtype=torch.float32 has whole sums.  To plain rows,
    and to 8-bit rows with a float32 y, matrix elements of 2^128 and more are infinite."""
    packed = isinstance(x, (Act8, Mx4))
    return _mx4_fwd(x.q if packed else x, x, w, expert_offsets, dtype, y, stage_events,
                    stream=stream)


@_on_kernel_stream
def _mx4_fwd(x, rows, w, expert_offsets, dtype, y, stage_events):
    dev = x.device
    lead, K = _need_mx4(w, "w", dev)
    E, O, _ = _experts((*lead, K), expert_offsets, dev, "w")
    xs = None
    if rows is x:
        R, kx = _matrix(x, "x")
        kind, dt = B.ROWS_PLAIN, x.dtype
        if dtype is not None and dtype is not dt:
            raise TypeError(f"a {dt} x has y in {dt}, not {dtype}")
        ldx = _pitched(x, "x", (R, kx), dt, dev)
    else:
        dt = torch.bfloat16 if dtype is None else dtype
        xs = rows.scale
        R, kx = _matrix(x, "x.q")
        if isinstance(rows, Act8):
            kind = B.ROWS_ACT8
            _need_act8(rows, "x", R, kx, dev)
        else:
            kind = B.ROWS_MX4
            kx = _need_mx4(rows, "x", dev)[1]
        ldx = kx
    if kx != K:
        raise ValueError(f"x has {kx} channels, w {K}")
    code = _code(dt)
    if K % B.MX4_GROUP:
        B.check(B.ERR_BAD_SHAPE, "mx4_linear_fwd")
    y, ldy = _output(y, "y", R, O, dt, dev)
    _call("mx4_linear_fwd", dev, stage_events, x.data_ptr(), ldx, _ptr(xs), kind, w.q.data_ptr(),
          w.scale.data_ptr(), _ptr(expert_offsets), R, K, O, E, code, y.data_ptr(), ldy)
    return y


@functools.lru_cache(maxsize=256)
def mx4_linear_bwd_workspace_bytes(R: int, K: int, O: int, E: int = 1) -> int:
    return int(B.lib().mx4_linear_bwd_workspace_bytes(R, K, O, E))


@_on_kernel_stream
def mx4_linear_bwd(dy: torch.Tensor, w: Mx4, expert_offsets: Optional[torch.Tensor] = None, *,
                   dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None, stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """The gradient of a plain x of mx4_linear_fwd for dy [R, O]: dx[r] =
    w[e]^T dy[r] (zeros in rows of no expert).  The matrices are frozen: they
    have no gradient."""
    R, O = _matrix(dy, "dy")
    dev, dt = dy.device, dy.dtype
    code = _code(dt)
    lead, K = _need_mx4(w, "w", dev)
    E, wo, _ = _experts((*lead, K), expert_offsets, dev, "w")
    if wo != O:
        raise ValueError(f"dy has {O} channels, w {wo} rows")
    lddy = _pitched(dy, "dy", (R, O), dt, dev)
    wp, wn, ws = _scratch(mx4_linear_bwd_workspace_bytes(R, K, O, E), "mx4_linear_bwd", dev,
                          workspace)
    dx, lddx = _output(dx, "dx", R, K, dt, dev)
    _call("mx4_linear_bwd", dev, stage_events, dy.data_ptr(), lddy, w.q.data_ptr(),
          w.scale.data_ptr(), _ptr(expert_offsets), R, K, O, E, code, dx.data_ptr(), lddx, wp, wn)
    return dx
