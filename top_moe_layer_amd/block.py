"""Torch-tensor front end of the operators around an FFN / MoE block: rows by
expert and back, norms with gate and residual, activations in 8 bits
(include/topmoe.h).  As in ops.py: shape / dtype checks, output and workspace
allocation on the kernels' stream, the caller's stream (the current one by
default).  Nothing here computes any part of an operator."""
from __future__ import annotations

import functools
import inspect
import math
from typing import NamedTuple, Optional

import torch

from . import _binding as B
from .ops import _buffer, _dtype_code, _need, _ptr, _torch_stream


# The current stream's handle without a Stream object (0.1 us a call instead of 2.8).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_empty = torch.empty
_CODES = {torch.float32: B.DTYPE_FP32, torch.bfloat16: B.DTYPE_BF16}


def _on_kernel_stream(fn=None, *, of: int = 0):
    """Call ``fn`` with the stream its kernels run on as torch's current
    stream: ``stream`` (an object or a raw handle; ``fn`` itself never sees
    it) or, by default, the current stream of the device of its argument
    ``of``, where ``fn`` is called as it is."""
    if fn is None:
        return functools.partial(_on_kernel_stream, of=of)
    name = list(inspect.signature(fn).parameters)[of]

    @functools.wraps(fn)
    def wrapped(*args, stream=None, **kw):
        t = args[of] if len(args) > of else kw.get(name)
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{fn.__name__}: {name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (got {t.device}); the library has no "
                             f"CPU path")
        if stream is None and t.get_device() == torch.cuda.current_device():
            return fn(*args, **kw)
        ts = _torch_stream(t.device, stream)
        if ts.device != t.device:
            raise ValueError(f"stream is on {ts.device}, {name} on {t.device}")
        with torch.cuda.stream(ts):
            return fn(*args, **kw)
    return wrapped


def _code(dt: torch.dtype) -> int:
    code = _CODES.get(dt)
    return _dtype_code(dt) if code is None else code


def _is(t, name: str, shape, dt, dev) -> None:
    """ops._need, which words the refusal, behind the checks in their quickest order."""
    try:
        if t.shape == shape and t.dtype is dt and t.is_contiguous() and t.device == dev:
            return
    except AttributeError:
        pass
    _need(t, name, shape, dt, dev)


def _rows(t: torch.Tensor, name: str):
    """(N, H) of a contiguous [..., H] tensor."""
    shape = t.shape
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if len(shape) == 2:
        return shape
    if not shape:
        raise ValueError(f"{name} needs at least one dimension")
    return (t.numel() // shape[-1] if shape[-1] else 0), shape[-1]


def _scratch(nbytes: int, what: str, dev, ws: Optional[torch.Tensor]):
    """(pointer, bytes, tensor) of a workspace; nbytes 0 is a size the library refuses."""
    if nbytes == 0:
        B.check(B.ERR_BAD_SHAPE, what)
    if ws is None:
        ws = _empty(nbytes, dtype=torch.uint8, device=dev)
        return ws.data_ptr(), nbytes, ws
    _buffer(ws, "workspace", nbytes, dev)
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


# Entry points of more than one stage.
_STAGES = {"moe_dispatch_fwd_capacity": B.DISPATCH_STAGES, "block_prenorm_bwd": B.NORM_BWD_STAGES,
           "block_postnorm_bwd": B.NORM_BWD_STAGES, "ffn_swiglu_restore8": B.RESTORE8_STAGES,
           "moe_ffn_restore8": B.RESTORE8_STAGES, "moe_linear_bwd": B.LINEAR_BWD_STAGES,
           "mx4_linear_bwd": B.MX4_BWD_STAGES}


def _call(name: str, dev, events, *args) -> None:
    """The C entry point, on torch's current stream of ``dev``."""
    if events is not None:
        events = events.for_stages(_STAGES.get(name, 1))
    st = getattr(B.lib(), name)(*args, _raw_stream(dev.index), events)
    if st != B.OK:
        raise B.TopmoeError(st, name)


# ------------------------------------------------------------ rows by expert
class MoeRows(NamedTuple):
    """Rows by expert: xs [N*k, H]; expert_offsets [E+1]; row_entry [N*k] (the
    entry t*k + j of each kept row, then -1); entry_row [N, k] (the entry's
    row, or -1 - row of a zero row behind the kept ones)."""
    xs: torch.Tensor
    expert_offsets: torch.Tensor
    row_entry: torch.Tensor
    entry_row: torch.Tensor


class CombineGrads(NamedTuple):
    dys: torch.Tensor
    dalpha: torch.Tensor


def moe_dispatch_workspace_bytes(N: int, E: int, k: int) -> int:
    return int(B.lib().moe_dispatch_workspace_bytes(N, E, k))


def _capacity(factor: float, N: int, E: int, k: int) -> int:
    """Entries an expert keeps, ceil(factor * N * k / E) as Python evaluates it
    (the C entry point's float would take 1.2 for a little more); 0: all."""
    if factor == 0.0:
        return 0
    if not 0.0 < factor < math.inf:
        B.check(B.ERR_BAD_ARG, "moe_dispatch_fwd")
    c = factor * N * k / E
    return max(math.ceil(c), 1) if c < N * k else 0


@_on_kernel_stream
def moe_dispatch_fwd(x: torch.Tensor, topk_idx: torch.Tensor, E: int, *,
                     capacity_factor: float = 0.0, xs: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     stream=None, stage_events: Optional[B.StageEvents] = None) -> MoeRows:
    """The tokens' rows sorted by expert (stable: ascending token within an
    expert).  x [..., H]; topk_idx [N, k] int32, entries outside [0, E) (a
    padding token's -1) belong to no expert.  ``capacity_factor`` > 0 keeps
    the first ceil(capacity_factor * N * k / E) entries of each expert, in
    Python's floats.  Entries not kept have zero rows behind the experts'
    (from expert_offsets[E])."""
    dev, dt = x.device, x.dtype
    code = _code(dt)
    N, H = _rows(x, "x")
    if not isinstance(topk_idx, torch.Tensor) or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be a [N, k] tensor")
    k = topk_idx.shape[1]
    _is(topk_idx, "topk_idx", (N, k), torch.int32, dev)
    if not 1 <= E <= B.DISPATCH_MAX_EXPERTS:
        B.check(B.ERR_BAD_SHAPE, "moe_dispatch_fwd")
    cap = _capacity(float(capacity_factor), N, E, k)
    wp = wn = ws = None
    if (workspace is not None or N * k > B.DISPATCH_ONE or
            N * (k + 1) * H * x.element_size() >= B.DISPATCH_ONE_BYTES):
        nbytes = moe_dispatch_workspace_bytes(N, E, k)
        wp, wn, ws = _scratch(nbytes, "moe_dispatch_fwd", dev, workspace)
    if xs is None:
        xs = _empty(N * k, H, dtype=dt, device=dev)
    else:
        _is(xs, "xs", (N * k, H), dt, dev)
    offsets = _empty(E + 1, dtype=torch.int32, device=dev)
    row_entry = _empty(N * k, dtype=torch.int32, device=dev)
    entry_row = torch.empty_like(topk_idx)
    _call("moe_dispatch_fwd_capacity", dev, stage_events, x.data_ptr(), topk_idx.data_ptr(), N, H,
          E, k, cap, code, xs.data_ptr(), offsets.data_ptr(), row_entry.data_ptr(),
          entry_row.data_ptr(), wp, wn or 0)
    return MoeRows(xs, offsets, row_entry, entry_row)


def _entry_rows(rows: torch.Tensor, name: str, entry_row: torch.Tensor):
    """(N, H, k) of [N*k, H] rows and their entry_row [N, k]."""
    if not isinstance(entry_row, torch.Tensor) or entry_row.dim() != 2:
        raise ValueError("entry_row must be a [N, k] tensor")
    N, k = entry_row.shape
    _is(entry_row, "entry_row", (N, k), torch.int32, rows.device)
    if rows.dim() != 2:
        raise ValueError(f"{name} must be a [N*k, H] tensor")
    H = rows.shape[1]
    _is(rows, name, (N * k, H), rows.dtype, rows.device)
    return N, H, k


@_on_kernel_stream
def moe_dispatch_bwd(dxs: torch.Tensor, entry_row: torch.Tensor, *,
                     dx: Optional[torch.Tensor] = None,
                     stream=None, stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """Gradient of the dispatch: dx [N, H], each token's kept rows of dxs
    [N*k, H] added in slot order (fp32, rounded once)."""
    N, H, k = _entry_rows(dxs, "dxs", entry_row)
    dev, dt = dxs.device, dxs.dtype
    code = _code(dt)
    if dx is None:
        dx = _empty(N, H, dtype=dt, device=dev)
    else:
        _is(dx, "dx", (N, H), dt, dev)
    _call("moe_dispatch_bwd", dev, stage_events, dxs.data_ptr(), entry_row.data_ptr(), N, H, k,
          code, dx.data_ptr())
    return dx


@_on_kernel_stream
def moe_combine_fwd(ys: torch.Tensor, entry_row: torch.Tensor, alpha: torch.Tensor, *,
                    residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                    stream=None, stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """Experts' rows back to tokens: y [N, H] = residual (or 0; it may be y)
    + the sum over the token's kept entries, in slot order, of alpha [N, k]
    (float32) times their rows of ys [N*k, H]."""
    dev, dt = ys.device, ys.dtype
    N, H, k = _entry_rows(ys, "ys", entry_row)
    code = _code(dt)
    _is(alpha, "alpha", (N, k), torch.float32, dev)
    if residual is not None:
        _is(residual, "residual", (N, H), dt, dev)
    if y is None:
        y = _empty(N, H, dtype=dt, device=dev)
    else:
        _is(y, "y", (N, H), dt, dev)
    _call("moe_combine_fwd", dev, stage_events, ys.data_ptr(), entry_row.data_ptr(),
          alpha.data_ptr(), _ptr(residual), N, H, k, code, y.data_ptr())
    return y


@_on_kernel_stream
def moe_combine_bwd(dy: torch.Tensor, ys: torch.Tensor, entry_row: torch.Tensor,
                    alpha: torch.Tensor, *,
                    stream=None, stage_events: Optional[B.StageEvents] = None) -> CombineGrads:
    """Gradients of the combine for dy [N, H]: dys [N*k, H] (zero rows for
    entries that are not kept) and dalpha [N, k] float32.  entry_row must name
    each row once, as moe_dispatch_fwd's does."""
    dev, dt = ys.device, ys.dtype
    N, H, k = _entry_rows(ys, "ys", entry_row)
    code = _code(dt)
    _is(dy, "dy", (N, H), dt, dev)
    _is(alpha, "alpha", (N, k), torch.float32, dev)
    dys, dalpha = torch.empty_like(ys), torch.empty_like(alpha)
    _call("moe_combine_bwd", dev, stage_events, dy.data_ptr(), ys.data_ptr(), entry_row.data_ptr(),
          alpha.data_ptr(), N, H, k, code, dys.data_ptr(), dalpha.data_ptr())
    return CombineGrads(dys, dalpha)


# ------------------------------------------------------------ norms
class PrenormOutput(NamedTuple):
    n: torch.Tensor
    rstd: torch.Tensor


class PrenormGrads(NamedTuple):
    dx: torch.Tensor
    dw: torch.Tensor


class PostnormOutput(NamedTuple):
    out: torch.Tensor
    rstd: Optional[torch.Tensor]
    n: Optional[torch.Tensor]
    next_rstd: Optional[torch.Tensor]


class PostnormGrads(NamedTuple):
    dy: torch.Tensor
    dresidual: torch.Tensor
    dw: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dnext_w: Optional[torch.Tensor]


@functools.lru_cache(maxsize=256)  # of three numbers; 0.5 us of a 14 us call
def block_norm_bwd_workspace_bytes(N: int, H: int, gate_rows: int = 1) -> int:
    return int(B.lib().block_norm_bwd_workspace_bytes(N, H, gate_rows))


@_on_kernel_stream
def block_prenorm_fwd(x: torch.Tensor, w: torch.Tensor, *, eps: float = 1e-5,
                      n: Optional[torch.Tensor] = None,
                      stream=None, stage_events: Optional[B.StageEvents] = None) -> PrenormOutput:
    """RMS norm before a block: n = w * x * rstd, rstd = 1 / sqrt(mean(x^2) +
    eps) over the last dimension.  x [..., H], w [H]; n has x's shape, rstd
    [N] is float32 (for the backward)."""
    dev, dt = x.device, x.dtype
    code = _code(dt)
    N, H = _rows(x, "x")
    _is(w, "w", (H,), dt, dev)
    if n is None:
        n = torch.empty_like(x)
    else:
        _is(n, "n", x.shape, dt, dev)
    rstd = _empty(N, dtype=torch.float32, device=dev)
    _call("block_prenorm_fwd", dev, stage_events, x.data_ptr(), w.data_ptr(), N, H, float(eps),
          code, n.data_ptr(), rstd.data_ptr())
    return PrenormOutput(n, rstd)


@_on_kernel_stream
def block_prenorm_bwd(dn: torch.Tensor, x: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor, *,
                      dresidual: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None,
                      stream=None, stage_events: Optional[B.StageEvents] = None) -> PrenormGrads:
    """Gradients of block_prenorm_fwd for dn (x's shape).  ``dresidual``: the
    gradient that reaches x along the residual stream, added to dx in the
    same pass."""
    dev, dt = x.device, x.dtype
    code = _code(dt)
    N, H = _rows(x, "x")
    _is(dn, "dn", x.shape, dt, dev)
    _is(w, "w", (H,), dt, dev)
    _is(rstd, "rstd", (N,), torch.float32, dev)
    if dresidual is not None:
        _is(dresidual, "dresidual", x.shape, dt, dev)
    nbytes = block_norm_bwd_workspace_bytes(N, H)
    wp, wn, ws = _scratch(nbytes, "block_prenorm_bwd", dev, workspace)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    _call("block_prenorm_bwd", dev, stage_events, dn.data_ptr(), x.data_ptr(), w.data_ptr(),
          rstd.data_ptr(), _ptr(dresidual), N, H, code, dx.data_ptr(), dw.data_ptr(), wp, wn)
    return PrenormGrads(dx, dw)


def _rows_in_order(lead, of) -> bool:
    """Whether a gate's rows, leading dimensions ``lead``, belong to runs of
    consecutive tokens of a tensor with leading dimensions ``of`` whichever way
    one reads them: one dimension of rows (then only ones), the tensor's own
    dimensions up to one of them, or, beside a tensor of another rank, rows
    none of which stands behind a 1 that could be broadcast over."""
    n = len(lead)
    while n and lead[n - 1] == 1:
        n -= 1
    return n <= 1 or (lead[:n] == of[:n] if len(lead) == len(of) else 1 not in lead[:n])


def _gate(gate: Optional[torch.Tensor], y_shape, N: int, H: int, dt, dev):
    """(gate_mode, gate_rows) of a gate [H], [G, H] / [B, 1, H] (N a multiple
    of the rows) or [..., 1] with one value per token."""
    if gate is None:
        return B.GATE_NONE, 1
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a torch.Tensor")
    shape = tuple(gate.shape)
    _is(gate, "gate", shape, dt, dev)
    if len(shape) > 1 and shape[-1] == 1 and gate.numel() == N:
        if len(shape) != len(y_shape) or _rows_in_order(shape[:-1], tuple(y_shape[:-1])):
            return B.GATE_TOKEN, 1
    if shape and shape[-1] == H:
        rows = gate.numel() // H
        if ((rows and N % rows == 0) or (rows == 0 and N == 0)) and (
                len(shape) < 3 or rows == 0 or _rows_in_order(shape[:-1], tuple(y_shape[:-1]))):
            return B.GATE_CHANNEL, rows
    raise ValueError(f"gate has shape {shape}; expected ({H},), (G, {H}) with G dividing the {N} "
                     f"tokens, or one value per token in a last dimension of 1, with rows in the "
                     f"order of the tokens {tuple(y_shape[:-1])} (a row per position is expanded "
                     f"over the batch first)")


@_on_kernel_stream
def block_postnorm_fwd(y: torch.Tensor, residual: torch.Tensor, w: Optional[torch.Tensor] = None, *,
                       gate: Optional[torch.Tensor] = None, next_w: Optional[torch.Tensor] = None,
                       residual_scale: float = 1.0, eps: float = 1e-5,
                       out: Optional[torch.Tensor] = None,
                       stream=None, stage_events: Optional[B.StageEvents] = None) -> PostnormOutput:
    """After a block with output y [..., H]: out = residual_scale * residual +
    gate * w * y / rms(y), without the norm where ``w`` is None, and with
    ``next_w`` the next block's norm n = next_w * out / rms(out) in the same
    pass.  ``gate``: [H]; [G, H], each row for N / G consecutive tokens, as
    [B, 1, H] is for y [B, S, H]; or one value per token [..., 1].  Gates are
    not broadcast: a [1, S, H], a row per position, is refused unless B is 1.
    ``out`` may be the residual itself."""
    dev, dt = y.device, y.dtype
    code = _code(dt)
    N, H = _rows(y, "y")
    _is(residual, "residual", y.shape, dt, dev)
    if w is not None:
        _is(w, "w", (H,), dt, dev)
    if next_w is not None:
        _is(next_w, "next_w", (H,), dt, dev)
    mode, gate_rows = _gate(gate, y.shape, N, H, dt, dev)
    if out is None:
        out = torch.empty_like(y)
    else:
        _is(out, "out", y.shape, dt, dev)
    rstd = n = next_rstd = None
    if w is not None:
        rstd = _empty(N, dtype=torch.float32, device=dev)
    if next_w is not None:
        n = torch.empty_like(y)
        next_rstd = _empty(N, dtype=torch.float32, device=dev)
    _call("block_postnorm_fwd", dev, stage_events, y.data_ptr(), residual.data_ptr(), _ptr(w),
          _ptr(gate), _ptr(next_w), N, H, mode, gate_rows, float(residual_scale), float(eps), code,
          out.data_ptr(), _ptr(rstd), _ptr(n), _ptr(next_rstd))
    return PostnormOutput(out, rstd, n, next_rstd)


@_on_kernel_stream(of=1)
def block_postnorm_bwd(dout: Optional[torch.Tensor], y: torch.Tensor,
                       w: Optional[torch.Tensor] = None, *, rstd: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None, dn: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, next_w: Optional[torch.Tensor] = None,
                       next_rstd: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                       workspace: Optional[torch.Tensor] = None,
                       stream=None, stage_events: Optional[B.StageEvents] = None) -> PostnormGrads:
    """Gradients of block_postnorm_fwd for dout (and, with ``next_w``, dn; dout
    None is then the gradient of n alone): dy, dresidual (y's shape), dw,
    dnext_w [H] and dgate (the gate's shape).  ``rstd``, ``out`` and ``next_rstd`` as the forward returned them."""
    dev, dt = y.device, y.dtype
    code = _code(dt)
    N, H = _rows(y, "y")
    if dout is not None or next_w is None:
        _is(dout, "dout", y.shape, dt, dev)
    if w is not None:
        _is(w, "w", (H,), dt, dev)
        _is(rstd, "rstd", (N,), torch.float32, dev)
    if next_w is not None:
        _is(next_w, "next_w", (H,), dt, dev)
        _is(dn, "dn", y.shape, dt, dev)
        _is(out, "out", y.shape, dt, dev)
        _is(next_rstd, "next_rstd", (N,), torch.float32, dev)
    elif dn is not None:
        raise ValueError("dn needs next_w")
    mode, gate_rows = _gate(gate, y.shape, N, H, dt, dev)
    nbytes = block_norm_bwd_workspace_bytes(N, H, gate_rows)
    wp, wn, ws = _scratch(nbytes, "block_postnorm_bwd", dev, workspace)
    new = torch.empty_like
    dy, dresidual = new(y), new(y)
    dw = new(w) if w is not None else None
    dnext_w = new(next_w) if next_w is not None else None
    dgate = new(gate) if gate is not None else None
    _call("block_postnorm_bwd", dev, stage_events, _ptr(dout), _ptr(dn), y.data_ptr(),
          _ptr(out), _ptr(w), _ptr(gate), _ptr(next_w), _ptr(rstd), _ptr(next_rstd), N, H, mode,
          gate_rows, float(residual_scale), code, dy.data_ptr(), dresidual.data_ptr(), _ptr(dw),
          _ptr(dgate), _ptr(dnext_w), wp, wn)
    return PostnormGrads(dy, dresidual, dw, dgate, dnext_w)


# ------------------------------------------------------------ 8-bit activations
class Act8(NamedTuple):
    """An activation [R, C] in 8 bits: q float8_e4m3fn [R, C] and scale uint8
    [R, ceil(C / 32)], value = q * 2^(scale - 127)."""
    q: torch.Tensor
    scale: torch.Tensor


class SwigluAct8(NamedTuple):
    h: torch.Tensor
    g8: Act8
    u8: Act8


class SwigluAct8Grads(NamedTuple):
    dg: torch.Tensor
    du: torch.Tensor
    h: Optional[torch.Tensor]


def _pitched(t: torch.Tensor, name: str, shape, dt, dev) -> int:
    """Row pitch of a [R, C] tensor whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape == shape and t.dtype is dt and t.is_contiguous() and t.device == dev:
        return shape[1]
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev} (the library has no CPU path)")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dt:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dt}")
    if t.stride(1) != 1 or t.stride(0) < shape[1]:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.stride(0)


def _need_act8(a: Act8, name: str, R: int, C: int, dev) -> None:
    _is(a.q, f"{name}.q", (R, C), torch.float8_e4m3fn, dev)
    _is(a.scale, f"{name}.scale", (R, -(-C // B.ACT8_GROUP)), torch.uint8, dev)


def _new_act8(R: int, C: int, dev) -> Act8:
    return Act8(_empty(R, C, dtype=torch.float8_e4m3fn, device=dev),
                _empty((R, -(-C // B.ACT8_GROUP)), dtype=torch.uint8, device=dev))


def _matrix(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a [R, C] tensor, got shape {tuple(t.shape)}")
    return t.shape


@_on_kernel_stream
def act8_pack(x: torch.Tensor, *, stream=None,
              stage_events: Optional[B.StageEvents] = None) -> Act8:
    """x [R, C] (contiguous rows; a row pitch is fine) in 8 bits."""
    R, C = _matrix(x, "x")
    dev, dt = x.device, x.dtype
    code = _code(dt)
    ld = _pitched(x, "x", (R, C), dt, dev)
    a = _new_act8(R, C, dev)
    _call("act8_pack", dev, stage_events, x.data_ptr(), ld, R, C, code, a.q.data_ptr(),
          a.scale.data_ptr())
    return a


@_on_kernel_stream
def act8_unpack(q: torch.Tensor, scale: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16,
                x: Optional[torch.Tensor] = None,
                stream=None, stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """The activation that act8_pack kept, [R, C] in ``dtype`` (or into ``x``,
    whose rows may be pitched)."""
    R, C = _matrix(q, "q")
    dev = q.device
    _need_act8(Act8(q, scale), "act8", R, C, dev)
    if x is None:
        x = _empty(R, C, dtype=dtype, device=dev)
    code = _code(x.dtype)
    ld = _pitched(x, "x", (R, C), x.dtype, dev)
    _call("act8_unpack", dev, stage_events, q.data_ptr(), scale.data_ptr(), R, C, code,
          x.data_ptr(), ld)
    return x


@_on_kernel_stream
def swiglu_act8_fwd(g: torch.Tensor, u: torch.Tensor, *, h: Optional[torch.Tensor] = None,
                    stream=None, stage_events: Optional[B.StageEvents] = None) -> SwigluAct8:
    """h = SiLU(g) * u, with g and u [R, C] kept in 8 bits for
    swiglu_act8_bwd.  g and u may be the halves of one [R, 2C] projection."""
    R, C = _matrix(g, "g")
    dev, dt = g.device, g.dtype
    code = _code(dt)
    ldg = _pitched(g, "g", (R, C), dt, dev)
    ldu = _pitched(u, "u", (R, C), dt, dev)
    if h is None:
        h = _empty(R, C, dtype=dt, device=dev)
    else:
        _is(h, "h", (R, C), dt, dev)
    g8, u8 = _new_act8(R, C, dev), _new_act8(R, C, dev)
    _call("swiglu_act8_fwd", dev, stage_events, g.data_ptr(), ldg, u.data_ptr(), ldu, R, C, code,
          h.data_ptr(), g8.q.data_ptr(), g8.scale.data_ptr(), u8.q.data_ptr(), u8.scale.data_ptr())
    return SwigluAct8(h, g8, u8)


@_on_kernel_stream
def swiglu_act8_bwd(dh: torch.Tensor, g8: Act8, u8: Act8, *, with_h: bool = True,
                    dg: Optional[torch.Tensor] = None, du: Optional[torch.Tensor] = None,
                    stream=None, stage_events: Optional[B.StageEvents] = None) -> SwigluAct8Grads:
    """Gradients of swiglu_act8_fwd from the kept g and u for dh [R, C]: dg,
    du and, with ``with_h``, h again (for the down projection's gradient).  By
    default dg and du are the halves of one new [R, 2C] tensor."""
    R, C = _matrix(dh, "dh")
    dev, dt = dh.device, dh.dtype
    code = _code(dt)
    _is(dh, "dh", (R, C), dt, dev)
    _need_act8(g8, "g8", R, C, dev)
    _need_act8(u8, "u8", R, C, dev)
    if (dg is None) != (du is None):
        raise ValueError("dg and du go together")
    if dg is None:
        dgu = _empty(R, 2 * C, dtype=dt, device=dev)
        dg, du = dgu[:, :C], dgu[:, C:]
    lddg = _pitched(dg, "dg", (R, C), dt, dev)
    lddu = _pitched(du, "du", (R, C), dt, dev)
    h = torch.empty_like(dh) if with_h else None
    _call("swiglu_act8_bwd", dev, stage_events, g8.q.data_ptr(), g8.scale.data_ptr(),
          u8.q.data_ptr(), u8.scale.data_ptr(), dh.data_ptr(), R, C, code, dg.data_ptr(), lddg,
          du.data_ptr(), lddu, _ptr(h))
    return SwigluAct8Grads(dg, du, h)


# ------------------------------------------------ the FFN's own activations in 8 bits
def ffn_keep8_bytes(N: int, H: int, I: int, dtype: torch.dtype) -> int:
    return int(B.lib().ffn_keep8_bytes(N, H, I, _dtype_code(dtype)))


def moe_keep8_bytes(N: int, H: int, I: int, E: int, k: int, dtype: torch.dtype) -> int:
    return int(B.lib().moe_keep8_bytes(N, H, I, E, k, _dtype_code(dtype)))


def _keep8(name: str, src: torch.Tensor, sizes, need: int, dst: Optional[torch.Tensor], what: str,
           events) -> torch.Tensor:
    """``src`` (a byte buffer the entry point checks) into ``dst`` of ``need`` bytes."""
    if need == 0:
        B.check(B.ERR_BAD_SHAPE, name)
    if dst is None:
        dst = torch.empty(need, dtype=torch.uint8, device=src.device)
    else:
        _buffer(dst, what, need, src.device)
    if not src.is_contiguous():
        raise ValueError("the kept or saved buffer must be contiguous")
    _call(name, src.device, events, src.data_ptr(), src.numel() * src.element_size(), *sizes,
          dst.data_ptr(), dst.numel() * dst.element_size())
    return dst


@_on_kernel_stream
def ffn_swiglu_keep8(saved: torch.Tensor, N: int, H: int, I: int, dtype: torch.dtype, *,
                     kept: Optional[torch.Tensor] = None, stream=None,
                     stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """g and u of a training forward (ffn_swiglu_fwd(..., saved=saved)) in 8
    bits: a byte buffer of ffn_keep8_bytes, after which ``saved`` is free."""
    return _keep8("ffn_swiglu_keep8", saved, (N, H, I, _code(dtype)),
                  ffn_keep8_bytes(N, H, I, dtype), kept, "kept", stage_events)


@_on_kernel_stream
def ffn_swiglu_restore8(kept: torch.Tensor, N: int, H: int, I: int, dtype: torch.dtype, *,
                        workspace: Optional[torch.Tensor] = None, stream=None,
                        stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """A backward workspace from the kept bytes, for ffn_swiglu_bwd(...,
    workspace=..., from_saved=True)."""
    return _keep8("ffn_swiglu_restore8", kept, (N, H, I, _code(dtype)),
                  int(B.lib().ffn_bwd_workspace_bytes(N, H, I, _code(dtype))), workspace,
                  "workspace", stage_events)


@_on_kernel_stream
def moe_ffn_keep8(saved: torch.Tensor, N: int, H: int, I: int, E: int, k: int,
                  dtype: torch.dtype, *, kept: Optional[torch.Tensor] = None, stream=None,
                  stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """As ffn_swiglu_keep8 for moe_ffn_fwd(..., saved=saved): the routing as it
    is, g and u in 8 bits (moe_keep8_bytes)."""
    return _keep8("moe_ffn_keep8", saved, (N, H, I, E, k, _code(dtype)),
                  moe_keep8_bytes(N, H, I, E, k, dtype), kept, "kept", stage_events)


@_on_kernel_stream
def moe_ffn_restore8(kept: torch.Tensor, N: int, H: int, I: int, E: int, k: int,
                     dtype: torch.dtype, *, workspace: Optional[torch.Tensor] = None, stream=None,
                     stage_events: Optional[B.StageEvents] = None) -> torch.Tensor:
    """A backward workspace from the kept bytes, for moe_ffn_bwd(...,
    workspace=..., from_saved=True)."""
    return _keep8("moe_ffn_restore8", kept, (N, H, I, E, k, _code(dtype)),
                  int(B.lib().moe_bwd_workspace_bytes(N, H, I, E, k, _code(dtype))), workspace,
                  "workspace", stage_events)
