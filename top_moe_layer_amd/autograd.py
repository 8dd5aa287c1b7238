"""torch.autograd bindings: the forward and backward entry points of the C ABI
as autograd Functions, so the FFN / MoE sub-layer trains inside a PyTorch
graph.  Argument marshalling only: both passes run in the library's kernels.
The backward recomputes the routing from the saved inputs; the gate/up
activations it either recomputes or, with ``keep_activations`` (the
default), takes from the buffer the training forward filled, which holds
them until the backward has run, or in 8 bits from a small buffer of their own
(``keep_activations="act8"``).  The operators of the block around them
(block.py) follow, each as one Function."""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import block, linear, ops


def _keep_mode(keep_activations) -> int:
    """0 recompute, 1 keep, 2 keep in 8 bits; 0 under no_grad (no backward)."""
    if isinstance(keep_activations, str) and keep_activations != "act8":
        raise ValueError(f"keep_activations is True, False or \"act8\", got {keep_activations!r}")
    if not torch.is_grad_enabled():
        return 0
    return 2 if keep_activations == "act8" else int(bool(keep_activations))


def _grad(t: torch.Tensor) -> torch.Tensor:
    """An upstream gradient as the kernels take it: contiguous, and 16-byte
    aligned, which a piece of a larger one (of a concatenation, say) need not be."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _SwiGLUFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, Wg, Wu, Wd, residual, keep):
        ctx.has_residual = residual is not None
        ctx.saved = saved = kept = None
        if keep and any(ctx.needs_input_grad[:4]):
            H, I = x.shape[-1], Wg.shape[0]
            N = x.numel() // H
            nb = ops.ffn_bwd_workspace_bytes(N, H, I, x.dtype)
            saved = torch.empty(max(nb, 256), dtype=torch.uint8, device=x.device)
        y = ops.ffn_swiglu_fwd(x, Wg, Wu, Wd, residual=residual, saved=saved)
        if saved is not None and keep == 2:
            kept = block.ffn_swiglu_keep8(saved, N, H, I, x.dtype)
        else:
            ctx.saved = saved
        ctx.save_for_backward(x, Wg, Wu, Wd, kept)  # released by the backward, as the inputs are
        return y

    @staticmethod
    def backward(ctx, dy):
        x, Wg, Wu, Wd, kept = ctx.saved_tensors
        saved = ctx.saved
        if kept is not None:
            H, I = x.shape[-1], Wg.shape[0]
            saved = block.ffn_swiglu_restore8(kept, x.numel() // H, H, I, x.dtype)
        g = ops.ffn_swiglu_bwd(x, Wg, Wu, Wd, _grad(dy), workspace=saved,
                               from_saved=saved is not None)
        ctx.saved = None
        return g.dx, g.dWg, g.dWu, g.dWd, (dy if ctx.has_residual else None), None


def swiglu_ffn(x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor,
               residual: Optional[torch.Tensor] = None, *,
               keep_activations=True) -> torch.Tensor:
    """Differentiable dense SwiGLU FFN: y = residual + Wd (SiLU(Wg x) * Wu x).
    ``keep_activations``: the forward keeps g, u for the backward (one backward
    workspace held from the forward to the backward) instead of the backward
    recomputing them; the results are the same bits either way.  "act8" keeps
    them in 8 bits (about 2 N I bytes held); y is the same, the gradients are
    those of the 8-bit g and u: within 2^-4 of themselves, but an element 2^-14
    and less of the largest of its 32 channels ever more coarsely, and as 0
    from about 2^-18 on."""
    return _SwiGLUFunction.apply(x, Wg, Wu, Wd, residual, _keep_mode(keep_activations))


class _MoEFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, Wr, Wg, Wu, Wd, residual, k, aux_coef, z_coef, capacity_factor,
                norm_topk_prob, keep):
        ctx.saved = saved = kept = None
        if keep and any(ctx.needs_input_grad[:5]):
            H, (E, I) = x.shape[-1], Wg.shape[:2]
            N = x.numel() // H
            nb = ops.moe_bwd_workspace_bytes(N, H, I, E, k, x.dtype)
            saved = torch.empty(max(nb, 256), dtype=torch.uint8, device=x.device)
        out = ops.moe_ffn_fwd(x, Wr, Wg, Wu, Wd, k, aux_coef, residual=residual,
                              norm_topk_prob=norm_topk_prob, z_coef=z_coef,
                              capacity_factor=capacity_factor, return_lists=False,
                              saved=saved)
        if saved is not None and keep == 2:
            kept = block.moe_ffn_keep8(saved, N, H, I, E, k, x.dtype)
        else:
            ctx.saved = saved
        ctx.save_for_backward(x, Wr, Wg, Wu, Wd, kept)
        ctx.cfg = (k, aux_coef, z_coef, capacity_factor, norm_topk_prob, residual is not None)
        z = out.z_loss if out.z_loss is not None else torch.zeros(1, dtype=torch.float32,
                                                                   device=x.device)
        ctx.mark_non_differentiable(out.topk_idx, out.alpha)
        return out.y, out.aux_loss, z, out.topk_idx, out.alpha

    @staticmethod
    def backward(ctx, dy, daux, dz, _didx, _dalpha):
        x, Wr, Wg, Wu, Wd, kept = ctx.saved_tensors
        k, aux_coef, z_coef, capacity_factor, norm, has_res = ctx.cfg
        if dy is None:
            dy = torch.zeros_like(x)
        # the loss terms' upstream gradients stay on the device (the kernel
        # reads them): no host synchronisation in the backward
        f32 = lambda t: t.reshape(-1)[:1].to(torch.float32).contiguous()
        aux_grad = f32(daux) if daux is not None else 0.0
        z_grad = f32(dz) if dz is not None else 0.0
        saved = ctx.saved
        if kept is not None:
            H, (E, I) = x.shape[-1], Wg.shape[:2]
            saved = block.moe_ffn_restore8(kept, x.numel() // H, H, I, E, k, x.dtype)
        g = ops.moe_ffn_bwd(x, Wr, Wg, Wu, Wd, _grad(dy), k, aux_coef, aux_grad=aux_grad,
                            norm_topk_prob=norm, z_coef=z_coef, z_grad=z_grad,
                            capacity_factor=capacity_factor, workspace=saved,
                            from_saved=saved is not None)
        ctx.saved = None
        return (g.dx, g.dWr, g.dWg, g.dWu, g.dWd, (dy if has_res else None),
                None, None, None, None, None, None)


def moe_ffn(x: torch.Tensor, Wr: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
            Wd: torch.Tensor, k: int, aux_coef: float, *, residual: Optional[torch.Tensor] = None,
            z_coef: float = 0.0, capacity_factor: float = 0.0, norm_topk_prob: bool = True,
            keep_activations=True):
    """Differentiable top-k MoE FFN.  Returns (y, aux_loss [1], z_loss [1],
    topk_idx, alpha); y, aux_loss and z_loss carry gradients to x and every
    weight (topk_idx and alpha are the router's choices, not differentiable).
    ``keep_activations`` as for swiglu_ffn."""
    return _MoEFunction.apply(x, Wr, Wg, Wu, Wd, residual, k, aux_coef, z_coef, capacity_factor,
                              norm_topk_prob, _keep_mode(keep_activations))


# ------------------------------------------------------------ rows by expert
class _DispatchFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, topk_idx, E, capacity_factor):
        r = block.moe_dispatch_fwd(x, topk_idx, E, capacity_factor=capacity_factor)
        ctx.shape = x.shape
        ctx.save_for_backward(r.entry_row)
        ctx.mark_non_differentiable(r.expert_offsets, r.row_entry, r.entry_row)
        return tuple(r)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs, _off, _re, _er):
        entry_row, = ctx.saved_tensors
        dx = block.moe_dispatch_bwd(_grad(dxs), entry_row)
        return dx.view(ctx.shape), None, None, None


def moe_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, E: int, *,
                 capacity_factor: float = 0.0) -> block.MoeRows:
    """Differentiable moe_dispatch_fwd: the tokens' rows by expert; gradients
    of ``xs`` go back to ``x``."""
    return block.MoeRows(*_DispatchFunction.apply(x, topk_idx, E, capacity_factor))


class _CombineFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, entry_row, alpha, residual):
        ctx.save_for_backward(ys, entry_row, alpha)
        return block.moe_combine_fwd(ys, entry_row, alpha, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, entry_row, alpha = ctx.saved_tensors
        dys = dalpha = None
        if ctx.needs_input_grad[0] or ctx.needs_input_grad[2]:
            dys, dalpha = block.moe_combine_bwd(_grad(dy), ys, entry_row, alpha)
        return dys, None, dalpha, dy if ctx.needs_input_grad[3] else None


def moe_combine(ys: torch.Tensor, entry_row: torch.Tensor, alpha: torch.Tensor,
                residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable moe_combine_fwd: gradients to ``ys``, ``alpha`` and
    ``residual``."""
    return _CombineFunction.apply(ys, entry_row, alpha, residual)


# ------------------------------------------------------------ products by expert
class _LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, expert_offsets):
        y = linear.moe_linear_fwd(x, w, expert_offsets)
        ctx.save_for_backward(x if ctx.needs_input_grad[1] else None, w, expert_offsets)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, expert_offsets = ctx.saved_tensors
        dx, dw = linear.moe_linear_bwd(_grad(dy), x, w, expert_offsets,
                                       need_dx=ctx.needs_input_grad[0],
                                       need_dw=ctx.needs_input_grad[1])
        return dx, dw, None


def moe_linear(x: torch.Tensor, w: torch.Tensor,
               expert_offsets: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable moe_linear_fwd: gradients to ``x`` and ``w``."""
    return _LinearFunction.apply(x, w, expert_offsets)


class _Mx4LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, q, scale, expert_offsets):
        ctx.save_for_backward(q, scale, expert_offsets)
        return linear.mx4_linear_fwd(x, linear.Mx4(q, scale), expert_offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        q, scale, expert_offsets = ctx.saved_tensors
        return linear.mx4_linear_bwd(_grad(dy), linear.Mx4(q, scale), expert_offsets), None, None, None


def mx4_linear(x: torch.Tensor, w: linear.Mx4,
               expert_offsets: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable mx4_linear_fwd of a plain x over frozen 4-bit matrices (as
    adapters are trained around them): gradients to ``x``."""
    return _Mx4LinearFunction.apply(x, w.q, w.scale, expert_offsets)


# ------------------------------------------------------------ norms
class _PrenormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, eps):
        n, rstd = block.block_prenorm_fwd(x, w, eps=eps)
        ctx.save_for_backward(x, w, rstd)
        return n

    @staticmethod
    @once_differentiable
    def backward(ctx, dn):
        x, w, rstd = ctx.saved_tensors
        g = block.block_prenorm_bwd(_grad(dn), x, w, rstd)
        return g.dx, g.dw, None


def block_prenorm(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable RMS norm before a block: w * x / rms(x)."""
    return _PrenormFunction.apply(x, w, eps)


class _PostnormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, residual, w, gate, next_w, residual_scale, eps):
        ctx.set_materialize_grads(False)
        o = block.block_postnorm_fwd(y, residual, w, gate=gate, next_w=next_w,
                                     residual_scale=residual_scale, eps=eps)
        ctx.scale = residual_scale
        out = o.out if next_w is not None else None  # only the next norm's gradient reads it
        ctx.save_for_backward(y, w, gate, next_w, out, o.rstd, o.next_rstd)
        return (o.out, o.n) if next_w is not None else o.out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dn=None):
        y, w, gate, next_w, out, rstd, next_rstd = ctx.saved_tensors
        if dout is None and dn is None:
            return (None,) * 7
        dout = None if dout is None else _grad(dout)  # None: the gradient of n alone
        if dn is None:  # n was not used: its norm has no gradient
            next_w = out = next_rstd = None
        else:
            dn = _grad(dn)
        g = block.block_postnorm_bwd(dout, y, w, rstd=rstd, gate=gate, dn=dn, out=out,
                                     next_w=next_w, next_rstd=next_rstd, residual_scale=ctx.scale)
        return g.dy, g.dresidual, g.dw, g.dgate, g.dnext_w, None, None


def block_postnorm(y: torch.Tensor, residual: torch.Tensor, w: Optional[torch.Tensor] = None, *,
                   gate: Optional[torch.Tensor] = None, next_w: Optional[torch.Tensor] = None,
                   residual_scale: float = 1.0, eps: float = 1e-5):
    """Differentiable block_postnorm_fwd: out = residual_scale * residual +
    gate * w * y / rms(y), and with ``next_w`` the pair (out, n) with the next
    block's norm n = next_w * out / rms(out); their gradients join in one pass."""
    return _PostnormFunction.apply(y, residual, w, gate, next_w, residual_scale, eps)


# ------------------------------------------------------------ 8-bit activations
class _SwigluAct8Function(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g, u):
        ctx.fused = u is None
        ctx.shape = g.shape
        C = g.shape[-1] // 2 if u is None else g.shape[-1]
        if u is None:
            if g.shape[-1] % 2:
                raise ValueError(f"[g | u] needs an even last dimension, got {g.shape[-1]}")
            gu = g.reshape(-1, 2 * C)
            g2, u2 = gu[:, :C], gu[:, C:]
        else:
            if u.shape != g.shape:
                raise ValueError(f"u has shape {tuple(u.shape)}, expected g's {tuple(g.shape)}")
            g2, u2 = g.reshape(-1, C), u.reshape(-1, C)
        o = block.swiglu_act8_fwd(g2, u2)
        ctx.save_for_backward(*o.g8, *o.u8)
        return o.h.view(*ctx.shape[:-1], C)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        gq, gs, uq, us = ctx.saved_tensors
        R, C = gq.shape
        dgu = torch.empty((R, 2 * C) if ctx.fused else (2, R, C), dtype=dh.dtype, device=dh.device)
        dg, du = (dgu[:, :C], dgu[:, C:]) if ctx.fused else (dgu[0], dgu[1])
        block.swiglu_act8_bwd(_grad(dh.reshape(R, C)), block.Act8(gq, gs),
                              block.Act8(uq, us), with_h=False, dg=dg, du=du)
        if ctx.fused:
            return dgu.view(ctx.shape), None
        return dg.view(ctx.shape), du.view(ctx.shape)


def swiglu_act8(g: torch.Tensor, u: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable SiLU(g) * u that keeps g and u in 8 bits for the backward
    instead of in their dtype.  g, u [..., C]; without ``u``, g [..., 2C] is one
    projection's output [g | u], and so is its gradient."""
    return _SwigluAct8Function.apply(g, u)
