"""torch.autograd binding of libflce: per-token log-probs (and entropy) of a linear
LM head as a differentiable op, in the manner of the autograd function the
Liger-Kernel commit "native Blackwell tensor-parallel fused scaled linear
cross-entropy" lists among its code entry points ("Code entry points", PyTorch
autograd row), and the layer norm in front of it.

Argument marshalling only: the head's forward is one flce.forward call, its backward one
flce.backward call with the incoming gradients as grad_logprob / grad_entropy.  The
logits are never materialised; the backward recomputes them on the GPU.  The norm's are
flce.layer_norm_forward and flce.layer_norm_backward.
"""
from __future__ import annotations

import torch

from . import flce


class FusedLinearLogprob(torch.autograd.Function):
    """(logprob, entropy) = f(X, W) for targets; entropy only with compute_entropy."""

    @staticmethod
    def forward(ctx, X, W, targets, ignore_index: int, scale: float, compute_entropy: bool):
        lp, lse, ent = flce.forward(X, W, targets, ignore_index, scale, compute_entropy)
        ctx.save_for_backward(X, W, targets, lse, ent)
        ctx.cfg = (int(ignore_index), float(scale))
        # an unused output's gradient arrives as None rather than a tensor of zeros
        ctx.set_materialize_grads(False)
        if compute_entropy:
            return lp, ent
        return lp

    @staticmethod
    def backward(ctx, g_lp, g_ent=None):
        X, W, targets, lse, ent = ctx.saved_tensors
        ignore_index, scale = ctx.cfg
        glp = None if g_lp is None else g_lp.float().contiguous()
        gent = None if g_ent is None else g_ent.float().contiguous()
        dX = dW = None
        if ctx.needs_input_grad[0] or ctx.needs_input_grad[1]:
            dX, dW = flce.backward(X, W, targets, lse, ent if gent is not None else None, glp,
                                   gent, ignore_index, scale)
        return (dX if ctx.needs_input_grad[0] else None,
                dW if ctx.needs_input_grad[1] else None, None, None, None, None)


def linear_logprob(X, W, targets, ignore_index: int = -100, scale: float = 1.0,
                   compute_entropy: bool = False):
    """Differentiable per-token log-probs of targets under softmax(scale X W^T), and the
    per-token entropy when compute_entropy is set.  X [M, H], W [V, H] bf16 on the GPU,
    targets [M] int64; rows whose target is ignore_index or outside [0, V) give 0."""
    return FusedLinearLogprob.apply(X, W, targets, ignore_index, scale, compute_entropy)


class FusedLayerNorm(torch.autograd.Function):
    """y = f(x, weight, bias) over the last axis; keeps x, or an 8-bit copy of it."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps: float, out_dtype, checkpoint):
        rows = x.reshape(-1, x.shape[-1])
        if rows.stride(1) != 1 or (rows.shape[0] > 1 and rows.stride(0) < rows.shape[1]):
            rows = rows.contiguous()
        y, mean, rstd, *kept = flce.layer_norm_forward(rows, weight, bias, eps, out_dtype, checkpoint)
        if checkpoint is None:
            ctx.save_for_backward(mean, rstd, weight, rows)
        else:
            ctx.save_for_backward(mean, rstd, weight, kept[0].codes, kept[0].scales)
        ctx.cfg = (checkpoint, x.shape, x.dtype, None if bias is None else bias.dtype)
        return y.view(x.shape)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        mean, rstd, weight, *saved = ctx.saved_tensors
        checkpoint, shape, x_dtype, bias_dtype = ctx.cfg
        x = saved[0] if checkpoint is None else flce.MXTensor(*saved, checkpoint, shape[-1])
        dy = dy.reshape(-1, shape[-1])
        if dy.stride(1) != 1 or (dy.shape[0] > 1 and dy.stride(0) < dy.shape[1]):
            dy = dy.contiguous()
        need = ctx.needs_input_grad
        dx, dw, db = flce.layer_norm_backward(
            dy, x, mean, rstd, weight, dx_dtype=x_dtype, need_params=need[1] or need[2],
            param_dtype=bias_dtype if weight is None else None)
        return (dx.view(shape) if need[0] else None, dw if need[1] else None,
                db if need[2] else None, None, None, None)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out_dtype=None, checkpoint=None):
    """Differentiable layer norm over the last axis of x (bf16 or fp32 on the GPU), in 32
    bits; y has out_dtype (x's by default).  With checkpoint "mxfp8" or "mxint8" the graph
    keeps an 8-bit copy of x instead of x: y is unchanged, and the gradients are those of the
    copy's values (about half a step of the format from x: 2^-4 relative for "mxfp8", 2^-7 of
    the largest of 32 neighbours for "mxint8").  To capture forward and backward in a graph,
    first let go of eager results that lead back to the same leaves: torch would make the
    captured backward wait for their stream."""
    return FusedLayerNorm.apply(x, weight, bias, eps, out_dtype, checkpoint)
