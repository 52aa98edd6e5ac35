"""torch.autograd binding of libflce: per-token log-probs (and entropy) of a linear
LM head as a differentiable op, in the manner of the autograd function the
Liger-Kernel commit "native Blackwell tensor-parallel fused scaled linear
cross-entropy" lists among its code entry points ("Code entry points", PyTorch
autograd row), and the layer norm in front of it.

Argument marshalling only: the head's forward is one flce.forward call, its backward one
flce.backward call with the incoming gradients as grad_logprob / grad_entropy.  The
logits are never materialised; the backward recomputes them on the GPU.  The norm's are
flce.layer_norm_forward and flce.layer_norm_backward.  The residual block (linear, dropout) and
the log-probs read off a matrix of logits (token_logprobs) likewise make one call each way.
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


def _as_rows(t, cols):
    """t as a matrix of `cols` columns whose rows are contiguous and apart."""
    t = t.reshape(-1, cols)
    if (t.stride(1) != 1 and cols > 1) or (t.shape[0] > 1 and t.stride(0) < cols):
        t = t.contiguous()
    return t


def _as_operand(t, cols):
    """_as_rows with rows as the matrix product takes them: 16-byte aligned, at most 2^21 elements apart."""
    t = _as_rows(t, cols)
    if t.data_ptr() % 16 or (t.shape[0] > 1 and (t.stride(0) % 8 or t.stride(0) > 1 << 21)):
        t = t.clone(memory_format=torch.contiguous_format)
    return t


class FusedLinear(torch.autograd.Function):
    """y = act(x W^T + bias) + residual; keeps x, W and, with an activation, its argument in bf16."""

    @staticmethod
    def forward(ctx, x, weight, bias, activation, residual, out_dtype):
        K, N = x.shape[-1], weight.shape[0]
        X, W = _as_operand(x, K), _as_operand(weight, K)
        r = None if residual is None else _as_rows(residual, N)
        keep = activation is not None and any(ctx.needs_input_grad[:3])
        y = flce.linear_forward(X, W, bias, activation, r, out_dtype, keep)
        y, pre = y if keep else (y, None)
        ctx.save_for_backward(X, W, pre)
        ctx.cfg = (activation, x.shape, None if bias is None else bias.dtype,
                   None if residual is None else residual.dtype)
        return y.view(*x.shape[:-1], N)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        X, W, pre = ctx.saved_tensors
        activation, shape, bias_dtype, residual_dtype = ctx.cfg
        need = ctx.needs_input_grad
        dx = dw = db = None
        if need[0] or need[1] or need[2]:
            dx, dw, db = flce.linear_backward(_as_rows(dy, W.shape[0]), X, W, pre, activation, need[0], need[1],
                                              bias_dtype if need[2] else None)
        return (dx.view(shape) if need[0] else None, dw, db, None,
                dy.to(residual_dtype) if need[4] else None, None)


def linear(x, weight, bias=None, activation=None, residual=None, out_dtype=None):
    """Differentiable act(x weight^T + bias) + residual over the last axis of x, as
    flce.linear_forward: x and weight bf16, bias and residual bf16 or fp32, y bf16 (the default) or
    fp32.  residual has y's shape.  The graph keeps x and, with an activation, its argument in bf16.
    For a backward captured into a graph see layer_norm."""
    if residual is not None and residual.shape != (*x.shape[:-1], weight.shape[0]):
        raise ValueError(f"residual: expected shape {(*x.shape[:-1], weight.shape[0])}, got {tuple(residual.shape)}")
    return FusedLinear.apply(x, weight, bias, activation, residual, out_dtype)


class FusedDropout(torch.autograd.Function):
    """y = residual + dropout(x); keeps nothing but the seed."""

    @staticmethod
    def forward(ctx, x, p: float, seed, offset: int, residual, out_dtype):
        H = x.shape[-1]
        r = None if residual is None else _as_rows(residual, H)
        if isinstance(seed, torch.Tensor):
            seed = seed.clone()   # the caller may write the next one there before the backward runs
        y = flce.dropout(_as_rows(x, H), p, seed, offset, r, out_dtype)
        ctx.seed = seed
        ctx.cfg = (p, offset, x.shape, x.dtype, None if residual is None else residual.dtype)
        return y.view(x.shape)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        p, offset, shape, x_dtype, residual_dtype = ctx.cfg
        need, dx = ctx.needs_input_grad, None
        if need[0]:
            dx = flce.dropout_backward(_as_rows(dy, shape[-1]), p, ctx.seed, offset, x_dtype).view(shape)
        return dx, None, None, None, dy.to(residual_dtype) if need[4] else None, None


def dropout(x, p: float, seed, offset: int = 0, residual=None, out_dtype=None):
    """Differentiable residual + dropout(x) over x [..., H], as flce.dropout (rows are those of x as
    a matrix of H columns).  No mask is kept; a seed given as a tensor is copied.  For a backward
    captured into a graph see layer_norm."""
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual: expected shape {tuple(x.shape)}, got {tuple(residual.shape)}")
    return FusedDropout.apply(x, p, seed, offset, residual, out_dtype)


class LogitsLogprobs(torch.autograd.Function):
    """Log-probs of given tokens, entropy and alternatives of logits; keeps the logits."""

    @staticmethod
    def forward(ctx, logits, tokens, ignore_index: int, scale: float, n_top: int, compute_entropy: bool):
        r = flce.token_logprobs(logits, tokens, ignore_index, scale, n_top, compute_entropy)
        ctx.save_for_backward(logits, tokens, r.stats, r.entropy, r.top_ids)
        ctx.cfg = (int(ignore_index), float(scale))
        ctx.set_materialize_grads(False)
        if r.top_ids is not None:
            ctx.mark_non_differentiable(r.top_ids)
        ctx.mark_non_differentiable(r.stats)
        return tuple(r)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_lp, g_lse, g_ent, g_ids, g_top, g_stats):
        logits, tokens, stats, entropy, top_ids = ctx.saved_tensors
        ignore_index, scale = ctx.cfg
        f = lambda g: None if g is None else g.float().contiguous()
        d = flce.token_logprobs_backward(logits, tokens, stats, entropy, top_ids, f(g_lp), f(g_top), f(g_ent),
                                         f(g_lse), ignore_index, scale)
        return d, None, None, None, None, None


def token_logprobs(logits, tokens=None, ignore_index: int = -100, scale: float = 1.0, n_top: int = 0,
                   compute_entropy: bool = False):
    """flce.token_logprobs with gradients of logprob, lse, entropy and top_logprob with respect to
    the logits [M, V]; stats carries none.  The graph keeps the logits.  For a backward captured into
    a graph see layer_norm."""
    return flce.TokenLogprobs(*LogitsLogprobs.apply(logits, tokens, ignore_index, scale, n_top, compute_entropy))
