"""torch.autograd wrappers over the C ABI, for use inside a PyTorch training step:
the loss as a differentiable function of the hidden states H and the LM head W, and
the norm in front of it as one of its input, weight and bias; the log-probabilities as
a function of H and W, and the losses over given log-probabilities.

The loss's forward is grpo_loss_fwd; the backward is grpo_loss_bwd with the upstream
gradient of the loss as its grad_loss (Unsloth docs, "Offloading activations
for log softmax": the backward recomputes the chunk's logits instead of
keeping them).  Marshalling only: both passes run in libgrpo.so.
"""
from __future__ import annotations

import torch

from ._lib import AGG_TOKEN_MEAN, KL_REVERSE, _opts, grpo_loss_bwd, grpo_loss_fwd
from ._losses import (PREF_SIGMOID, RATIO_TOKEN, _logprobs_bwd, _logprobs_saved_fwd,
                      grpo_clip_loss_bwd, grpo_clip_loss_fwd, grpo_pref_loss_bwd,
                      grpo_pref_loss_fwd)
from ._ops import NORM_LAYER, NORM_RMS, _on, grpo_norm_bwd, grpo_norm_fwd


class _GrpoLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, y, mask, adv, ref_lp, B, L, beta, chunk, opts):
        loss, lp, kl, lse = grpo_loss_fwd(H, W, y, mask, adv, ref_lp, B, L, beta, chunk,
                                          opts=opts)
        ctx.save_for_backward(H, W, y, mask, adv, ref_lp, lp, lse)
        ctx.args = (B, L, beta, chunk, opts)
        ctx.mark_non_differentiable(lp, kl)
        return loss.reshape(()), lp, kl

    @staticmethod
    def backward(ctx, g_loss, g_lp, g_kl):
        H, W, y, mask, adv, ref_lp, lp, lse = ctx.saved_tensors
        B, L, beta, chunk, opts = ctx.args
        # the C ABI takes the upstream scalar by value: one host read of it
        g = 0.0 if g_loss is None else float(g_loss)
        need_h, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if not (need_h or need_w) or g == 0.0:
            return (torch.zeros_like(H) if need_h else None,
                    torch.zeros_like(W) if need_w else None) + (None,) * 9
        dH, dW = grpo_loss_bwd(H, W, y, mask, adv, ref_lp, lp, lse, B, L, beta, g, chunk,
                               opts=opts)
        return (dH if need_h else None,
                (dW if W.dtype == torch.float32 else dW.to(W.dtype)) if need_w else None) \
            + (None,) * 9


def grpo_loss(H, W, y, mask, adv, ref_lp, B: int, L: int, beta: float = 0.04,
              chunk: int = 4096, opts=None):
    """(loss, lp, kl): loss is a 0-d float32 tensor differentiable with respect to H
    and W; lp and kl ([N] float32) carry no gradient.  Arguments as for
    grpo_loss_fwd.  W's gradient is formed in float32 and returned in W's dtype: a
    bfloat16 W receives it rounded to bfloat16 (grpo_loss_bwd with a float32 dW
    accumulator keeps it in float32).  The backward reads the upstream gradient of
    the loss on the host (one synchronisation)."""
    return _GrpoLoss.apply(H, W, y, mask, adv, ref_lp, B, L, beta, chunk, opts)


def _refuse_capture(name, direct):
    """The node that adds up a leaf's gradient is made by the first graph that uses the leaf,
    is shared by all later ones while any of them lives, and runs on the stream on which it
    was made.  A captured backward that reaches one of an eager graph joins that stream,
    which is not captured: the capture fails and the process ends.  Whether such a graph
    lives cannot be seen from here."""
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{name}'s backward cannot be captured: call {direct}, which can")


class _GrpoNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, weight, bias, eps, kind):
        Y, mean, rstd = grpo_norm_fwd(X, weight, bias, eps, kind)
        ctx.save_for_backward(X, weight, rstd, *([mean] if kind == NORM_LAYER else []))
        ctx.kind = kind
        ctx.shapes = weight.shape, None if bias is None else bias.shape
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        _refuse_capture("grpo_norm", "grpo_norm_bwd")
        X, weight, rstd, *mean = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        # an upstream gradient may be a broadcast view (that of a sum is)
        dX, dw, db = grpo_norm_bwd(dY.contiguous(), X, weight, mean[0] if mean else None, rstd,
                                   ctx.kind, bias=need_b)
        w_shape, b_shape = ctx.shapes
        return (dX if need_x else None, dw.to(weight.dtype).view(w_shape) if need_w else None,
                db.to(weight.dtype).view(b_shape) if need_b else None, None, None)


def grpo_norm(X, weight, bias=None, eps: float = 1e-5, kind: int = NORM_RMS):
    """The norm of the rows of X [rows, cols], differentiable (once) with respect to X,
    weight and bias.  Arguments as for grpo_norm_fwd.  The gradients of weight and bias
    are formed in float32 and returned in the weight's type (grpo_norm_bwd with float32
    accumulators keeps them in float32).  The backward raises while its stream is captured
    into a graph, since an eager graph of the same leaves that is still alive would end the
    process there; grpo_norm_fwd and grpo_norm_bwd can be captured."""
    return _GrpoNorm.apply(X, weight, bias, eps, kind)


class _GrpoLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, y, chunk, opts):
        lp, lse, ctx.args = _logprobs_saved_fwd(H, W, y, chunk, _opts(opts))
        ctx.save_for_backward(H, W, y, lp, lse)
        return lp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_lp):
        _refuse_capture("grpo_logprobs", "grpo_logprobs_bwd")
        H, W, y, lp, lse = ctx.saved_tensors
        chunk, opts, sizes = ctx.args
        need_h, need_w = ctx.needs_input_grad[:2]
        grad_lp = grad_lp.contiguous()       # it may be a broadcast view (that of a sum is)
        dH, dW = _logprobs_bwd(H, W, y, lp, lse, grad_lp, chunk, None, None, None, opts, need_h, need_w,
                               sizes, _on(H, grad_lp), like_w=True)
        return dH, dW if dW is None or dW.dtype == W.dtype else dW.to(W.dtype), None, None, None


def grpo_logprobs(H, W, y, chunk: int = 4096, opts=None):
    """The log-probabilities [N] float32 of y, differentiable (once) with respect to H and W:
    for any loss over them.  Arguments as for grpo_logprobs_fwd.  W's gradient is summed in
    float32 and returned in W's type (grpo_logprobs_bwd with a float32 dW accumulator keeps it
    in float32); tokens whose gradient is 0 have no part in it, whatever their hidden states
    hold.  The backward raises while its stream is captured into a graph, as grpo_norm's does."""
    return _GrpoLogprobs.apply(H, W, y, chunk, opts)


class _GrpoClipLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, lp, mask, adv, B, L, old_lp, ref_lp, how):
        loss, stats, weights = grpo_clip_loss_fwd(lp, mask, adv, B, L, old_lp, ref_lp, **how)
        ctx.save_for_backward(lp, mask, adv, weights, old_lp, ref_lp)
        ctx.args = B, L, how
        ctx.mark_non_differentiable(stats)
        return loss.reshape(()), stats

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_loss, g_stats):
        _refuse_capture("grpo_clip_loss", "grpo_clip_loss_bwd")
        lp, mask, adv, weights, old_lp, ref_lp = ctx.saved_tensors
        B, L, how = ctx.args
        g = grpo_clip_loss_bwd(lp, mask, adv, weights, B, L, old_lp, ref_lp, grad_loss=g_loss, **how)
        return (g.view(lp.shape),) + (None,) * 7


def grpo_clip_loss(lp, mask, adv, B: int, L: int, old_lp=None, ref_lp=None, beta: float = 0.0,
                   clip_low: float = 0.2, clip_high: float = 0.2, clip_dual: float = 0.0,
                   ratio: int = RATIO_TOKEN, kl_estimator: int = KL_REVERSE,
                   aggregation: int = AGG_TOKEN_MEAN):
    """(loss, stats): the clipped policy loss as a 0-d float32 tensor, differentiable (once) with
    respect to lp, and its statistics [4], which carry no gradient; adv, old_lp and ref_lp are
    constants.  Arguments as for grpo_clip_loss_fwd.  The backward raises while its stream is
    captured into a graph, as grpo_norm's does."""
    how = dict(beta=beta, clip_low=clip_low, clip_high=clip_high, clip_dual=clip_dual, ratio=ratio,
               kl_estimator=kl_estimator, aggregation=aggregation)
    return _GrpoClipLoss.apply(lp, mask, adv, B, L, old_lp, ref_lp, how)


class _GrpoPrefLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, lp, mask, P, L, ref_lp, how):
        loss, rewards, weights = grpo_pref_loss_fwd(lp, mask, P, L, ref_lp, **how)
        ctx.save_for_backward(mask, weights)
        ctx.args = P, L, lp.shape
        ctx.mark_non_differentiable(rewards)
        return loss.reshape(()), rewards

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_loss, g_rewards):
        _refuse_capture("grpo_pref_loss", "grpo_pref_loss_bwd")
        mask, weights = ctx.saved_tensors
        P, L, shape = ctx.args
        return (grpo_pref_loss_bwd(mask, weights, P, L, grad_loss=g_loss).view(shape),) + (None,) * 5


def grpo_pref_loss(lp, mask, P: int, L: int, ref_lp=None, beta: float = 0.1,
                   kind: int = PREF_SIGMOID, length_mean: bool = False,
                   label_smoothing: float = 0.0, margin: float = 0.0, nll_weight: float = 0.0):
    """(loss, rewards): the preference loss as a 0-d float32 tensor, differentiable (once) with
    respect to lp, and the sequences' rewards [2 P], which carry no gradient; ref_lp is a
    constant.  Arguments as for grpo_pref_loss_fwd.  The backward raises while its stream is
    captured into a graph, as grpo_norm's does."""
    how = dict(beta=beta, kind=kind, length_mean=length_mean, label_smoothing=label_smoothing,
               margin=margin, nll_weight=nll_weight)
    return _GrpoPrefLoss.apply(lp, mask, P, L, ref_lp, how)
