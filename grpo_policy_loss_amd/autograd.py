"""torch.autograd wrappers over the C ABI, for use inside a PyTorch training step:
the loss as a differentiable function of the hidden states H and the LM head W, and
the norm in front of it as one of its input, weight and bias.

The loss's forward is grpo_loss_fwd; the backward is grpo_loss_bwd with the upstream
gradient of the loss as its grad_loss (Unsloth docs, "Offloading activations
for log softmax": the backward recomputes the chunk's logits instead of
keeping them).  Marshalling only: both passes run in libgrpo.so.
"""
from __future__ import annotations

import torch

from ._lib import grpo_loss_bwd, grpo_loss_fwd
from ._ops import NORM_LAYER, NORM_RMS, grpo_norm_bwd, grpo_norm_fwd


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
        if torch.cuda.is_current_stream_capturing():
            # The node that adds up a leaf's gradient is made by the first graph that uses the leaf,
            # is shared by all later ones while any of them lives, and runs on the stream on which it
            # was made.  A captured backward that reaches one of an eager graph joins that stream,
            # which is not captured: the capture fails and the process ends.  Whether such a graph
            # lives cannot be seen from here.
            raise RuntimeError("grpo_norm's backward cannot be captured: call grpo_norm_bwd, which can")
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
