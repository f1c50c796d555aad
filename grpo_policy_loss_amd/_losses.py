"""ctypes binding of the losses over given log-probabilities (include/grpo.h): the
log-probabilities with their gradient, the clipped policy loss and the preference loss.

Argument marshalling only, as in _lib.  Every call checks that its tensors share
one GPU and runs on that GPU's current torch stream, whichever device is current.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import (AGG_TOKEN_MEAN, GRPO_F32, GRPO_OP_LOGPROBS_BWD, GRPO_OP_LOGPROBS_FWD, KL_REVERSE,
                   ClipOpts, PrefOpts, _arg, _check, _dt, _matrix, _opts, _ptr, auto_chunk,
                   grpo_workspace_bytes, lib)
from ._ops import _on, _workspace

# grpo_ratio and grpo_pref_kind
RATIO_TOKEN, RATIO_SEQUENCE = 0, 1
PREF_SIGMOID, PREF_HINGE, PREF_SQUARE = 0, 1, 2


# ---------------------------------------------------------------- log-probabilities
def _head(H, W, y):
    N, d = _matrix(H, "H")
    dt = _dt(H)
    V = _matrix(W, "W")[0]
    _arg(W, "W", dtype=H.dtype, shape=(V, d))
    _arg(y, "y", dtype=torch.int32, numel=N)
    return N, d, V, dt


def _lse_size(N, dt):
    return 2 * N if dt == GRPO_F32 else N


@functools.lru_cache(maxsize=256)
def _head_bytes(op, N, d, V, dt, chunk):
    need = grpo_workspace_bytes(op, N, d, V, dt, chunk)
    if need == 0:
        _check("grpo_workspace_bytes", -1)
    return need


def _logprobs_saved_fwd(H, W, y, chunk, opts):
    """The forward for autograd: (lp, lse, (chunk, opts, sizes)).  A small workspace lies behind
    lse in one tensor, since each allocation costs a small call some 4 us in all."""
    sizes = N, d, V, dt = _head(H, W, y)
    ctx, stream = _on(H, W, y)
    dev = H.device
    with ctx:
        if chunk == 0:
            chunk = auto_chunk(1, N, d, V, dt)
        need = _head_bytes(GRPO_OP_LOGPROBS_FWD, N, d, V, dt, chunk)
        at = -(-4 * _lse_size(N, dt) // 256) * 256
        lp = torch.empty(N, dtype=torch.float32, device=dev)
        lse = torch.empty((at + (need if need <= 1 << 20 else 0)) // 4, dtype=torch.float32, device=dev)
        if need <= 1 << 20:
            ws = lse.data_ptr() + at
        else:
            apart = torch.empty(need, dtype=torch.uint8, device=dev)
            ws = apart.data_ptr()
        _check("grpo_logprobs_fwd", lib().grpo_logprobs_fwd(
            H.data_ptr(), W.data_ptr(), y.data_ptr(), N, d, V, dt, chunk, opts, lp.data_ptr(),
            lse.data_ptr(), ws, need, stream))
    return lp, lse, (chunk, opts, sizes)


def _logprobs_bwd(H, W, y, lp, lse, grad_lp, chunk, dW, dH, workspace, opts, need_h, need_w, sizes, on,
                  like_w=False):
    """The call itself, of tensors that were checked: (dH, dW).  like_w: a dW that is made is of
    W's type where one chunk takes all tokens."""
    N, d, V, dt = sizes
    ctx, stream = on
    dev = H.device
    accumulate = int(need_w and dW is not None)
    with ctx:
        if chunk == 0:
            chunk = auto_chunk(1, N, d, V, dt)
        ws = _workspace(_head_bytes(GRPO_OP_LOGPROBS_BWD, N, d, V, dt, chunk), dev, workspace)
        if not need_h:
            dH = None
        elif dH is None:
            dH = torch.empty(N, d, dtype=H.dtype, device=dev)
        dw_type = GRPO_F32
        if not need_w:
            dW = None
        elif dW is None:
            like_w = like_w and N <= chunk
            dW = torch.empty(V, d, dtype=W.dtype if like_w else torch.float32, device=dev)
            dw_type = dt if like_w else GRPO_F32
        _check("grpo_logprobs_bwd", lib().grpo_logprobs_bwd(
            H.data_ptr(), W.data_ptr(), y.data_ptr(), lp.data_ptr(), lse.data_ptr(),
            grad_lp.data_ptr(), N, d, V, dt, chunk, opts, accumulate, dw_type, _ptr(dH), _ptr(dW),
            ws.data_ptr(), ws.numel(), stream))
    return dH, dW


def grpo_logprobs_fwd(H, W, y, chunk: int = 4096, workspace=None, opts=None):
    """(lp [N], lse), float32: the log-probability of y under softmax of the logits of H [N, d]
    (float32 or bfloat16) and W [V, d], and the log-sum-exp that the backward takes ([N]; for
    float32 [2 N], its rounding behind it).  `opts` and chunk as for grpo_loss_fwd; of the
    options the logit transform counts."""
    N, d, V, dt = _head(H, W, y)
    ctx, stream = _on(*(t for t in (H, W, y, workspace) if t is not None))
    with ctx:
        if chunk == 0:
            chunk = auto_chunk(1, N, d, V, dt)
        ws = _workspace(_head_bytes(GRPO_OP_LOGPROBS_FWD, N, d, V, dt, chunk), H.device, workspace)
        lp = torch.empty(N, dtype=torch.float32, device=H.device)
        lse = torch.empty(_lse_size(N, dt), dtype=torch.float32, device=H.device)
        _check("grpo_logprobs_fwd", lib().grpo_logprobs_fwd(
            _ptr(H), _ptr(W), _ptr(y), N, d, V, dt, chunk, _opts(opts), _ptr(lp), _ptr(lse), _ptr(ws),
            ws.numel(), stream))
    return lp, lse


def grpo_logprobs_bwd(H, W, y, lp, lse, grad_lp, chunk: int = 4096, dW=None, dH=None,
                      workspace=None, opts=None, need_h: bool = True, need_w: bool = True):
    """(dH [N, d] in H's type, dW [V, d] float32) of a loss whose gradient with respect to
    lp is grad_lp [N] float32.  Tokens with a gradient of 0 have no part in it: their rows of dH
    are 0.  dW is accumulated into when given.  need_h or need_w false: that one is not
    formed, and None.  lp, lse and `opts` are the forward's."""
    sizes = N, d, V, dt = _head(H, W, y)
    for t, name, n in ((lp, "lp", N), (lse, "lse", _lse_size(N, dt)), (grad_lp, "grad_lp", N)):
        _arg(t, name, dtype=torch.float32, numel=n)
    if not (need_h or need_w):
        raise ValueError("one of need_h and need_w must be true")
    if dH is not None:
        _arg(dH, "dH", dtype=H.dtype, shape=(N, d))
    if dW is not None:
        _arg(dW, "dW", dtype=torch.float32, shape=(V, d))
    on = _on(*(t for t in (H, W, y, lp, lse, grad_lp, dH, dW, workspace) if t is not None))
    return _logprobs_bwd(H, W, y, lp, lse, grad_lp, chunk, dW, dH, workspace, _opts(opts), need_h, need_w,
                         sizes, on)


# ---------------------------------------------------------------- clipped policy loss
@functools.lru_cache(maxsize=256)
def _clip_bytes(B, L):
    need = int(lib().grpo_clip_loss_workspace_bytes(B, L))
    if need == 0:
        _check("grpo_clip_loss_workspace_bytes", -1)
    return need


@functools.lru_cache(maxsize=256)
def _clip_opts(*fields):
    return ctypes.pointer(ClipOpts(*fields))


def _clip_args(lp, mask, adv, B, L, old_lp, ref_lp, beta, clip_low, clip_high, clip_dual, ratio,
               kl_estimator, aggregation):
    """The tensors there are, and the options."""
    if B < 1 or L < 1:
        raise ValueError(f"B and L must be positive, got {B} and {L}")
    N = B * L
    ts = [_arg(lp, "lp", dtype=torch.float32, numel=N), _arg(mask, "mask", dtype=torch.uint8, numel=N)]
    _arg(adv, "adv", dtype=torch.float32)
    if adv.numel() != B and adv.numel() != N:
        raise ValueError(f"adv must have {B} elements (one a sequence) or {N} (one a token), got {adv.numel()}")
    ts.append(adv)
    for t, name in ((old_lp, "old_lp"), (ref_lp, "ref_lp")):
        if t is not None:
            ts.append(_arg(t, name, dtype=torch.float32, numel=N))
    return ts, _clip_opts(float(clip_low), float(clip_high), float(clip_dual), float(beta), int(ratio),
                          int(kl_estimator), int(aggregation), int(adv.numel() != B))


def grpo_clip_loss_fwd(lp, mask, adv, B: int, L: int, old_lp=None, ref_lp=None, beta: float = 0.0,
                       clip_low: float = 0.2, clip_high: float = 0.2, clip_dual: float = 0.0,
                       ratio: int = RATIO_TOKEN, kl_estimator: int = KL_REVERSE,
                       aggregation: int = AGG_TOKEN_MEAN, workspace=None):
    """(loss [1], stats [4], weights) of the clipped policy loss of lp [B * L] float32 (the
    policy's log-probabilities) against old_lp (the sampling policy's; None: lp's own values),
    with adv [B] (one a sequence) or [B * L] (one a token) and the KL term beta kl(ref_lp - lp)
    where beta is not 0; all three under the same logit transform.  The ratio is clipped to [1 - clip_low, 1 + clip_high], and for negative
    advantages to clip_dual from above; 0 switches each off.  stats: the means over the unmasked
    tokens of kl, of being clipped from below and from above, and of r - 1 - log r.  weights
    [2 B + 1] is what grpo_clip_loss_bwd takes.  See grpo_clip_loss_fwd in include/grpo.h."""
    ts, opts = _clip_args(lp, mask, adv, B, L, old_lp, ref_lp, beta, clip_low, clip_high, clip_dual,
                          ratio, kl_estimator, aggregation)
    need = _clip_bytes(B, L)
    if workspace is not None:
        ts.append(_workspace(need, lp.device, workspace))
    ctx, stream = _on(*ts)
    dev = lp.device
    with ctx:
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        stats = torch.empty(4, dtype=torch.float32, device=dev)
        weights = torch.empty(2 * B + 1, dtype=torch.float32, device=dev)
        ws = _workspace(need, dev, workspace)
        _check("grpo_clip_loss_fwd", lib().grpo_clip_loss_fwd(
            lp.data_ptr(), _ptr(old_lp), _ptr(ref_lp), mask.data_ptr(), adv.data_ptr(), B, L, opts,
            loss.data_ptr(), stats.data_ptr(), weights.data_ptr(), ws.data_ptr(), ws.numel(), stream))
    return loss, stats, weights


def grpo_clip_loss_bwd(lp, mask, adv, weights, B: int, L: int, old_lp=None, ref_lp=None,
                       beta: float = 0.0, clip_low: float = 0.2, clip_high: float = 0.2,
                       clip_dual: float = 0.0, ratio: int = RATIO_TOKEN,
                       kl_estimator: int = KL_REVERSE, aggregation: int = AGG_TOKEN_MEAN,
                       grad_loss=None, out=None):
    """grad_lp [B * L] float32, the gradient of grpo_clip_loss_fwd's loss with respect to lp
    (0 where masked), times grad_loss (a float32 tensor of one element; None: 1).  weights is
    the forward's, and so are the other arguments."""
    ts, opts = _clip_args(lp, mask, adv, B, L, old_lp, ref_lp, beta, clip_low, clip_high, clip_dual,
                          ratio, kl_estimator, aggregation)
    ts.append(_arg(weights, "weights", dtype=torch.float32, numel=2 * B + 1))
    if grad_loss is not None:
        ts.append(_arg(grad_loss, "grad_loss", dtype=torch.float32, numel=1))
    if out is not None:
        ts.append(_arg(out, "out", dtype=torch.float32, numel=B * L))
    ctx, stream = _on(*ts)
    with ctx:
        out = torch.empty(B * L, dtype=torch.float32, device=lp.device) if out is None else out
        _check("grpo_clip_loss_bwd", lib().grpo_clip_loss_bwd(
            lp.data_ptr(), _ptr(old_lp), _ptr(ref_lp), mask.data_ptr(), adv.data_ptr(),
            weights.data_ptr(), _ptr(grad_loss), B, L, opts, out.data_ptr(), stream))
    return out


# ---------------------------------------------------------------- preference loss
@functools.lru_cache(maxsize=256)
def _pref_bytes(P, L):
    need = int(lib().grpo_pref_loss_workspace_bytes(P, L))
    if need == 0:
        _check("grpo_pref_loss_workspace_bytes", -1)
    return need


@functools.lru_cache(maxsize=256)
def _pref_opts(*fields):
    return ctypes.pointer(PrefOpts(*fields))


def grpo_pref_loss_fwd(lp, mask, P: int, L: int, ref_lp=None, beta: float = 0.1,
                       kind: int = PREF_SIGMOID, length_mean: bool = False,
                       label_smoothing: float = 0.0, margin: float = 0.0, nll_weight: float = 0.0,
                       workspace=None):
    """(loss [1], rewards [2 P], weights [2 P]) of the preference loss over P pairs of sequences
    of padded length L: lp [2 P * L] float32, sequence 2p the chosen one of pair p and 2p + 1 the
    rejected one.  rewards are beta times the sequences' log ratios (their sums, or means with
    length_mean) to ref_lp (None: none is subtracted).  weights is what grpo_pref_loss_bwd
    takes.  See grpo_pref_loss_fwd in include/grpo.h."""
    if P < 1 or L < 1:
        raise ValueError(f"P and L must be positive, got {P} and {L}")
    N = 2 * P * L
    ts = [_arg(lp, "lp", dtype=torch.float32, numel=N), _arg(mask, "mask", dtype=torch.uint8, numel=N)]
    if ref_lp is not None:
        ts.append(_arg(ref_lp, "ref_lp", dtype=torch.float32, numel=N))
    need = _pref_bytes(P, L)
    if workspace is not None:
        ts.append(_workspace(need, lp.device, workspace))
    opts = _pref_opts(float(beta), float(label_smoothing), float(margin), float(nll_weight), int(kind),
                      int(length_mean))
    ctx, stream = _on(*ts)
    dev = lp.device
    with ctx:
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        rewards = torch.empty(2 * P, dtype=torch.float32, device=dev)
        weights = torch.empty(2 * P, dtype=torch.float32, device=dev)
        ws = _workspace(need, dev, workspace)
        _check("grpo_pref_loss_fwd", lib().grpo_pref_loss_fwd(
            lp.data_ptr(), _ptr(ref_lp), mask.data_ptr(), P, L, opts, loss.data_ptr(),
            rewards.data_ptr(), weights.data_ptr(), ws.data_ptr(), ws.numel(), stream))
    return loss, rewards, weights


def grpo_pref_loss_bwd(mask, weights, P: int, L: int, grad_loss=None, out=None):
    """grad_lp [2 P * L] float32, the gradient of grpo_pref_loss_fwd's loss with respect to lp
    (0 where masked), times grad_loss (a float32 tensor of one element; None: 1)."""
    if P < 1 or L < 1:
        raise ValueError(f"P and L must be positive, got {P} and {L}")
    N = 2 * P * L
    ts = [_arg(mask, "mask", dtype=torch.uint8, numel=N),
          _arg(weights, "weights", dtype=torch.float32, numel=2 * P)]
    if grad_loss is not None:
        ts.append(_arg(grad_loss, "grad_loss", dtype=torch.float32, numel=1))
    if out is not None:
        ts.append(_arg(out, "out", dtype=torch.float32, numel=N))
    ctx, stream = _on(*ts)
    with ctx:
        out = torch.empty(N, dtype=torch.float32, device=mask.device) if out is None else out
        _check("grpo_pref_loss_bwd", lib().grpo_pref_loss_bwd(
            mask.data_ptr(), weights.data_ptr(), _ptr(grad_loss), P, L, out.data_ptr(), stream))
    return out
