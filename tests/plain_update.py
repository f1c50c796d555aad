"""The losses over given log-probabilities, their way back to the head and the gradients' norm, in
plain float64 torch on the CPU, from their formulas (the tests' oracle for them; nothing here is
shared with the library).  Tokens are taken one sequence after the other, masked ones left out."""
import math

import torch

U = 2.0 ** -24      # half a step of float32, relative


def kl(kind, x, lp):
    """(value, slope in lp) of the estimators of grpo_opts, x = ref_lp - lp."""
    e = x.exp()
    if kind == 0:
        return x.expm1() - x, -x.expm1()
    if kind == 1:
        return e * x - x.expm1(), -x * e
    return lp.exp() * (x.expm1() - x), -x * lp.exp()


def kl_error(kind, x, lp):
    """Bounds of the float32 errors of value and slope, in units of U.  x is off by |x|.  Below 1/2
    the series and its products cost 8 relative roundings, and x's own |x| |e^x - 1| is below 2.6
    values; above, e^x has 2 and the differences one each of terms up to e^x + |x| + 1.  The slope of
    the first likewise; products with x or e^lp (|lp| + 4 relative roundings) add theirs."""
    v, s = (t.abs() for t in kl(kind, x, lp))
    wide = 8 * (x.exp() * (1 + x.abs()) ** 2 + x.abs() + 1)
    small = x.abs() < 0.5
    q = lp.exp() if kind == 2 else torch.ones_like(x)
    more = (lp.abs() + 8) if kind == 2 else 8
    value = torch.where(small, 16 * v, wide * q) + more * v
    slope = torch.where(small, 8 * s + 4 * x.abs() * q, wide * q) + more * s
    return value, slope


def clip_loss(lp, old, ref, mask, adv, B, L, beta=0.0, low=0.0, high=0.0, dual=0.0, sequence=False,
              kind=0, seq_mean=False, g=1.0):
    """A dict of loss, stats, grad and bounds of the float32 errors of each."""
    wide = lambda v: None if v is None else v.detach().cpu().double().flatten()  # noqa: E731
    lp, old, ref, adv = wide(lp), wide(old), wide(ref), wide(adv)
    keep = mask.cpu().bool().flatten()
    n = max(1, int(keep.sum()))
    grad, tol = torch.zeros(B * L, dtype=torch.float64), torch.zeros(B * L, dtype=torch.float64)
    loss = loss_tol = 0.0
    stats, stats_tol = torch.zeros(4, dtype=torch.float64), torch.zeros(4, dtype=torch.float64)
    for b in range(B):
        at = torch.arange(b * L, (b + 1) * L)[keep[b * L:(b + 1) * L]]
        if not len(at):
            continue
        w = 1 / (B * len(at)) if seq_mean else 1 / n
        p = lp[at]
        D = p - old[at] if old is not None else torch.zeros_like(p)
        if sequence:
            D = D.mean().expand(len(at))
        A = adv[at] if adv.numel() == B * L and adv.numel() != B else adv[b].expand(len(at))
        r = D.exp()
        above = (A >= 0) & (r > 1 + high) if high else torch.zeros_like(A, dtype=torch.bool)
        below = (A < 0) & (r < 1 - low) if low else torch.zeros_like(above)
        far = (A < 0) & (r > dual) if dual else torch.zeros_like(above)
        s = r.masked_fill(above, 1 + high).masked_fill(below, 1 - low).masked_fill(far, dual)
        l, slope = -A * s, torch.where(above | below | far, 0.0, -A * r)
        # the ratio: (float)D costs |D|, the exponential 4, products and sums 8
        l_tol, slope_tol = l.abs() * (D.abs() + 12), slope.abs() * (D.abs() + 12)
        if ref is not None:
            x = ref[at] - p
            v, sl = kl(kind, x, p)
            ve, se = kl_error(kind, x, p)
            l, slope = l + beta * v, slope + beta * sl
            l_tol, slope_tol = l_tol + abs(beta) * (ve + 4 * v.abs()), slope_tol + abs(beta) * (se + 4 * sl.abs())
            stats[0] += v.sum() / n
            stats_tol[0] += (ve + 4 * v).sum() / n
        excess = r - 1 - D
        stats[1] += below.sum() / n
        stats[2] += (above | far).sum() / n
        stats[3] += excess.sum() / n
        stats_tol[3] += (kl_error(0, D, p)[0] + 4 * excess).sum() / n
        loss += (w * l).sum()
        loss_tol += (w * (l_tol + 4 * l.abs())).sum()
        grad[at] = g * w * slope
        tol[at] = abs(g) * w * (slope_tol + 8 * slope.abs())
    return {"loss": loss, "loss_tol": U * (loss_tol + 2 * abs(loss)) + 1e-38, "stats": stats,
            "stats_tol": U * (stats_tol + 4 * stats.abs()) + 1e-38, "grad": grad, "grad_tol": U * tol + 1e-38}


def pref_loss(lp, ref, mask, P, L, beta=0.1, kind=0, averaged=False, smoothing=0.0, margin=0.0, nll=0.0, g=1.0):
    """A dict of loss, rewards, grad and bounds of the float32 errors of each."""
    lp = lp.detach().cpu().double().flatten()
    r = lp if ref is None else lp - ref.cpu().double().flatten()
    keep = mask.cpu().bool().flatten()
    s, like, count = [], [], []
    for b in range(2 * P):
        at = torch.arange(b * L, (b + 1) * L)[keep[b * L:(b + 1) * L]]
        count.append(max(1, len(at)))
        s.append(r[at].sum() / (count[-1] if averaged else 1))
        like.append(lp[at].sum() / count[-1])
    s, like, count = torch.stack(s), torch.stack(like), torch.tensor(count, dtype=torch.float64)
    h = s[0::2] - s[1::2]
    x = beta * h - margin
    if kind == 0:
        lo, hi = torch.logaddexp(torch.zeros_like(x), -x), torch.logaddexp(torch.zeros_like(x), x)
        each = (1 - smoothing) * lo + smoothing * hi
        slope = beta * (smoothing * torch.sigmoid(x) - (1 - smoothing) * torch.sigmoid(-x))
        # softplus and sigmoid in float32 from a float64 x: e^-|x| and log1p or a quotient, 8 roundings
        each_tol = 10 * each
        slope_tol = 10 * beta * (smoothing * torch.sigmoid(x) + (1 - smoothing) * torch.sigmoid(-x))
    elif kind == 1:
        each, slope = (1 - x).clamp(min=0), torch.where(x < 1, -beta, 0.0).double()
        each_tol, slope_tol = each, slope.abs()
    else:
        each, slope = (h - margin - 1 / (2 * beta)) ** 2, 2 * (h - margin - 1 / (2 * beta))
        each_tol, slope_tol = each, slope.abs()
    weight, weight_tol = torch.zeros(2 * P, dtype=torch.float64), torch.zeros(2 * P, dtype=torch.float64)
    for k, sign in ((0, 1.0), (1, -1.0)):
        per = count[k::2] if averaged else 1.0
        weight[k::2] = sign * slope / P / per
        weight_tol[k::2] = slope_tol / P / per
    each = each - nll * like[0::2]
    weight[0::2] -= nll / count[0::2] / P
    weight_tol += 4 * weight.abs()
    of = torch.arange(2 * P).repeat_interleave(L)
    grad, tol = (torch.where(keep, v[of], 0.0) for v in (g * weight, abs(g) * weight_tol))
    loss = each.mean()
    return {"loss": loss, "loss_tol": U * (each_tol.mean() + 2 * loss.abs()) + 1e-38,
            "rewards": beta * s, "rewards_tol": U * 2 * (beta * s).abs() + 1e-38, "grad": grad, "grad_tol": U * tol + 1e-38}


def logprobs(H, W, y, g, k=1.0, cap=0.0, half=U):
    """lp, dH and dW of logits k (h . w), capped by cap tanh(. / cap) first where cap is not 0, and
    bounds of their errors: products of K terms in float32, dZ stored with `half` steps (2^-8 for
    bfloat16) and dH rounded so once more."""
    H, W, g = H.detach().cpu().double(), W.detach().cpu().double(), g.cpu().double()
    y = y.cpu().long()
    rows = torch.arange(len(y))
    raw, size = H @ W.t(), H.abs() @ W.abs().t()
    z, slope = raw * k, torch.full_like(raw, k)
    if cap:
        t = torch.tanh(raw / cap)
        z, slope = k * cap * t, k * (1 - t * t)
    lse = z.logsumexp(1)
    lp = z[rows, y] - lse
    # a logit's error, absolute: its product's, the transform's few roundings (and the hyperbolic
    # tangent's 2^-20 of the cap)
    ez = (k * (H.shape[1] + 8) * U * size + 8 * U * z.abs() + (k * cap * 2.0 ** -20 if cap else 0)).amax(1)
    lp_tol = 2 * ez + U * (16 + 4 * lse.abs() + 4 * lp.abs())
    dz = -(z - lse[:, None]).exp() * g[:, None] * slope
    # exp's argument carries the logit's and lse's errors; the target's 1 - p comes from lp
    wide = dz.abs() * (2 * ez + lp_tol + 16 * U * (1 + lse.abs()))[:, None]
    dz[rows, y] = -torch.expm1(lp) * g * slope[rows, y]
    wide[rows, y] = (lp.exp() * lp_tol + 8 * U) * (g * slope[rows, y]).abs()
    if cap:
        wide += dz.abs() * 2.0 ** -17 + (g[:, None] * (z - lse[:, None]).exp()).abs() * k * 2.0 ** -19
        wide[rows, y] += g.abs() * k * 2.0 ** -19
    dead = g == 0
    dz[dead], wide[dead] = 0.0, 0.0
    wide += half * dz.abs()
    dH, dW = dz @ W, dz.t() @ H
    V, N = W.shape[0], len(y)
    dH_tol = wide @ W.abs() + (V + 8) * U * (dz.abs() @ W.abs()) + half * dH.abs()
    dW_tol = wide.t() @ H.abs() + (N + 8) * U * (dz.abs().t() @ H.abs())
    return {"lp": lp, "lp_tol": lp_tol, "dH": dH, "dH_tol": dH_tol + 1e-38, "dW": dW, "dW_tol": dW_tol + 1e-38}


def grad_norm(grads, biggest=False):
    if biggest:
        return max([float(x.double().abs().max()) for x in grads if x.numel()] or [0.0])
    return math.sqrt(sum(float(x.cpu().double().square().sum()) for x in grads))
