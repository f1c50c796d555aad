"""The operators around the loss in plain float64 torch on the CPU, from their
formulas (the tests' oracle for them; nothing here is shared with the library)."""
import numpy as np
import torch


def _sqrt(x):
    """Correctly rounded, which torch's own on the CPU is not everywhere (some hosts give 1/2 for the
    root of the float64 below 1/4)."""
    return torch.from_numpy(np.sqrt(x.numpy()))


def norm_fwd(x, w, b, eps, layer):
    """(y, mean or None, rstd) of the rows of x."""
    x, w = x.double(), w.double()
    mean = x.mean(1) if layer else torch.zeros(x.shape[0], dtype=torch.float64)
    rstd = 1 / ((x - mean[:, None]).square().mean(1) + eps).sqrt()
    y = (x - mean[:, None]) * rstd[:, None] * w
    return (y if b is None else y + b.double()), mean, rstd


def norm_bwd(dy, x, w, mean, rstd, layer):
    """(dx, dw, db) with the given statistics."""
    dy, x, w, r = dy.double(), x.double(), w.double(), rstd.double()[:, None]
    xh = (x - (mean.double()[:, None] if layer else 0)) * r
    g = dy * w
    dx = r * (g - (g.mean(1, keepdim=True) if layer else 0) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def moment_codes(x, squared):
    """(codes, scales) of a moment in 8 bits, blocks of 256."""
    n = x.numel()
    b = torch.zeros(-(-n // 256) * 256, dtype=torch.float64)
    b[:n] = x.double().flatten()
    b = b.view(b.numel() // 256, 256)
    a = b.abs().amax(1).float()
    bad = ~b.isfinite().all(1)
    q = torch.where((a > 0)[:, None], b.abs() / a.double()[:, None], 0.0)
    if squared:
        c = (255 * _sqrt(_sqrt(q)) + 0.5).floor().clamp(max=255)
        c = torch.where(b > 0, c.clamp(min=1), c)
        c = torch.where(a[:, None] == 0, 0.0, c)
    else:
        c = (127 * _sqrt(q) + 0.5).floor().clamp(max=127) * b.sign()
    c[bad] = 0
    a = torch.where(bad, float("nan"), a)
    return c.flatten()[:n].to(torch.uint8 if squared else torch.int8), a


def moment_values(codes, scales):
    c = codes.double().flatten()
    c = (c / 255) ** 4 if codes.dtype == torch.uint8 else c.sign() * (c / 127) ** 2
    return c * scales.double().repeat_interleave(256)[:c.numel()]


def adamw(w, g, m, v, step, lr, betas, eps, wd, scale=1.0):
    """(w, m, v) after the step, all float64."""
    w, g, m, v = w.double(), g.double() * scale, m.double(), v.double()
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    mh, vh = m / (1 - betas[0] ** step), v / (1 - betas[1] ** step)
    return w - lr * wd * w - lr * mh / (vh.sqrt() + eps), m, v


def sample(x, u, T=1.0, k=0, p=1.0, min_p=0.0):
    """(token, lp) of one row of logits; (-1, nan) where nothing can be drawn."""
    x = x.double()
    T = 1.0 if T == 0 else T
    if x.isnan().any() or (x == float("inf")).any() or x.max() == float("-inf") or not 0 < T < float("inf"):
        return -1, float("nan")
    z = x / T
    e = (z - z.max()).exp()
    order = sorted(range(x.numel()), key=lambda i: (-x[i].item(), i)) if x.numel() < 300 else \
        x.sort(descending=True, stable=True).indices.tolist()
    if 0 < k < len(order):
        order = order[:k]
    if 0 < p < 1:
        w = e[order]
        up = w.cumsum(0)
        before = torch.cat([torch.zeros(1, dtype=torch.float64), up[:-1]])
        order = [i for i, keep in zip(order, (before < p * up[-1]).tolist()) if keep]
    keep = torch.zeros_like(e)
    keep[order] = 1
    if min_p > 0:
        keep *= e >= min(min_p, 1.0)
    run = (e * keep).cumsum(0)
    hit = (run > min(max(u, 0.0), 1.0) * run[-1]).nonzero()
    token = hit[0].item() if len(hit) else (e * keep).nonzero()[-1].item()
    return token, (z[token] - z.max() - e.sum().log()).item()
