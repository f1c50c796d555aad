"""The operators around the loss in plain float64 torch on the CPU, from their
formulas (the tests' oracle for them; nothing here is shared with the library)."""
import torch


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
        c = (255 * q ** 0.25 + 0.5).floor().clamp(max=255)
        c = torch.where(b > 0, c.clamp(min=1), c)
        c = torch.where(a[:, None] == 0, 0.0, c)
    else:
        c = (127 * q.sqrt() + 0.5).floor().clamp(max=127) * b.sign()
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
