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
