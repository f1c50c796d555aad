"""The gradients of tests/plain_update.py against differences of its losses, in float64 on the CPU."""
import pytest
import torch

from tests import plain_update


def difference(f, x, grad):
    """|central difference - gradient| along a direction, h = 2^-17: the curvature's h^2 (2^-34) and
    the loss's 2^-53 / h = 2^-36 are both below 10^-9 of values near 1."""
    v = torch.randn(x.numel(), generator=torch.Generator().manual_seed(5), dtype=torch.float64).view(x.shape)
    h = 2.0 ** -17
    slope = (f(x + h * v) - f(x - h * v)) / (2 * h)
    want = (grad * v).sum()
    assert abs(slope - want) <= 1e-8 * (1 + abs(want)), (slope, want)


def inputs(B, L, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    lp = -rnd(B * L).abs()
    mask = (torch.rand(B * L, generator=g) < 0.7).to(torch.uint8)
    mask[:L] = 0
    return lp, lp + 0.2 * rnd(B * L), lp + 0.3 * rnd(B * L), mask, rnd(B)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("sequence", [False, True])
@pytest.mark.parametrize("seq_mean", [False, True])
def test_clip_loss(kind, sequence, seq_mean):
    lp, old, ref, mask, adv = inputs(4, 9)
    how = dict(beta=0.3, low=0.1, high=0.15, dual=1.3, sequence=sequence, kind=kind, seq_mean=seq_mean)
    f = lambda x: plain_update.clip_loss(x, old, ref, mask, adv, 4, 9, **how)  # noqa: E731
    difference(lambda x: f(x)["loss"], lp, f(lp)["grad"])


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("averaged", [False, True])
def test_pref_loss(kind, averaged):
    lp, _, ref, mask, _ = inputs(6, 7, 1)
    how = dict(beta=0.4, kind=kind, averaged=averaged, smoothing=0.2 if kind == 0 else 0.0, margin=0.1, nll=0.3)
    f = lambda x: plain_update.pref_loss(x, ref, mask, 3, 7, **how)  # noqa: E731
    difference(lambda x: f(x)["loss"], lp, f(lp)["grad"])


@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_logprobs(cap):
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    H, W, up = rnd(5, 6), rnd(11, 6), rnd(5)
    up[2] = 0
    y = torch.tensor([0, 10, 3, 3, 7])
    f = lambda H, W: plain_update.logprobs(H, W, y, up, k=0.8, cap=cap)  # noqa: E731
    difference(lambda x: (f(x, W)["lp"] * up).sum(), H, f(H, W)["dH"])
    difference(lambda x: (f(H, x)["lp"] * up).sum(), W, f(H, W)["dW"])
