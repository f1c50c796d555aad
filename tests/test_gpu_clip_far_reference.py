"""The forward KL estimator, x e^x - e^x + 1 with x = ref_lp - lp, of tokens that the reference thinks far less
likely: it tends to 1 and must not carry the rounding of x."""
import math

import pytest
import torch

import grpo_policy_loss_amd as gp

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def one(x, lp, L):
    """kl of tokens that are all alike: the mean over L of them, and the slope of beta kl."""
    p = torch.full((L,), lp, device="cuda")
    ref = torch.full((L,), x + lp, device="cuda")
    x = (ref.double() - p.double())[0].item()
    mask, adv = torch.ones(L, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
    how = dict(ref_lp=ref, beta=1.0, kl_estimator=gp.KL_FORWARD)
    loss, stats, w = gp.grpo_clip_loss_fwd(p, mask, adv, 1, L, **how)
    return x, loss.item(), stats[0].item(), gp.grpo_clip_loss_bwd(p, mask, adv, w, 1, L, **how)


@pytest.mark.parametrize("L", [1, 5, 1500])
@pytest.mark.parametrize("x", [-3e8, -123456.789, -1e4, -1234.567, -150.0, -100.0, -50.0, -20.0, -9.0, -3.0, -1.0, -0.51, -0.49, -0.01, 0.0, 0.3, 0.6,
                               2.0, 20.0])
def test_far_and_near(x, L):
    """e^x is off by |x| + 4 half steps, the products and differences by one each of their terms, and near
    0 the series by 16 of the value."""
    x, loss, kl, grad = one(x, -0.25, L)
    e = math.exp(x)
    want = x * e - math.expm1(x)
    tol = U * ((abs(x) + 1) * e * (abs(x) + 4) + abs(math.expm1(x)) + 4 * want) if abs(x) >= 0.5 else 24 * U * want
    assert abs(kl - want) <= tol + 1e-38 and abs(loss - want) <= tol + 1e-38
    slope = -x * e / L
    assert ((grad.double() - slope).abs() <= (abs(x) + 8) * U * abs(slope) + 1e-38).all()
