"""The clipped loss's sums: policy terms are summed in float64 from the first token on, so that large ones that
cancel leave the small ones, and terms near float32's largest number do not overflow together."""
import math

import pytest
import torch

import grpo_policy_loss_amd as gp

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def forward(L, lp, old=None, ref=None, adv=None, **how):
    lp, old, ref, adv = (None if x is None else torch.tensor(x).repeat(-(-L // len(x)))[:L].cuda() for x in (lp, old, ref, adv))
    mask = torch.ones(L, dtype=torch.uint8, device="cuda")
    if adv is None:
        adv = torch.ones(1, device="cuda")
    return gp.grpo_clip_loss_fwd(lp, mask, adv, 1, L, old_lp=old, ref_lp=ref, clip_low=0.0, clip_high=0.0, **how)[:2]


@pytest.mark.parametrize("L", [4, 8, 1024, 3000, 20480])
@pytest.mark.parametrize("aggregation", [gp.AGG_TOKEN_MEAN, gp.AGG_SEQUENCE_MEAN])
def test_large_advantages_that_cancel(L, aggregation):
    """Whole numbers below 2^53: the sum -L / 2 is exact, and so is its mean."""
    loss, _ = forward(L, [-1.0], adv=[1e8, 1.0, -1e8, 1.0], aggregation=aggregation)
    assert loss.item() == -0.5


@pytest.mark.parametrize("L", [4, 1024, 3000])
def test_cancelling_terms_of_moved_tokens(L):
    """Ratios e^0.75 for all: products of 24 and 27 bits are exact in float64, so what is left is the
    ratio's own error, (|D| + 4) half steps, and the result's rounding."""
    loss, _ = forward(L, [-1.0], old=[-1.75], adv=[1e8, 1.0, -1e8, 1.0])
    want = -0.5 * math.exp(0.75)
    assert abs(loss.item() - want) <= (0.75 + 4 + 1) * U * abs(want)


@pytest.mark.parametrize("L", [4, 1024, 3000])
def test_terms_near_the_largest_number(L):
    """e^88.5 is 2.7e38: four of them overflow float32, their mean does not."""
    big = math.exp(88.5)
    loss, stats = forward(L, [-88.5], ref=[0.0], beta=0.01)
    assert abs(stats[0].item() - big) <= (88.5 + 8) * U * big
    assert abs(loss.item() - 0.01 * big) <= (88.5 + 8) * U * 0.01 * big
    loss, stats = forward(L, [0.0], old=[-88.5], adv=[1.0])
    assert abs(stats[3].item() - big) <= (88.5 + 8) * U * big
    assert abs(loss.item() + big) <= (88.5 + 8) * U * big
