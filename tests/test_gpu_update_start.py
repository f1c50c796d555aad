"""The first step of an update on a rollout, as README's example makes it: the weights are those that
sampled, and with one logit transform for both policies no ratio is clipped or away from 1."""
import pytest
import torch

import grpo_policy_loss_amd as gp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ratio", [gp.RATIO_TOKEN, gp.RATIO_SEQUENCE])
def test_unchanged_weights_have_a_ratio_of_one(t, ratio):
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    B, L, d, V = 6, 20, 64, 700
    g, W = (1 + 0.1 * rnd(d)).to(t).requires_grad_(), (rnd(V, d) / 4).to(t).requires_grad_()
    y = torch.randint(0, V, (B * L,), generator=gen, dtype=torch.int32).cuda()
    mask = (torch.rand(B * L, generator=gen) < 0.7).to(torch.uint8).cuda()
    H = gp.grpo_norm(rnd(B * L, d).to(t), g, eps=1e-6)
    ref, adv = rnd(B * L) - 6, rnd(B)

    opts = {"temperature": 0.9}
    old = gp.grpo_logprobs_fwd(H, W, y, opts=opts)[0]
    lp = gp.grpo_logprobs(H, W, y, opts=opts)
    loss, stats = gp.grpo_clip_loss(lp, mask, adv, B, L, old, ref, beta=0.04, clip_low=0.2, clip_high=0.28, ratio=ratio)
    loss.backward()
    assert stats[0].item() > 0 and stats[1:].tolist() == [0.0, 0.0, 0.0]
    assert loss.isfinite() and g.grad.any() and W.grad.any()
    # of another transform they are other distributions: tokens are clipped though nothing was learnt
    other = gp.grpo_logprobs_fwd(H, W, y)[0]
    stats = gp.grpo_clip_loss_fwd(lp.detach(), mask, adv, B, L, other, clip_low=0.01, clip_high=0.01, ratio=ratio)[1]
    assert stats[1] + stats[2] > 0.2 and stats[3] > 0
