"""The operators around the loss in one step, as a trainer calls them: logits of the
normed hidden states, sampled tokens, the loss on them, its gradients through the norm,
and an AdamW step of the norm's weight and the head.  Checked against the same step in
float64, with the tokens that were drawn.

The step is float32 (d 64, V 512, 96 tokens), so each stage adds relative errors of some
K 2^-24 with K the length of its sums (64 to 512): 512 * 2^-24 = 3e-5 of the largest value
of each gradient bounds them together."""
import pytest
import torch

import grpo_policy_loss_amd as gp
from tests import plain_ops

pytestmark = pytest.mark.gpu
G, L, PROMPTS, D, V = 4, 8, 3, 64, 512
B = G * PROMPTS
N = B * L
BETA, T = 0.04, 0.8


def plain_loss(x, g, W, y, mask, adv, ref):
    h = plain_ops.norm_fwd(x, torch.ones_like(g), None, 1e-6, False)[0] * g
    lp = torch.log_softmax(h @ W.t() / T, 1).gather(1, y[:, None])[:, 0]
    r = ref - lp
    kl = r.exp() - r - 1
    ratio = (lp - lp.detach()).exp()
    loss = -(ratio * adv.repeat_interleave(L) - BETA * kl)
    return (loss * mask).sum() / mask.sum(), lp


def test_rollout_and_training_step():
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(N, D, generator=gen) * (0.5 + torch.rand(N, 1, generator=gen))
    g = 1 + 0.1 * torch.randn(D, generator=gen)
    W = 0.2 * torch.randn(V, D, generator=gen)
    u, rewards = torch.rand(N, generator=gen), torch.rand(B, generator=gen)
    mask = (torch.rand(N, generator=gen) < 0.8).to(torch.uint8)
    xc, gc, Wc = (v.clone().cuda().requires_grad_() for v in (x, g, W))
    opts = {"temperature": T}

    # the rollout
    h = gp.grpo_norm(xc, gc, None, 1e-6)
    token, lp_drawn = gp.grpo_sample(gp.grpo_gemm_nt(h.detach(), Wc.detach()), u.cuda(), temperature=T)
    want, _ = zip(*(plain_ops.sample(row, float(v), T=T) for row, v in
                    zip((h.detach().cpu().double() @ W.double().t()), u)))
    # the logits here are float32 products: a token may differ where u is that near a border
    assert (token.cpu() == torch.tensor(want)).float().mean() > 0.98

    # the step
    adv = gp.grpo_advantages(rewards.cuda(), G)
    ref = (lp_drawn + 0.05 * torch.randn(N, generator=gen).cuda()).contiguous()
    loss, lp, kl = gp.grpo_loss(h, Wc, token, mask.cuda(), adv, ref, B, L, BETA, 64, opts)
    assert (lp - lp_drawn).abs().max() <= 1e-5 * lp.abs().max()
    loss.backward()
    leaves = [v.double().requires_grad_() for v in (x, g, W)]
    want_loss, want_lp = plain_loss(*leaves, token.cpu().long(), mask.double(), adv.cpu().double(), ref.cpu().double())
    want_loss.backward()
    assert abs(loss.item() - want_loss.item()) <= 3e-5 * (1 + abs(want_loss.item()))
    for got, leaf in zip((xc, gc, Wc), leaves):
        far = (got.grad.cpu().double() - leaf.grad).abs().max()
        assert far <= 3e-5 * leaf.grad.abs().max(), far

    # the optimizer: norm weight and head together
    params, grads = [gc.detach(), Wc.detach()], [gc.grad, Wc.grad]
    m, v = gp.adamw_moments(params)
    plan = gp.adamw_plan(params, grads, m, v)
    hyper = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
    clip = (1.0 / torch.linalg.vector_norm(torch.cat([t.flatten() for t in grads]))).clamp(max=1.0).reshape(1).contiguous()
    before = [p.cpu().clone() for p in params]
    gp.grpo_adamw(plan, 1, grad_scale=clip, **hyper)
    for p, old, grad in zip(params, before, grads):
        w, _, _ = plain_ops.adamw(old, grad.cpu(), torch.zeros_like(old), torch.zeros_like(old), 1, 1e-2, (0.9, 0.99), 1e-6, 0.1, clip.item())
        # 4 roundings of the weight, and 32 of a step of at most lr (with zero moments m / sqrt v is
        # at most 1)
        assert ((p.cpu().double() - w).abs() <= 2.0 ** -24 * (4 * old.abs() + 32 * 1e-2)).all()
    # the parameters that autograd knows have moved
    assert not torch.equal(gc.detach().cpu(), g) and not torch.equal(Wc.detach().cpu(), W)


def test_step_without_autograd_in_eight_bits():
    """The C ABI's order of calls with preallocated buffers and bfloat16 weights, captured
    where the calls allow it: norm forward and backward and the optimizer replay."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, dy = rnd(256, D).bfloat16(), rnd(256, D).bfloat16()
    weight = (1 + 0.1 * rnd(D)).bfloat16()
    master = weight.float()
    dw, m, v = torch.zeros(D, device="cuda"), *gp.adamw_moments([weight], 8)
    plan = gp.adamw_plan([weight], [dw], m, v, master=[master])
    step = torch.ones(1, dtype=torch.int64, device="cuda")

    def once():
        dw.zero_()
        _, _, rstd = gp.grpo_norm_fwd(x, weight)
        gp.grpo_norm_bwd(dy, x, weight, None, rstd, dweight=dw)
        gp.grpo_adamw(plan, step, lr=1e-2)
        step.add_(1)
    keep = [t.clone() for t in (weight, master, m[0].codes, m[0].scales, v[0].codes, v[0].scales, step)]
    for _ in range(4):
        once()
    torch.cuda.synchronize()
    want = [t.clone() for t in (weight, master, m[0].codes, v[0].codes)]
    for t, k in zip((weight, master, m[0].codes, m[0].scales, v[0].codes, v[0].scales, step), keep):
        t.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for t, k in zip((weight, master, m[0].codes, m[0].scales, v[0].codes, v[0].scales, step), keep):
        t.copy_(k)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
    for a, b in zip((weight, master, m[0].codes, v[0].codes), want):
        assert torch.equal(a, b)
