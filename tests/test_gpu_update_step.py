"""Several updates on one rollout, and a step on preference pairs, as a trainer calls them: the head's
log-probabilities, a loss over them, its gradients, their norm, and AdamW's step by the clipping
factor.  float32, against the same in float64: gradients within 512 * 2^-24 = 3e-5 of the largest
value of each, as in the on-policy step's test; later steps start from weights that differ by the
first one's roundings, which a factor of ten takes in."""
import pytest
import torch

import grpo_policy_loss_amd as gp
from tests import plain_ops, plain_update

pytestmark = pytest.mark.gpu
G, L, PROMPTS, D, V = 4, 8, 3, 64, 512
B = G * PROMPTS
N = B * L


def start(seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(N, D, generator=gen)
    W = 0.2 * torch.randn(V, D, generator=gen)
    g = 1 + 0.1 * torch.randn(D, generator=gen)
    y = torch.randint(0, V, (N,), generator=gen, dtype=torch.int32)
    mask = (torch.rand(N, generator=gen) < 0.8).to(torch.uint8)
    return x, g, W, y, mask, gen


def plain_lp(x, g, W, y):
    h = plain_ops.norm_fwd(x, torch.ones_like(g), None, 1e-6, False)[0] * g
    return torch.log_softmax(h @ W.t() / 0.8, 1).gather(1, y.long()[:, None])[:, 0]


def step(loss_of, plain_loss, leaves, plain_leaves, plan_of, k, tol):
    """One update of both, compared."""
    gc, Wc = leaves
    for p in leaves:
        p.grad = None
    loss = loss_of()
    loss.backward()
    grads = [gc.grad, Wc.grad]
    gplan = gp.grad_plan(grads)
    norm, scale = gp.grpo_grad_norm(gplan, max_norm=0.05)
    params, m, v = plan_of
    plan = gp.adamw_plan([p.detach() for p in params], grads, m, v)
    gp.grpo_adamw(plan, k, lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.0, grad_scale=scale)

    want = plain_loss()
    pg = torch.autograd.grad(want, plain_leaves["w"])
    assert abs(loss.item() - want.item()) <= tol * (1 + abs(want.item()))
    for got, w in zip(grads, pg):
        assert (got.cpu().double() - w).abs().max() <= tol * w.abs().max()
    n = torch.sqrt(sum(w.square().sum() for w in pg)).item()
    assert abs(norm.item() - n) <= tol * n and abs(scale.item() - min(1.0, 0.05 / (n + 1e-6))) <= tol
    for i, (w, p) in enumerate(zip(plain_leaves["w"], pg)):
        new, plain_leaves["m"][i], plain_leaves["v"][i] = plain_ops.adamw(
            w.detach(), p, plain_leaves["m"][i], plain_leaves["v"][i], k, 1e-2, (0.9, 0.99), 1e-6, 0.0, min(1.0, 0.05 / (n + 1e-6)))
        plain_leaves["w"][i] = new.requires_grad_()
    return loss.item()


def run(seed, loss_of, plain_of):
    x, g, W, y, mask, gen = start(seed)
    gc, Wc = g.clone().cuda().requires_grad_(), W.clone().cuda().requires_grad_()
    xc, yc, mc = x.cuda(), y.cuda(), mask.cuda()
    plain = dict(w=[g.double().requires_grad_(), W.double().requires_grad_()], m=[torch.zeros(D).double(), torch.zeros(V, D).double()],
                 v=[torch.zeros(D).double(), torch.zeros(V, D).double()])
    m, v = gp.adamw_moments([gc, Wc])
    lp_of = lambda: gp.grpo_logprobs(gp.grpo_norm(xc, gc, None, 1e-6), Wc, yc, opts={"temperature": 0.8})  # noqa: E731
    ours, theirs = loss_of(lp_of, mc, gen), plain_of(lambda: plain_lp(x.double(), *plain["w"], y), mask)
    for k in (1, 2, 3):
        step(ours, theirs, (gc, Wc), plain, ([gc, Wc], m, v), k, 3e-5 if k == 1 else 3e-4)


def test_several_updates_on_one_rollout():
    gen = torch.Generator().manual_seed(11)
    adv, shift, drift = torch.randn(B, generator=gen), 0.02 * torch.randn(N, generator=gen), 0.1 * torch.randn(N, generator=gen)
    x, g, W, y, mask, _ = start(1)
    old = (plain_lp(x.double(), g.double(), W.double(), y) + shift).float()
    ref = old + drift
    how = dict(beta=0.04, clip_low=0.2, clip_high=0.28)
    run(1, lambda lp_of, mc, _: lambda: gp.grpo_clip_loss(lp_of(), mc, adv.cuda(), B, L, old.cuda(), ref.cuda(), **how)[0],
        lambda lp_of, mask: lambda: differentiable_clip(lp_of(), old, ref, mask, adv))


def differentiable_clip(lp, old, ref, mask, adv):
    r = (lp - old.double()).exp()
    A = adv.double().repeat_interleave(L)
    x = ref.double() - lp
    l = -torch.minimum(r * A, r.clamp(0.8, 1.28) * A) + 0.04 * (x.exp() - x - 1)
    keep = mask != 0
    return l[keep].mean()


def test_steps_on_preference_pairs():
    x, g, W, y, mask, _ = start(2)
    ref = plain_lp(x.double(), g.double(), W.double(), y).float()
    P = B // 2

    def plain(lp, mask):
        s = torch.where(mask != 0, lp - ref.double(), 0.0).view(B, L).sum(1)
        n = mask.view(B, L).ne(0).sum(1)[0::2].clamp(min=1)
        like = torch.where(mask != 0, lp, 0.0).view(B, L).sum(1)[0::2] / n
        return (torch.nn.functional.softplus(-0.5 * (s[0::2] - s[1::2])) - 0.1 * like).mean()
    run(2, lambda lp_of, mc, _: lambda: gp.grpo_pref_loss(lp_of(), mc, P, L, ref.cuda(), beta=0.5, nll_weight=0.1)[0],
        lambda lp_of, mask: lambda: plain(lp_of(), mask))


def test_direct_calls_in_one_graph():
    """Log-probabilities, loss, gradients, norm and optimizer captured together and replayed."""
    x, g, W, y, mask, gen = start(3)
    H, Wc, yc, mc = x.cuda(), W.cuda(), y.cuda(), mask.cuda()
    adv, old = torch.randn(B, generator=gen).cuda(), gp.grpo_logprobs_fwd(H, Wc, yc)[0].clone()
    dW = torch.zeros(V, D, device="cuda")
    m, v = gp.adamw_moments([Wc])
    plan, gplan, at = gp.adamw_plan([Wc], [dW], m, v), gp.grad_plan([dW]), torch.ones(1, dtype=torch.int64, device="cuda")

    def once():
        dW.zero_()
        lp, lse = gp.grpo_logprobs_fwd(H, Wc, yc)
        loss, stats, w = gp.grpo_clip_loss_fwd(lp, mc, adv, B, L, old_lp=old)
        grad = gp.grpo_clip_loss_bwd(lp, mc, adv, w, B, L, old_lp=old)
        gp.grpo_logprobs_bwd(H, Wc, yc, lp, lse, grad, dW=dW)
        norm, scale = gp.grpo_grad_norm(gplan, 0.1)
        gp.grpo_adamw(plan, at, lr=1e-2, grad_scale=scale)
        at.add_(1)
        return loss, stats, norm
    state = [Wc, m[0], v[0], at]
    keep = [t.clone() for t in state]
    wants = []
    for _ in range(4):
        wants.append([t.clone() for t in (*once(), *state)])
    for t, s in zip(state, keep):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = once()
    for t, s in zip(state, keep):
        t.copy_(s)
    for want in wants:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*outs, *state), want))
