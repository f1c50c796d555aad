"""The preference loss on the GPU against the formulas in float64, within the bounds of the float32
errors that tests/plain_update.py counts."""
import math

import pytest
import torch

import grpo_policy_loss_amd as gp
from tests import plain_update

pytestmark = pytest.mark.gpu


def inputs(P, L, seed=0, garbage=True, empty=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    N = 2 * P * L
    lp = -rnd(N).abs()
    mask = torch.zeros(2 * P, L, dtype=torch.uint8)
    for b in range(2 * P):
        mask[b, int(torch.randint(0, L, (1,), generator=g)):] = 1 + b % 3
    if empty and P > 1:
        mask[1], mask[2], mask[3] = 0, 0, 0       # a rejected one, and a whole pair
    mask = mask.view(-1)
    i = dict(lp=lp, ref=lp + 0.2 * rnd(N), mask=mask)
    if garbage:
        i["lp"] = torch.where(mask == 0, torch.tensor(math.nan), lp)
        i["ref"] = torch.where(mask == 0, torch.tensor(-math.inf), i["ref"])
    return i


NAMES = dict(averaged="length_mean", smoothing="label_smoothing", nll="nll_weight")


def run(i, P, L, g=None, ref=True, **how):
    d = {k: v.cuda() for k, v in i.items()}
    kw = {NAMES.get(k, k): v for k, v in how.items()}
    loss, rewards, w = gp.grpo_pref_loss_fwd(d["lp"], d["mask"], P, L, ref_lp=d["ref"] if ref else None, **kw)
    up = None if g is None else torch.full((1,), g, device="cuda")
    return loss, rewards, gp.grpo_pref_loss_bwd(d["mask"], w, P, L, grad_loss=up)


def check(i, P, L, g=None, ref=True, **how):
    got = [t.cpu().double() for t in run(i, P, L, g, ref, **how)]
    want = plain_update.pref_loss(i["lp"], i["ref"] if ref else None, i["mask"], P, L, g=1.0 if g is None else g, **how)
    for name, x in zip(("loss", "rewards", "grad"), got):
        over = (x - want[name]).abs() - want[name + "_tol"]
        assert (over <= 0).all(), (name, over.max(), x.flatten()[over.argmax()], want[name].flatten()[over.argmax()])
    assert not got[2][i["mask"] == 0].any()


@pytest.mark.parametrize("P,L", [(1, 1), (3, 1), (2, 2), (5, 3), (4, 5), (1, 64), (9, 63), (2, 257), (70, 300), (3, 1024), (2, 1025),
                                 (1, 9001), (5, 5000), (1200, 9), (600, 65)])
@pytest.mark.parametrize("averaged", [False, True])
def test_lengths(P, L, averaged):
    i = inputs(P, L, seed=P + L)
    check(i, P, L, averaged=averaged)
    check(i, P, L, averaged=averaged, ref=False, nll=0.3, margin=0.2, smoothing=0.1)


@pytest.mark.parametrize("L", [40, 1300])
@pytest.mark.parametrize("how", [dict(kind=0), dict(kind=0, smoothing=0.3), dict(kind=0, margin=-0.5, nll=1.5), dict(kind=1), dict(kind=1, margin=0.4),
                                 dict(kind=2), dict(kind=2, margin=0.1, nll=0.2)])
def test_kinds(L, how):
    for averaged in (False, True):
        for ref in (False, True):
            check(inputs(6, L, seed=1), 6, L, g=0.37, beta=0.25, averaged=averaged, ref=ref, **how)


def test_far_apart():
    """Log ratios of hundreds and thousands: neither exponential overflows, and a sure pair has a loss."""
    for s in (1.0, 30.0, 300.0, 5000.0):
        for sign in (1, -1):
            i = dict(lp=torch.tensor([0.0, sign * s]), ref=torch.tensor([0.0, 0.0]), mask=torch.ones(2, dtype=torch.uint8))
            for kind in (0, 1, 2):
                check(i, 1, 1, beta=0.3, kind=kind)
            check(i, 1, 1, beta=0.3, smoothing=0.2)


@pytest.mark.parametrize("L", [30, 1100])
def test_a_nan_in_use_is_seen(L):
    for kind in (0, 1, 2):
        for where in ("lp", "ref"):
            i = inputs(3, L, garbage=False, empty=False)
            i["mask"].fill_(1)
            i[where][2 * L + 5] = math.nan
            loss, rewards, grad = run(i, 3, L, kind=kind)
            assert math.isnan(loss.item()) and rewards[2].isnan() and not rewards[[0, 1, 3, 4, 5]].isnan().any()
            assert grad[2 * L:4 * L].isnan().all() and not grad[:2 * L].isnan().any() and not grad[4 * L:].isnan().any()


def test_nothing_unmasked():
    for P, L in ((3, 10), (2, 2000)):
        i = inputs(P, L)
        i["mask"].zero_()
        i["lp"].fill_(math.nan)
        loss, rewards, grad = run(i, P, L, nll=1.0, averaged=True)
        assert abs(loss.item() - math.log(2)) <= 4 * plain_update.U and not rewards.any() and not grad.any()


def test_gradient_against_differences():
    """As the clipped loss's: h |v| = 2^-7 of a direction with entries up to 1, sums of up to 300 of them
    times beta 0.02, so that the third derivative adds less than (300 * 0.02 / 128)^2 / 6 < 4e-4."""
    P, L = 3, 300
    i = inputs(P, L, garbage=False)
    for how in (dict(), dict(smoothing=0.2, nll=0.4), dict(kind=2, averaged=True)):
        how = dict(beta=0.02 if not how.get("kind") else 0.5) | how
        grad = run(i, P, L, **how)[2].cpu()
        v = grad / grad.abs().max()
        h = 2.0 ** -7
        up, down = (run(i | {"lp": i["lp"] + s * h * v}, P, L, **how)[0].double().item() for s in (1, -1))
        slope, want = (up - down) / (2 * h), (grad.double() * v.double()).sum().item()
        assert abs(slope - want) <= 4e-4 * abs(want) + 2.0 ** -22 * max(abs(up), abs(down)) / h


def test_bitwise_the_same_on_another_stream_and_when_captured():
    for P, L in ((200, 100), (2, 7001)):
        i = {k: v.cuda() for k, v in inputs(P, L).items()}
        out = {}

        def once():
            out["loss"], out["rewards"], w = gp.grpo_pref_loss_fwd(i["lp"], i["mask"], P, L, ref_lp=i["ref"], nll_weight=0.1)
            out["grad"] = gp.grpo_pref_loss_bwd(i["mask"], w, P, L)
        once()
        first = dict(out)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            once()
        side.synchronize()
        assert all(torch.equal(first[k], out[k]) for k in out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            once()
        held = dict(out)
        for k in range(4):
            i["ref"].add_(0.02)
            graph.replay()
            torch.cuda.synchronize()
            once()
            assert all(torch.equal(held[n], out[n]) for n in out)


def test_any_alignment_and_neighbours():
    for P, L in ((3, 37), (1, 2049)):
        i = inputs(P, L)
        N = 2 * P * L
        d = {}
        for k, v in i.items():
            flat = torch.empty(N + 3, dtype=v.dtype, device="cuda")
            flat[3:] = v.cuda()
            d[k] = flat[3:]
        loss, rewards, w = gp.grpo_pref_loss_fwd(d["lp"], d["mask"], P, L, ref_lp=d["ref"])
        flat = torch.full((N + 9,), 7.0, device="cuda")
        gp.grpo_pref_loss_bwd(d["mask"], w, P, L, out=flat[1:N + 1])
        for x, y in zip((loss, rewards, flat[1:N + 1]), run(i, P, L)):
            assert torch.equal(x, y)
        assert flat[0] == 7 and (flat[N + 1:] == 7).all()


def test_autograd():
    P, L = 2, 20
    i = {k: v.cuda() for k, v in inputs(P, L, garbage=False).items()}
    lp = i["lp"].clone().requires_grad_()
    loss, rewards = gp.grpo_pref_loss(lp, i["mask"], P, L, i["ref"], beta=0.2, nll_weight=0.1)
    assert loss.dim() == 0 and not rewards.requires_grad
    (2 * loss).backward()
    _, _, w = gp.grpo_pref_loss_fwd(i["lp"], i["mask"], P, L, i["ref"], beta=0.2, nll_weight=0.1)
    assert torch.equal(lp.grad, gp.grpo_pref_loss_bwd(i["mask"], w, P, L, grad_loss=torch.full((1,), 2.0, device="cuda")))


def test_many_pairs():
    """More pairs than the first form's grid holds at once, and pairs of segments."""
    for P, L in ((30000, 70), (3000, 1500)):
        g = torch.Generator(device="cuda").manual_seed(P)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        lp = -rnd(2 * P * L).abs()
        mask = (torch.rand(2 * P * L, generator=g, device="cuda") < 0.6).to(torch.uint8)
        loss, rewards, w = gp.grpo_pref_loss_fwd(lp, mask, P, L, length_mean=True, beta=2.0, margin=0.5)
        grad = gp.grpo_pref_loss_bwd(mask, w, P, L)
        keep = mask.view(2 * P, L) != 0
        n = keep.sum(1)
        s = torch.where(keep, lp.view(2 * P, L).double(), 0.0).sum(1) / n.clamp(min=1)
        x = 2.0 * (s[0::2] - s[1::2]) - 0.5
        want = torch.nn.functional.softplus(-x)
        assert abs(loss.item() - want.mean().item()) <= 16 * plain_update.U * want.mean().item()
        assert ((rewards.double() - 2 * s).abs() <= 2 * plain_update.U * (2 * s).abs()).all()
        slope = torch.stack([-2 * torch.sigmoid(-x), 2 * torch.sigmoid(-x)], 1).view(-1) / P / n
        far = (grad.view(2 * P, L).double() - torch.where(keep, slope[:, None], 0.0)).abs()
        assert (far <= 16 * plain_update.U * slope.abs()[:, None]).all()
