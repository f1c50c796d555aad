"""The clipped policy loss on the GPU against the formulas in float64, within the bounds of the
float32 errors that tests/plain_update.py counts."""
import math

import pytest
import torch

import grpo_policy_loss_amd as gp
from tests import plain_update

pytestmark = pytest.mark.gpu


def inputs(B, L, seed=0, per_token=False, empty=True, garbage=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    N = B * L
    lp = -rnd(N).abs() * torch.rand(N, generator=g)
    mask = torch.zeros(B, L, dtype=torch.uint8)
    for b in range(B):
        n = int(torch.randint(0, L + 1, (1,), generator=g))
        start = int(torch.randint(0, L - n + 1, (1,), generator=g))
        mask[b, start:start + n] = 1 if b % 2 else 255      # any value but 0 counts
    if empty:
        mask[B // 2] = 0
    mask = mask.view(-1)
    i = dict(lp=lp, old=lp + 0.2 * rnd(N), ref=lp + 0.4 * rnd(N), mask=mask, adv=rnd(N if per_token else B))
    i["old"][::7] = lp[::7]          # tokens that have not moved
    i["ref"][::5] = lp[::5] + 1e-4 * rnd(N)[::5]
    if garbage:
        for k, v in (("lp", math.nan), ("old", math.inf), ("ref", -math.inf)):
            i[k] = torch.where(mask == 0, torch.tensor(v), i[k])
        if per_token:
            i["adv"] = torch.where(mask == 0, torch.tensor(math.nan), i["adv"])
    return i


def run(i, B, L, g=None, **how):
    names = dict(low="clip_low", high="clip_high", dual="clip_dual", kind="kl_estimator")
    kw = {names.get(k, k): v for k, v in how.items() if k not in ("sequence", "seq_mean", "old", "ref")}
    kw = dict(clip_low=0.0, clip_high=0.0) | kw
    kw["ratio"] = gp.RATIO_SEQUENCE if how.get("sequence") else gp.RATIO_TOKEN
    kw["aggregation"] = gp.AGG_SEQUENCE_MEAN if how.get("seq_mean") else gp.AGG_TOKEN_MEAN
    d = {k: v.cuda() for k, v in i.items()}
    kw["old_lp"] = d["old"] if how.get("old", True) else None
    kw["ref_lp"] = d["ref"] if how.get("ref", True) else None
    loss, stats, weights = gp.grpo_clip_loss_fwd(d["lp"], d["mask"], d["adv"], B, L, **kw)
    up = None if g is None else torch.full((1,), g, device="cuda")
    grad = gp.grpo_clip_loss_bwd(d["lp"], d["mask"], d["adv"], weights, B, L, grad_loss=up, **kw)
    return loss, stats, grad


def check(i, B, L, g=None, **how):
    loss, stats, grad = (t.cpu().double() for t in run(i, B, L, g, **how))
    plain = {k: v for k, v in how.items() if k not in ("old", "ref")}
    want = plain_update.clip_loss(i["lp"], i["old"] if how.get("old", True) else None, i["ref"] if how.get("ref", True) else None,
                                  i["mask"], i["adv"], B, L, g=1.0 if g is None else g, **plain)
    assert abs(loss.item() - want["loss"]) <= want["loss_tol"], (loss.item(), want["loss"], want["loss_tol"])
    near = (stats - want["stats"]).abs() <= want["stats_tol"]
    assert (near | (stats == want["stats"].float().double())).all(), (stats, want["stats"])      # (beyond float32)
    over = (grad - want["grad"]).abs() - want["grad_tol"]
    assert (over <= 0).all(), (over.max(), over.argmax())
    assert not grad[i["mask"] == 0].any()


SHAPES = [(1, 1), (3, 1), (1, 2), (5, 3), (7, 4), (4, 5), (9, 31), (2, 64), (8, 64), (3, 255), (5, 257), (33, 513), (2, 1023),
          (6, 1024), (3, 1025), (2, 4099), (1, 20000), (300, 17), (2051, 33)]


@pytest.mark.parametrize("B,L", SHAPES)
@pytest.mark.parametrize("sequence", [False, True])
@pytest.mark.parametrize("seq_mean", [False, True])
def test_lengths(B, L, sequence, seq_mean):
    i = inputs(B, L, seed=B + L)
    check(i, B, L, beta=0.04, low=0.2 if not sequence else 0.01, high=0.25 if not sequence else 0.02, sequence=sequence,
          seq_mean=seq_mean)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("how", [dict(), dict(low=0.1), dict(high=0.1), dict(dual=1.2), dict(low=0.1, high=0.3, dual=1.5), dict(low=2.0)])
@pytest.mark.parametrize("L", [100, 3000])
def test_clipping_and_estimators(kind, how, L):
    for sequence in (False, True):
        check(inputs(5, L, seed=kind), 5, L, g=-2.5, beta=0.5, kind=kind, sequence=sequence, **how)


@pytest.mark.parametrize("L", [50, 1500])
def test_without_reference_or_old_policy(L):
    i = inputs(4, L)
    check(i, 4, L, low=0.2, high=0.2, ref=False)
    check(i, 4, L, low=0.2, high=0.2, old=False, beta=0.1)
    check(i, 4, L, ref=False, old=False, seq_mean=True)
    check(i, 4, L, ref=False, old=False, sequence=True, low=0.2)
    check(i, 4, L, beta=0.0, low=0.2)               # kl in the statistics alone
    i["ref"].fill_(-math.inf)
    for sequence in (False, True):                  # and not in the loss where it is infinite
        loss, stats, grad = run(i, 4, L, low=0.2, sequence=sequence)
        assert stats[0].item() == math.inf and loss.isfinite() and grad.isfinite().all()
        assert torch.equal(loss, run(i, 4, L, low=0.2, sequence=sequence, ref=False)[0])


@pytest.mark.parametrize("L", [1, 77, 2500])
@pytest.mark.parametrize("seq_mean", [False, True])
def test_advantages_for_each_token(L, seq_mean):
    check(inputs(4, L, per_token=True, garbage=L > 1), 4, L, beta=0.1, low=0.2, high=0.2, dual=2.0, seq_mean=seq_mean)


def test_on_policy_equals_the_loss_of_the_head():
    """Without clipping or an older policy: grpo_loss's own loss, to float32's roundings of it."""
    i = inputs(6, 40, garbage=False)
    want = plain_update.clip_loss(i["lp"], None, i["ref"], i["mask"], i["adv"], 6, 40, beta=0.04)
    x = i["ref"].double() - i["lp"].double()
    kl = x.expm1() - x
    l = (-i["adv"].double().repeat_interleave(40) + 0.04 * kl)[i["mask"] != 0]
    assert abs(want["loss"] - l.mean()) < 1e-12
    check(i, 6, 40, beta=0.04, old=False)


def test_nothing_unmasked():
    for B, L in ((3, 20), (2, 3000)):
        i = inputs(B, L)
        i["mask"].zero_()
        for k in ("lp", "old", "ref"):
            i[k].fill_(math.nan)
        for sequence in (False, True):
            for seq_mean in (False, True):
                loss, stats, grad = run(i, B, L, beta=0.1, low=0.2, high=0.2, sequence=sequence, seq_mean=seq_mean)
                assert loss.item() == 0 and not stats.any() and not grad.any()


@pytest.mark.parametrize("where", ["lp", "old", "ref", "adv"])
@pytest.mark.parametrize("L", [30, 1100])
def test_a_nan_in_use_is_seen(where, L):
    i = inputs(3, L, empty=False, garbage=False)
    i["mask"].fill_(1)
    i[where][1 if where == "adv" else L + 3] = math.nan
    for sequence in (False, True):
        loss, _, grad = run(i, 3, L, beta=0.1, low=0.2, high=0.2, sequence=sequence)
        assert math.isnan(loss.item()) and grad[L + 3].isnan()
        assert not grad[:L].isnan().any() and not grad[2 * L:].isnan().any()


def test_far_ratios():
    """Ratios that overflow float32, and ones that are 0: clipped ones have finite losses."""
    lp = torch.tensor([0.0, 0.0, -200.0, -200.0, -60.0, 0.0])
    old = torch.tensor([-200.0, -200.0, 0.0, 0.0, 0.0, -60.0])
    i = dict(lp=lp, old=old, ref=lp.clone(), mask=torch.ones(6, dtype=torch.uint8), adv=torch.tensor([1.0, -1, 1, -1, 1, -1]))
    check(i, 6, 1, low=0.2, high=0.2, dual=3.0)
    loss, stats, grad = run(i, 6, 1, low=0.2, high=0.2)
    assert loss.item() == math.inf and grad[1].item() == -math.inf * -1 and stats[3].item() == math.inf
    # a reference that is certain of another token, and one that is not at all
    i["ref"] = torch.tensor([-3e8, -1e4, -150.0, -250.0, -59.0, 0.0])
    check(i, 6, 1, low=0.2, high=0.2, dual=3.0, beta=0.01)


def test_gradient_against_differences():
    """The loss's difference over a step along the gradient's own direction, in places where no ratio
    is near a border.  With h |v| = 2^-7 the third derivative's h^2 / 6 adds 10^-5, and the two losses'
    roundings 2^-23 |loss| / (2 h)."""
    B, L = 4, 300
    for sequence in (False, True):
        i = inputs(B, L, seed=3, garbage=False)
        i["old"] = i["lp"] + torch.where(torch.rand(B * L, generator=torch.Generator().manual_seed(1)) < 0.5, 0.05, -0.5 if not sequence else 0.06)
        how = dict(beta=0.3, low=0.2, high=0.3, sequence=sequence)
        _, _, grad = run(i, B, L, **how)
        grad = grad.cpu()
        v = (grad / grad.abs().max()).float()
        h = 2.0 ** -7
        up, down = (run(i | {"lp": i["lp"] + s * h * v}, B, L, **how)[0].double().item() for s in (1, -1))
        slope, want = (up - down) / (2 * h), (grad.double() * v.double()).sum().item()
        assert abs(slope - want) <= 4e-5 * abs(want) + 2.0 ** -22 * max(abs(up), abs(down)) / h


def test_bitwise_the_same_twice_and_on_another_stream():
    for B, L in ((500, 300), (3, 20480)):
        i = inputs(B, L)
        a = run(i, B, L, beta=0.1, low=0.2, high=0.2, seq_mean=True)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            b = run(i, B, L, beta=0.1, low=0.2, high=0.2, seq_mean=True)
        side.synchronize()
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_any_alignment_and_neighbours(offset):
    for B, L in ((5, 37), (2, 2049)):
        i = inputs(B, L)
        d = {}
        for k, v in i.items():
            flat = torch.empty(v.numel() + offset, dtype=v.dtype, device="cuda")
            flat[offset:] = v.cuda()
            d[k] = flat[offset:]
        how = dict(old_lp=d["old"], ref_lp=d["ref"], beta=0.1)
        loss, stats, w = gp.grpo_clip_loss_fwd(d["lp"], d["mask"], d["adv"], B, L, **how)
        flat = torch.full((B * L + offset + 8,), 7.0, device="cuda")
        gp.grpo_clip_loss_bwd(d["lp"], d["mask"], d["adv"], w, B, L, out=flat[offset:offset + B * L], **how)
        want = run(i, B, L, beta=0.1, low=0.2, high=0.2)
        for x, y in zip((loss, stats, flat[offset:offset + B * L]), want):
            assert torch.equal(x, y)
        assert (flat[:offset] == 7).all() and (flat[offset + B * L:] == 7).all()


def test_captured_and_replayed():
    B, L = 6, 1500
    i = {k: v.cuda() for k, v in inputs(B, L).items()}
    how = dict(old_lp=i["old"], ref_lp=i["ref"], beta=0.1, aggregation=gp.AGG_SEQUENCE_MEAN)
    up = torch.ones(1, device="cuda")
    out = {}

    def once():
        out["loss"], out["stats"], w = gp.grpo_clip_loss_fwd(i["lp"], i["mask"], i["adv"], B, L, **how)
        out["grad"] = gp.grpo_clip_loss_bwd(i["lp"], i["mask"], i["adv"], w, B, L, grad_loss=up, **how)
    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    held = dict(out)
    for k in range(4):
        i["lp"].add_(0.01 * k)
        up.fill_(1.0 + k)
        graph.replay()
        torch.cuda.synchronize()
        once()
        for name in out:
            assert torch.equal(out[name].nan_to_num(5.0), held[name].nan_to_num(5.0)), name


def test_autograd():
    B, L = 4, 50
    i = {k: v.cuda() for k, v in inputs(B, L, garbage=False).items()}
    lp = i["lp"].clone().requires_grad_()
    loss, stats = gp.grpo_clip_loss(lp, i["mask"], i["adv"], B, L, i["old"], i["ref"], beta=0.1)
    assert loss.dim() == 0 and not stats.requires_grad
    (3 * loss).backward()
    _, _, w = gp.grpo_clip_loss_fwd(i["lp"], i["mask"], i["adv"], B, L, i["old"], i["ref"], beta=0.1)
    want = gp.grpo_clip_loss_bwd(i["lp"], i["mask"], i["adv"], w, B, L, i["old"], i["ref"], beta=0.1, grad_loss=torch.full((1,), 3.0, device="cuda"))
    assert torch.equal(lp.grad, want)
    two = i["lp"].clone().view(B, L).requires_grad_()        # log-probabilities in rows
    gp.grpo_clip_loss(two, i["mask"], i["adv"], B, L)[0].backward()
    assert two.grad.shape == (B, L)


def test_a_captured_backward_is_refused():
    lp = torch.zeros(8, device="cuda", requires_grad=True)
    mask, adv = torch.ones(8, dtype=torch.uint8, device="cuda"), torch.ones(2, device="cuda")
    loss, _ = gp.grpo_clip_loss(lp, mask, adv, 2, 4)
    from grpo_policy_loss_amd import autograd
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x = torch.zeros(1, device="cuda")      # a graph of something
        with pytest.raises(RuntimeError, match="cannot be captured"):
            autograd._refuse_capture("grpo_clip_loss", "grpo_clip_loss_bwd")
    graph.replay()
    assert x.item() == 0
    loss.backward()


def test_long_batches():
    """Many rows of one block each, more sequences than the first form's grid, and 2^24 tokens."""
    for B, L, sequence in ((9000, 1026, True), (70000, 3, False), (40000, 130, True)):
        g = torch.Generator(device="cuda").manual_seed(B)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        lp = -rnd(B * L).abs()
        old, adv = lp + 0.1 * rnd(B * L), rnd(B)
        mask = (torch.rand(B * L, generator=g, device="cuda") < 0.6).to(torch.uint8)
        how = dict(old_lp=old, clip_low=0.05, clip_high=0.05, ratio=int(sequence), aggregation=gp.AGG_SEQUENCE_MEAN)
        loss, stats, w = gp.grpo_clip_loss_fwd(lp, mask, adv, B, L, **how)
        grad = gp.grpo_clip_loss_bwd(lp, mask, adv, w, B, L, **how)
        keep = mask.view(B, L) != 0
        D = torch.where(keep, (lp.double() - old.double()).view(B, L), 0.0)
        n = keep.sum(1, keepdim=True).clamp(min=1)
        if sequence:
            D = (D.sum(1, keepdim=True) / n).expand(B, L)
        r, A = D.exp(), adv.double().view(B, 1)
        s = torch.where(A >= 0, r.clamp(max=1.05), r.clamp(min=0.95))
        want = (torch.where(keep, -A * s, 0.0) / n).sum() / B
        size = (torch.where(keep, (A * s).abs(), 0.0) / n).sum() / B
        assert abs(loss.item() - want.item()) <= 16 * plain_update.U * size.item()
        slope = torch.where(keep & (s == r), -A * r, 0.0) / n / B
        assert ((grad.view(B, L).double() - slope).abs() <= 24 * plain_update.U * slope.abs()).all()
        clipped = (keep & (s != r)).sum().item() / keep.sum().item()
        assert abs(stats[1].item() + stats[2].item() - clipped) <= 4 * plain_update.U
