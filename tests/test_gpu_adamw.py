"""The AdamW step on the GPU against the formula in float64.

Tolerances, with U = 2^-24: a float32 moment passes at most five roundings (two rounded
constants, two products, a sum; one more product for the scaled gradient); the quotient adds
its moments' errors and at most 16 U of its own (root, division, bias corrections of a few
units each); the weight adds 4 U of itself, a bfloat16 parameter half its eps.  Codes of
8-bit moments are those of the float64 moments: they are equal."""
import pytest
import torch

import grpo_policy_loss_amd as gp
from tests import plain_ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SIZES = [1, 0, 3, 255, 256, 257, 1023, 4095, 4096, 4097, 100003]
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def make(sizes, pt, gt, master, bits, packed, seed=0):
    """Lists of tensors, packed behind each other in one buffer or each in its own."""
    gen = torch.Generator().manual_seed(seed)

    def place(values, dtype):
        if not packed:
            return [v.to(dtype).cuda() for v in values]
        flat = torch.cat([torch.full((1,), 7.0)] + [v.float() for v in values] + [torch.full((3,), 7.0)]).to(dtype).cuda()
        out, at = [], 1
        for v in values:
            out.append(flat[at:at + v.numel()])
            at += v.numel()
        return out
    rnd = [torch.randn(n, generator=gen) for n in sizes]
    s = dict(p=place(rnd, pt), g=place([torch.randn(n, generator=gen) * 10 ** torch.randn(1, generator=gen) for n in sizes], gt))
    s["master"] = place([p.cpu().float() + 1e-4 for p in s["p"]], torch.float32) if master else None
    m = [torch.randn(n, generator=gen) * 0.1 for n in sizes]
    v = [torch.randn(n, generator=gen) ** 2 * 0.01 * 10 ** torch.randn(n, generator=gen) for n in sizes]
    if bits == 32:
        s["m"], s["v"] = place(m, torch.float32), place(v, torch.float32)
    else:
        for k, x in (("m", m), ("v", v)):
            enc = [plain_ops.moment_codes(y, k == "v") for y in x]
            codes = place([c.float() for c, _ in enc], torch.int8 if k == "m" else torch.uint8)
            s[k] = [gp.Moment8(c, a.cuda()) for c, (_, a) in zip(codes, enc)]
    return s


def state64(s, bits):
    cpu = lambda x: [t.detach().cpu().clone() for t in x]  # noqa: E731
    mom = cpu if bits == 32 else (lambda x: [plain_ops.moment_values(q.codes.cpu(), q.scales.cpu()) for q in x])
    return dict(w=cpu(s["master"] or s["p"]), g=cpu(s["g"]), m=mom(s["m"]), v=mom(s["v"]))


def check(s, old, bits, step, scale, hyper=HYPER):
    for i in range(len(s["p"])):
        w0, g, m0, v0 = (old[k][i].double().flatten() for k in "wgmv")
        w, m, v = plain_ops.adamw(w0, g, m0, v0, step, hyper["lr"], hyper["betas"], hyper["eps"], hyper["weight_decay"], scale)
        b1, b2 = hyper["betas"]
        x = (g * scale).abs()
        tol_m, tol_v = 6 * U * (m0.abs() * b1 + x * (1 - b1)), 7 * U * (v0 * b2 + x * x * (1 - b2))
        if bits == 32:
            assert ((s["m"][i].cpu().double().flatten() - m).abs() <= tol_m).all()
            assert ((s["v"][i].cpu().double().flatten() - v).abs() <= tol_v).all()
        else:
            for q, want in ((s["m"][i], m), (s["v"][i], v)):
                codes, scales = plain_ops.moment_codes(want, q.codes.dtype == torch.uint8)
                assert torch.equal(q.codes.cpu().flatten(), codes)
                assert torch.allclose(q.scales.cpu(), scales, rtol=2.0 ** -23, atol=0)
                got = gp.dequantize_moment(q).cpu().double().flatten()
                back = plain_ops.moment_values(q.codes.cpu(), q.scales.cpu())
                assert ((got - back).abs() <= U * back.abs() + 1e-45).all()
        den = (v / (1 - b2 ** step)).sqrt() + hyper["eps"]
        upd = hyper["lr"] / (1 - b1 ** step) / den
        tol = 4 * U * w0.abs() + upd * (tol_m + 16 * U * m.abs()) + 1e-45
        got = (s["master"] or s["p"])[i].cpu()
        if got.dtype == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * w.abs()
        assert ((got.double().flatten() - w).abs() <= tol).all()
        if s["master"]:
            assert torch.equal(s["p"][i].cpu(), got.bfloat16().view(s["p"][i].shape))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,gt,master", [
    (torch.float32, torch.float32, False), (torch.float32, torch.bfloat16, False),
    (torch.bfloat16, torch.float32, False), (torch.bfloat16, torch.bfloat16, False),
    (torch.bfloat16, torch.float32, True), (torch.bfloat16, torch.bfloat16, True)])
def test_steps(pt, gt, master, bits, packed):
    s = make(SIZES, pt, gt, master, bits, packed)
    plan = gp.adamw_plan(s["p"], s["g"], s["m"], s["v"], master=s["master"])
    for step, scale in ((1, 1.0), (2, 0.25), (1000, 1.0)):
        old = state64(s, bits)
        gp.grpo_adamw(plan, step, grad_scale=None if scale == 1.0 else torch.full((1,), scale, device="cuda"), **HYPER)
        check(s, old, bits, step, scale)
    if packed:      # what lies before and behind the tensors
        for x in (s["p"], s["g"], s["master"] or s["p"]):
            flat = x[0]._base if x[0]._base is not None else x[0]
            assert flat[0] == 7 and (flat[-3:] == 7).all()


def test_more_tensors_than_one_search_level():
    sizes = [(i * 37) % 613 for i in range(4500)]
    s = make(sizes, torch.float32, torch.float32, False, 32, True)
    old = state64(s, 32)
    gp.grpo_adamw(gp.adamw_plan(s["p"], s["g"], s["m"], s["v"]), 3, **HYPER)
    check(s, old, 32, 3, 1.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero_moments(bits):
    p = [torch.randn(777, device="cuda"), torch.randn(3, 5, device="cuda")]
    g = [torch.randn_like(x) for x in p]
    g[0][:256] = 0                                  # a block that stays zero
    g[0][300] = 1e-30                               # a square that leaves float32's range
    m, v = gp.adamw_moments(p, bits)
    s = dict(p=p, g=g, m=m, v=v, master=None)
    old = state64(s, bits)
    gp.grpo_adamw(gp.adamw_plan(p, g, m, v), 1, **HYPER)
    if bits == 8:
        assert (v[0].codes[:256] == 0).all() and v[0].scales[0] == 0
        assert v[0].codes[300] == 1                 # positive: never stored as zero
        check(s, old, bits, 1, 1.0)
    assert all(x.isfinite().all() for x in p)


def test_first_step_from_zero_float32_moments():
    gen = torch.Generator().manual_seed(4)
    p = [torch.randn(777, generator=gen).cuda(), torch.randn(3, 5, generator=gen).cuda()]
    g = [torch.randn(x.shape, generator=gen).cuda() for x in p]
    g[0][:256] = 0                                  # a block without a gradient
    m, v = gp.adamw_moments(p, 32)
    s = dict(p=p, g=g, m=m, v=v, master=None)
    old = state64(s, 32)
    gp.grpo_adamw(gp.adamw_plan(p, g, m, v), 1, **HYPER)
    check(s, old, 32, 1, 1.0)
    assert not m[0][:256].any() and not v[0][:256].any()


@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.9, 0.95), (0.95, 0.98)])
def test_scales_that_lie_between_two_float32_values(betas):
    """Bfloat16 gradients and old moments at their blocks' scales: the new scale is often an exact
    tie of float32, which the last bit of the float64 sum decides, and after the first step many
    moments are a quarter of their block's largest, a root of exactly 63 and a half.  Scales and
    codes are those of the formula's own order of operations, bit for bit, step after step."""
    n = 1 << 20
    gen = torch.Generator().manual_seed(2)
    p = [torch.randn(n, generator=gen).cuda()]
    g = [(1e-3 * torch.randn(n, generator=gen)).bfloat16().cuda()]
    m, v = gp.adamw_moments(p, 8)
    hyper = dict(lr=1e-4, betas=betas, eps=1e-8, weight_decay=0.0)
    plan = gp.adamw_plan(p, g, m, v)
    for step in (1, 2, 3, 4):
        g[0].mul_(torch.randn(n, generator=gen).cuda().sign())
        before = [plain_ops.moment_values(q.codes.cpu(), q.scales.cpu()) for q in (m[0], v[0])]
        gp.grpo_adamw(plan, step, **hyper)
        x = g[0].cpu().double()
        for q, old, new, b in ((m[0], before[0], x, betas[0]), (v[0], before[1], x * x, betas[1])):
            codes, scales = plain_ops.moment_codes(old * b + new * (1 - b), q.codes.dtype == torch.uint8)
            assert torch.equal(q.scales.cpu(), scales)
            assert torch.equal(q.codes.cpu(), codes)


def test_values_that_are_not_finite_stay_where_they_are():
    for bits in (32, 8):
        s = make([2000], torch.float32, torch.float32, False, bits, False)
        s["g"][0][700], s["g"][0][1500] = float("nan"), float("inf")
        gp.grpo_adamw(gp.adamw_plan(s["p"], s["g"], s["m"], s["v"]), 2, **HYPER)
        bad = ~s["p"][0].isfinite()
        assert bad.nonzero().flatten().tolist() == [700, 1500]
        if bits == 32:
            assert (~s["m"][0].isfinite()).nonzero().flatten().tolist() == [700, 1500]
        else:
            for q in (s["m"][0], s["v"][0]):
                lost = gp.dequantize_moment(q).isnan()
                blocks = torch.arange(2000, device="cuda") // 256
                assert torch.equal(lost, (blocks == 700 // 256) | (blocks == 1500 // 256))
                assert (q.codes[lost] == 0).all()


def test_betas_of_zero_and_no_decay():
    hyper = dict(lr=1e-2, betas=(0.0, 0.0), eps=1e-6, weight_decay=0.0)
    s = make([513], torch.float32, torch.float32, False, 32, False)
    old = state64(s, 32)
    gp.grpo_adamw(gp.adamw_plan(s["p"], s["g"], s["m"], s["v"]), 1, **hyper)
    check(s, old, 32, 1, 1.0, hyper)


@pytest.mark.parametrize("bits", [32, 8])
def test_an_eps_below_float32_keeps_what_has_no_gradient(bits):
    p = torch.full((600,), 2.0, device="cuda")
    g = torch.zeros_like(p)
    g[::2] = 3.0
    m, v = gp.adamw_moments([p], bits)
    gp.grpo_adamw(gp.adamw_plan([p], [g], m, v), step=1, lr=0.5, eps=1e-50, weight_decay=0.0)
    want = torch.where(g > 0, 1.5, 2.0)                  # m / sqrt(v) is 1 at the first step
    assert ((p - want).abs() <= 32 * U).all() and (p[1::2] == 2).all()


def test_a_plan_of_many_elements_is_that_of_its_pieces():
    sizes = [(1 << 26) - 12345, 300, 1, 60001]
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda n, t: torch.randn(n, generator=gen, device="cuda").to(t)  # noqa: E731
    p, g, w = ([rnd(n, t) for n in sizes] for t in (torch.bfloat16, torch.bfloat16, torch.float32))
    m, v = [rnd(n, torch.float32) for n in sizes], [rnd(n, torch.float32).square() for n in sizes]
    copies = [[t.clone() for t in x] for x in (p, m, v, w)]
    gp.grpo_adamw(gp.adamw_plan(p, g, m, v, w), step=3, lr=1e-2)
    for i, n in enumerate(sizes):
        for at in range(0, n, 40_000_001):
            q = [[x[i][at:at + 40_000_001]] for x in (copies[0], g, *copies[1:])]
            gp.grpo_adamw(gp.adamw_plan(*q), step=3, lr=1e-2)
    for got, want in zip((p, m, v, w), copies):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_follows_its_device_scalars(bits):
    a = make([5000, 300], torch.bfloat16, torch.float32, True, bits, False)
    b = make([5000, 300], torch.bfloat16, torch.float32, True, bits, False)
    step, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.full((1,), 1e-3, device="cuda")
    pa, pb = (gp.adamw_plan(s["p"], s["g"], s["m"], s["v"], master=s["master"]) for s in (a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gp.grpo_adamw(pa, step, lr=lr)
        step += 1
    for t in range(1, 6):
        lr.fill_(1e-3 / t)
        graph.replay()
        torch.cuda.synchronize()
        gp.grpo_adamw(pb, torch.full((1,), t, dtype=torch.int64, device="cuda"), lr=lr)
        torch.cuda.synchronize()
        for x, y in zip(a["master"] + a["p"], b["master"] + b["p"]):
            assert torch.equal(x, y)
    old = state64(b, bits)      # the device's step and the host's
    c = {k: (v if v is None else [x.clone() if torch.is_tensor(x) else gp.Moment8(x.codes.clone(), x.scales.clone()) for x in v])
         for k, v in b.items()}
    gp.grpo_adamw(pb, step, lr=lr, betas=HYPER["betas"], eps=HYPER["eps"], weight_decay=HYPER["weight_decay"])
    check(b, old, bits, 6, 1.0, {**HYPER, "lr": lr.item()})
    gp.grpo_adamw(gp.adamw_plan(c["p"], c["g"], c["m"], c["v"], master=c["master"]), 6, lr=lr,
                  betas=HYPER["betas"], eps=HYPER["eps"], weight_decay=HYPER["weight_decay"])
    check(c, old, bits, 6, 1.0, {**HYPER, "lr": lr.item()})


def test_another_stream():
    a, b = (make([100003], torch.bfloat16, torch.float32, True, 8, False) for _ in range(2))
    side = torch.cuda.Stream()
    plan = gp.adamw_plan(a["p"], a["g"], a["m"], a["v"], master=a["master"])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gp.grpo_adamw(plan, 1)
    del plan
    torch.cuda.current_stream().wait_stream(side)
    gp.grpo_adamw(gp.adamw_plan(b["p"], b["g"], b["m"], b["v"], master=b["master"]), 1)
    assert torch.equal(a["master"][0], b["master"][0]) and torch.equal(a["m"][0].codes, b["m"][0].codes)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [False, True])
def test_a_plan_tells_whether_it_holds_its_tensors(master, bits):
    p = [torch.nn.Parameter(torch.randn(300, 5, device="cuda").bfloat16()), torch.nn.Parameter(torch.randn(7, device="cuda").bfloat16())]
    for x in p:
        x.grad = torch.randn_like(x)
    w = [x.detach().float() for x in p] if master else None
    m, v = gp.adamw_moments(p, bits)

    def grads():
        return [x.grad for x in p]
    plan = gp.adamw_plan(p, grads(), m, v, w)
    gp.grpo_adamw(plan, 1)
    assert plan.holds(p, grads(), w)
    assert not plan.holds(p[:1], grads()[:1], w and w[:1])
    assert not plan.holds(p, grads(), None if master else [x.float() for x in p])
    assert not plan.holds(p[::-1], grads()[::-1], w and w[::-1])
    kept = p[1].grad
    p[1].grad = None                        # zero_grad's default
    assert not plan.holds(p, grads(), w)
    p[1].grad = torch.zeros_like(p[1])      # another one
    assert not plan.holds(p, grads(), w)
    p[1].grad = kept
    assert plan.holds(p, grads(), w)
    old = p[0].data
    p[0].data = old.clone()
    assert not plan.holds(p, grads(), w)
    p[0].data = old
    assert plan.holds(p, grads(), w)
    p[0].grad.untyped_storage().resize_(0)  # freed in place
    assert not plan.holds(p, grads(), w)
    moved = m[1].codes if bits == 8 else m[1]
    plan = gp.adamw_plan(p[1:], grads()[1:], m[1:], v[1:], w and w[1:])
    assert plan.holds(p[1:], grads()[1:], w and w[1:])
    moved.untyped_storage().resize_(0)
    assert not plan.holds(p[1:], grads()[1:], w and w[1:])


def test_autograd_sees_the_step():
    w = torch.randn(16, 8, device="cuda", requires_grad=True)
    g = torch.randn_like(w)
    m, v = gp.adamw_moments([w])
    y = (w * w).sum()
    gp.grpo_adamw(gp.adamw_plan([w], [g], m, v), 1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_offsets_beyond_32_bits():
    n = (1 << 31) + 300
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = gp.adamw_moments([p], 8)
    tail = 1000
    gen = torch.Generator().manual_seed(1)
    p[-tail:], g[-tail:] = (torch.randn(tail, generator=gen).cuda() for _ in range(2))
    g[0] = 1.0
    w0, g0 = p[-tail:].cpu(), g[-tail:].cpu()
    gp.grpo_adamw(gp.adamw_plan([p], [g], m, v), 1, **HYPER)
    want, em, _ = plain_ops.adamw(w0, g0, torch.zeros(tail), torch.zeros(tail), 1, HYPER["lr"], HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
    assert ((p[-tail:].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()
    assert abs(p[0].item() + HYPER["lr"]) < 1e-4 and (p[1:4096] == 0).all()
    last = n % 256
    assert abs(m[0].scales[-1].item() - em[-last:].abs().max().item()) < 1e-6
    assert (m[0].codes[1 << 20:(1 << 20) + 4096] == 0).all()


def test_refusals_on_the_gpu():
    p = torch.zeros(512, device="cuda")
    m, v = gp.adamw_moments([p])
    with pytest.raises(gp.GrpoError, match="overlap"):
        gp.adamw_plan([p, p], [torch.zeros_like(p)] * 2, m * 2, v * 2)
    with pytest.raises(ValueError, match="contiguous"):
        gp.adamw_plan([p[::2]], [p[256:].clone()], [m[0][:256]], [v[0][:256]])
    plan = gp.adamw_plan([p], [torch.zeros_like(p)], m, v)
    with pytest.raises(gp.GrpoError, match="step"):
        gp.grpo_adamw(plan, 0)
    with pytest.raises(TypeError, match="step"):
        gp.grpo_adamw(plan, torch.ones(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="grad_scale"):
        gp.grpo_adamw(plan, 1, grad_scale=torch.ones(2, device="cuda"))
