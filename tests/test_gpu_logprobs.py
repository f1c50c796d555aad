"""The log-probabilities with their gradient on the GPU, against the formulas in float64 and within
the bounds that tests/plain_update.py counts."""
import math

import pytest
import torch

import grpo_policy_loss_amd as gp
from tests import plain_update

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": plain_update.U, "bf16": 2.0 ** -8}


def inputs(N, d, V, t, seed=0, dead=0.3):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    W = (rnd(V, d) / math.sqrt(d)).to(TYPES[t])
    y = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    H = rnd(N, d) + 6 * torch.rand(N, 1, generator=g) * W[y.long()].float()     # some targets are likely
    up = rnd(N) * (torch.rand(N, generator=g) >= dead)
    return dict(H=H.to(TYPES[t]).cuda(), W=W.cuda(), y=y.cuda(), g=up.cuda())


def check(i, t, chunk=4096, opts=None, k=1.0, cap=0.0):
    lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"], chunk, opts=opts)
    dH, dW = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, i["g"], chunk, opts=opts)
    want = plain_update.logprobs(i["H"], i["W"], i["y"], i["g"], k=k, cap=cap, half=HALF[t])
    for name, x in (("lp", lp), ("dH", dH), ("dW", dW)):
        over = (x.cpu().double() - want[name]).abs() - want[name + "_tol"]
        assert (over <= 0).all(), (name, over.max())
    assert not dH[i["g"] == 0].any()
    return lp, lse, dH, dW


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("N,d,V,chunk", [(1, 8, 2, 1), (1, 64, 1000, 4096), (3, 16, 1, 2), (255, 40, 257, 4096), (256, 256, 256, 256),
                                         (300, 320, 1003, 128), (513, 72, 2051, 512), (40, 1024, 5003, 16), (65, 200, 6401, 4096),
                                         (64, 64, 20000, 4096), (1500, 64, 1100, 700), (130, 520, 64, 100)])
def test_sizes(t, N, d, V, chunk):
    check(inputs(N, d, V, t, seed=N), t, chunk)


@pytest.mark.parametrize("t,N,d,V,chunk", [("bf16", 700, 512, 12100, 256), ("bf16", 700, 512, 12100, 4096), ("f32", 2050, 1024, 8300, 4096),
                                           ("f32", 2050, 1024, 8300, 900), ("f32", 256, 256, 65500, 4096),
                                           ("f32", 2050, 1024, 24600, 4096), ("f32", 2050, 1024, 24600, 900)])
def test_sizes_of_the_large_tiles(t, N, d, V, chunk):
    i = inputs(N, d, V, t, seed=N)
    lp, lse, dH, dW = check(i, t, chunk)
    # dW written and dW added to, and each gradient alone
    args = (i["H"], i["W"], i["y"], lp, lse, i["g"], chunk)
    into = torch.full_like(dW, 0.5)
    gp.grpo_logprobs_bwd(*args, dW=into, need_h=False)
    assert ((into - 0.5 - dW).abs() <= 8 * plain_update.U * (1 + dW.abs())).all()
    assert torch.equal(gp.grpo_logprobs_bwd(*args, need_w=False)[0], dH)
    W = i["W"].clone().requires_grad_()
    gp.grpo_logprobs(i["H"], W, i["y"], chunk).backward(i["g"])
    assert torch.equal(W.grad, dW.to(W.dtype))
    i["g"].zero_()
    dH, dW = gp.grpo_logprobs_bwd(*args)
    assert not dH.any() and not dW.any()
    W.grad = None
    gp.grpo_logprobs(i["H"], W, i["y"], chunk).backward(i["g"])
    assert not W.grad.any()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("N,d,V,chunk", [(1100, 8, 2, 4096), (1024, 8, 1, 4096), (2100, 64, 130, 4096), (3001, 72, 1003, 1500), (4200, 328, 70, 8192),
                                         (1601, 256, 1100, 8192), (9001, 40, 5, 8192)])
def test_many_tokens_of_a_small_head(t, N, d, V, chunk):
    """dW's sums are split over the tokens."""
    i = inputs(N, d, V, t, seed=N)
    lp, lse, dH, dW = check(i, t, chunk)
    args = (i["H"], i["W"], i["y"], lp, lse, i["g"], chunk)
    assert torch.equal(gp.grpo_logprobs_bwd(*args, need_h=False)[1], dW)
    assert torch.equal(gp.grpo_logprobs_bwd(*args, need_w=False)[0], dH)
    into = torch.full_like(dW, 0.5)
    gp.grpo_logprobs_bwd(*args, dW=into)
    assert ((into - 0.5 - dW).abs() <= 8 * plain_update.U * (1 + dW.abs())).all()
    W = i["W"].clone().requires_grad_()
    gp.grpo_logprobs(i["H"], W, i["y"], chunk).backward(i["g"])
    assert torch.equal(W.grad, dW.to(W.dtype))


@pytest.mark.parametrize("N,d,V", [(2050, 1024, 8300), (256, 256, 65500), (2050, 1024, 24600)])
def test_large_tiles_with_a_cap(N, d, V):
    i = inputs(N, d, V, "f32", seed=1)
    check(i, "f32", 4096, {"logit_softcapping": 3.0, "temperature": 0.8}, 1 / 0.8, 3.0)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("opts,k,cap", [({"temperature": 0.7}, 1 / 0.7, 0.0), ({"logit_softcapping": 3.0}, 1.0, 3.0),
                                        ({"logit_softcapping": 3.0, "temperature": 0.8}, 1 / 0.8, 3.0), ({"logit_scale_multiply": 0.5}, 0.5, 0.0)])
def test_logit_transforms(t, opts, k, cap):
    check(inputs(130, 64, 700, t), t, 64, opts, k, cap)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_forward_is_the_reference_calls_and_the_loss_s(t):
    """bfloat16: lp and lse bitwise grpo_ref_logprobs's and the loss's; float32: within lse's rounding and
    that of the logits (64 products each way).  The loss's gradient given as grad_lp: the loss's
    backward up to the roundings of coefficients and of each."""
    B, L, d, V = 3, 50, 64, 900
    i = inputs(B * L, d, V, t)
    mask = (torch.rand(B * L, device="cuda") < 0.6).to(torch.uint8)
    adv = torch.randn(B, device="cuda")
    ref = gp.grpo_ref_logprobs(i["H"], i["W"], i["y"]) + 0.1
    lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"])
    plain = gp.grpo_ref_logprobs(i["H"], i["W"], i["y"])
    loss, lp2, kl, lse2 = gp.grpo_loss_fwd(i["H"], i["W"], i["y"], mask, adv, ref, B, L)
    if t == "bf16":
        assert torch.equal(lp, plain) and torch.equal(lp, lp2) and torch.equal(lse, lse2)
    else:
        near = plain_update.logprobs(i["H"], i["W"], i["y"], i["g"])["lp_tol"].cuda()
        assert ((lp - lp2).abs() <= 2 * near).all() and ((lse[:B * L] - lse2).abs() <= 2 * near).all()
    dH, dW = gp.grpo_loss_bwd(i["H"], i["W"], i["y"], mask, adv, ref, lp2, lse2, B, L)
    ours, stats, w = gp.grpo_clip_loss_fwd(lp, mask, adv, B, L, ref_lp=ref, beta=0.04)
    g = gp.grpo_clip_loss_bwd(lp, mask, adv, w, B, L, ref_lp=ref, beta=0.04)
    dH2, dW2 = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, g)
    assert abs(loss.item() - ours.item()) <= 1e-6 * (abs(loss.item()) + 1)
    # coefficients within 16 roundings of float32, and each dZ at most one step apart after that
    far = 16 * plain_update.U + 2 * HALF[t]
    want = plain_update.logprobs(i["H"], i["W"], i["y"], g, half=HALF[t])
    for a, b, n in ((dH, dH2, "dH"), (dW, dW2, "dW")):
        assert ((a.double() - b.double()).abs().cpu() <= 2 * want[n + "_tol"] + far * want[n].abs()).all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_accumulation_and_one_gradient_alone(t):
    i = inputs(200, 64, 600, t)
    lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"])
    args = (i["H"], i["W"], i["y"], lp, lse, i["g"])
    tol = plain_update.logprobs(i["H"], i["W"], i["y"], i["g"], half=HALF[t])["dW_tol"].cuda()
    for chunk in (64, 4096):
        dH, dW = gp.grpo_logprobs_bwd(*args, chunk=chunk)
        only_h, none = gp.grpo_logprobs_bwd(*args, chunk=chunk, need_w=False)
        assert none is None and torch.equal(only_h, dH)
        none, only_w = gp.grpo_logprobs_bwd(*args, chunk=chunk, need_h=False)
        assert none is None and torch.equal(only_w, dW)
        start = torch.randn(600, 64, device="cuda")
        into = start.clone()
        _, same = gp.grpo_logprobs_bwd(*args, chunk=chunk, dW=into)
        assert same is into
        # the same products, summed onto the start: one rounding of it for each chunk
        assert ((into.double() - start.double() - dW.double()).abs() <= 2 * tol + 6 * plain_update.U * start.abs()).all()


def test_no_token_has_a_gradient():
    for t in TYPES:
        i = inputs(70, 64, 300, t)
        i["H"][3] = math.nan                 # tokens without a gradient may hold anything
        i["g"].zero_()
        lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"])
        assert lp[3].isnan() and not lp[:3].isnan().any()
        for chunk in (16, 4096):
            dH, dW = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, i["g"], chunk)
            assert not dH.any() and not dW.any()
        i["g"][5] = -0.5
        i["g"][6] = -0.0
        dH, dW = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, i["g"])
        assert not dH.isnan().any() and not dW.isnan().any() and dH[5].any() and not dH[6].any()


def test_targets_outside_the_vocabulary():
    """Padding's -100: NaN log-probabilities, which a loss leaves out, and no gradient."""
    i = inputs(40, 64, 300, "bf16", dead=0.0)
    out = torch.arange(40, device="cuda") % 4 == 0
    i["y"][out] = torch.tensor([-100, 300], dtype=torch.int32, device="cuda").repeat(5)
    lp = gp.grpo_logprobs(i["H"], i["W"], i["y"])
    assert torch.equal(lp.isnan(), out)
    H, W = i["H"].requires_grad_(), i["W"].requires_grad_()
    lp = gp.grpo_logprobs(H, W, i["y"])
    loss, _ = gp.grpo_clip_loss(lp, (~out).to(torch.uint8), torch.randn(4, device="cuda"), 4, 10)
    loss.backward()
    assert not H.grad.isnan().any() and not W.grad.isnan().any() and not H.grad[out].any() and H.grad[~out].any(1).all()


def test_autograd():
    for t in TYPES:
        i = inputs(60, 64, 500, t)
        lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"], opts={"temperature": 0.9})
        dH, dW = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, i["g"], opts={"temperature": 0.9})
        H, W = i["H"].clone().requires_grad_(), i["W"].clone().requires_grad_()
        out = gp.grpo_logprobs(H, W, i["y"], opts={"temperature": 0.9})
        assert torch.equal(out, lp)
        out.backward(i["g"])
        assert torch.equal(H.grad, dH) and torch.equal(W.grad, dW.to(W.dtype))
        # several chunks: the sum over them is rounded, not the parts
        Wp = i["W"].clone().requires_grad_()
        gp.grpo_logprobs(i["H"], Wp, i["y"], chunk=20, opts={"temperature": 0.9}).backward(i["g"])
        parts = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, i["g"], chunk=20, opts={"temperature": 0.9})[1]
        assert torch.equal(Wp.grad, parts.to(W.dtype))
        # a frozen head, frozen hidden states, and a sum's broadcast gradient
        H = i["H"].clone().requires_grad_()
        gp.grpo_logprobs(H, i["W"], i["y"]).sum().backward()
        W = i["W"].clone().requires_grad_()
        gp.grpo_logprobs(i["H"], W, i["y"]).sum().backward()
        ones = torch.ones(60, device="cuda")
        lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"])
        dH, dW = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, ones)
        assert torch.equal(H.grad, dH) and torch.equal(W.grad, dW.to(W.dtype))


def test_gradient_against_differences():
    """float32: the log-probabilities' sum moved along dH and dW.  Their roundings are some 2^-20 each,
    300 of them at random: 2^-15; over 2 h = 2^-5 that is 2^-10 of a slope of the order of hundreds."""
    i = inputs(300, 64, 500, "f32", dead=0.2)
    lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"])
    grads = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, i["g"])
    for name, grad in zip("HW", grads):
        v = grad / grad.norm()
        h = 2.0 ** -6
        f = [(gp.grpo_logprobs_fwd(*(i[n] + s * h * v if n == name else i[n] for n in "HW"), i["y"])[0].double() * i["g"].double()).sum().item()
             for s in (1, -1)]
        slope, want = (f[0] - f[1]) / (2 * h), grad.double().norm().item()
        assert abs(slope - want) <= 1e-3 * want + 2.0 ** -9


def test_captured_and_replayed():
    i = inputs(300, 64, 700, "bf16")
    lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"], 128)
    out = {}

    def once():
        out["lp"], out["lse"] = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"], 128)
        out["dH"], out["dW"] = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], out["lp"], out["lse"], i["g"], 128)
    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    held = dict(out)
    for k in range(4):
        i["g"].mul_(-1.5)
        if k == 2:
            i["g"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        once()
        assert all(torch.equal(held[n], out[n]) for n in out)


@pytest.mark.parametrize("t,N,d,V", [("f32", 300, 64, 700), ("f32", 256, 256, 65500), ("bf16", 300, 64, 700), ("bf16", 700, 512, 12100)])
def test_bitwise_the_same_on_two_streams_at_once(t, N, d, V):
    i = inputs(N, d, V, t)
    lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"])
    want = (lp, lse, *gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, i["g"]))
    torch.cuda.synchronize()
    sides, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(3):
        for s in sides:
            with torch.cuda.stream(s):
                lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"])
                got.append((lp, lse, *gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, i["g"])))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("N,d,V", [(70, 64, 300), (700, 512, 12100)])
def test_neighbours_are_left_as_they_were(t, N, d, V):
    """Inputs and gradients inside larger buffers, filled with NaN around them."""
    i = inputs(N, d, V, t, seed=5)
    lp, lse = gp.grpo_logprobs_fwd(i["H"], i["W"], i["y"])
    want = gp.grpo_logprobs_bwd(i["H"], i["W"], i["y"], lp, lse, i["g"])

    def inside(x, fill=None):
        buf = torch.full((x.numel() + 128,), math.nan, dtype=x.dtype, device="cuda")
        view = buf[64:-64].view(x.shape)
        view.copy_(x if fill is None else torch.full_like(x, fill))
        return buf, view
    H, W = inside(i["H"])[1], inside(i["W"])[1]
    g = torch.full((N + 32,), math.nan, device="cuda")
    g[16:-16] = i["g"]
    lp2, lse2 = gp.grpo_logprobs_fwd(H, W, i["y"])
    assert torch.equal(lp, lp2) and torch.equal(lse, lse2)
    hb, dH = inside(want[0], 7.0)
    wb, dW = inside(want[1], 0.0)
    gp.grpo_logprobs_bwd(H, W, i["y"], lp2, lse2, g[16:-16], dH=dH, dW=dW)
    assert torch.equal(dH, want[0]) and torch.equal(dW, want[1])
    for b in (hb, wb):
        assert b[:64].isnan().all() and b[-64:].isnan().all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_offsets_beyond_32_bits(t):
    """2.25e9 elements of H, of which the last tokens alone have a gradient."""
    N, d, V, last = 2_200_000, 1024, 40, 200
    H = torch.empty(N, d, dtype=TYPES[t], device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    i = inputs(last, d, V, t, seed=2)
    H[-last:] = i["H"]
    y, g = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.zeros(N, device="cuda")
    y[-last:], g[-last:] = i["y"], i["g"]
    lp, lse = gp.grpo_logprobs_fwd(H, i["W"], y, 1 << 20)
    dH, dW = gp.grpo_logprobs_bwd(H, i["W"], y, lp, lse, g, 1 << 20)
    want = plain_update.logprobs(i["H"], i["W"], i["y"], i["g"], half=HALF[t])
    for name, x in (("lp", lp[-last:]), ("dH", dH[-last:]), ("dW", dW)):
        assert ((x.cpu().double() - want[name]).abs() <= want[name + "_tol"]).all(), name
    assert not dH[:-last].any()
