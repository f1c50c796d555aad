"""The gradients' norm, the clipping factor and clipping in place on the GPU.

Squares and sums are float64 (2^-53 each, some 10^7 of them: 10^-9 in all), so the float32 results
are within one rounding, U = 2^-24 relative, and 2^-26 for what float64 leaves."""
import math

import pytest
import torch

import grpo_policy_loss_amd as gp
from tests import plain_update

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"f": torch.float32, "b": torch.bfloat16}


def tensors(sizes, seed=0, packed=False, scale=1e-2):
    """sizes: "f1000 b37 ...": float32 or bfloat16 tensors, packed at any offset of one buffer or apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for s in sizes.split():
        t, n = TYPES[s[0]], int(s[1:])
        out.append((scale * torch.randn(n, generator=g, device="cuda")).to(t))
    if packed:
        for t in TYPES.values():
            mine = [i for i, x in enumerate(out) if x.dtype == t]
            flat = torch.zeros(sum(out[i].numel() for i in mine) + 1, dtype=t, device="cuda")
            at = 1
            for i in mine:
                view = flat[at:at + out[i].numel()]
                view.copy_(out[i])
                out[i], at = view, at + view.numel()
    return out


def check(grads, max_norm=1.0):
    plan = gp.grad_plan(grads)
    for kind in (gp.GRAD_NORM_L2, gp.GRAD_NORM_MAX):
        want = plain_update.grad_norm(grads, kind == gp.GRAD_NORM_MAX)
        norm, scale = gp.grpo_grad_norm(plan, max_norm, kind)
        assert abs(norm.item() - want) <= 1.25 * U * want
        factor = min(1.0, max_norm / (want + 1e-6)) if max_norm else 1.0
        assert abs(scale.item() - factor) <= 1.25 * U * factor
    return plan, scale


SIZES = ["f1", "b1", "f0 b7 f0", "f3 b5", "f8192", "f8193 b8191", "f1536 f1536", "b20000 f100 b3 f70001", "f131072", "f131073",
         "b131072 b131073 f5", " ".join(["f257", "b100"] * 40), " ".join(["b1"] * 3000 + ["f9000"]), "f30000000", "b40000003 f7"]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("packed", [False, True])
def test_norm_and_clipping(sizes, packed):
    grads = tensors(sizes, packed=packed)
    for max_norm in (0.0, 1e-3, 1e6):
        check(grads, max_norm)
    plan, scale = check(grads, 0.01)
    want = [(x.float() * scale).to(x.dtype) for x in grads]
    versions = [x._version for x in grads]
    gp.grpo_grad_clip(plan, scale)
    for x, w, v in zip(grads, want, versions):
        assert torch.equal(x, w) and x._version > v
    before = [x.clone() for x in grads]
    gp.grpo_grad_clip(plan, torch.ones(1, device="cuda"))
    assert all(torch.equal(x, w) for x, w in zip(grads, before))


def test_neighbours_are_left_alone():
    for t in TYPES.values():
        flat = torch.full((40000,), 3.0, dtype=t, device="cuda")
        grads = [flat[1:6], flat[7:9000], flat[9001:30001]]
        plan = gp.grad_plan(grads)
        gp.grpo_grad_clip(plan, torch.full((1,), 0.5, device="cuda"))
        keep = torch.ones(40000, dtype=torch.bool, device="cuda")
        keep[1:6] = keep[7:9000] = keep[9001:30001] = False
        assert (flat[keep] == 3).all() and (flat[~keep] == 1.5).all()


@pytest.mark.parametrize("t", list(TYPES.values()))
@pytest.mark.parametrize("n", [100, 300000])
def test_values_that_float32_squares_lose(t, n):
    for size in (1e25, 1e-25):
        check([torch.full((n,), size, device="cuda").to(t), torch.zeros(5, device="cuda")], size)


@pytest.mark.parametrize("n", [50, 200000])
@pytest.mark.parametrize("t", list(TYPES.values()))
def test_infinities_and_nan(n, t):
    for value, norm_is, scale_is in ((math.inf, math.inf, 0.0), (-math.inf, math.inf, 0.0), (math.nan, math.nan, math.nan)):
        g = torch.ones(n, device="cuda").to(t)
        g[n // 2] = value
        plan = gp.grad_plan([torch.ones(3, device="cuda"), g])
        for kind in (gp.GRAD_NORM_L2, gp.GRAD_NORM_MAX):
            norm, scale = gp.grpo_grad_norm(plan, 2.0, kind)
            same = lambda a, b: a == b or (math.isnan(a) and math.isnan(b))  # noqa: E731
            assert same(norm.item(), norm_is) and same(scale.item(), scale_is)
            assert gp.grpo_grad_norm(plan, 0.0, kind)[1].item() == 1.0


def test_nothing():
    for grads in ([torch.zeros(0, device="cuda")], [torch.zeros(100, device="cuda"), torch.zeros(0, dtype=torch.bfloat16, device="cuda")]):
        plan = gp.grad_plan(grads)
        norm, scale = gp.grpo_grad_norm(plan, 1.0)
        assert norm.item() == 0 and scale.item() == 1
        gp.grpo_grad_clip(plan, scale)


def test_beyond_32_bits():
    """A tensor of more than 2^32 elements: only its last and its first are not 0."""
    n = (1 << 32) + 5000
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[0], g[-1], g[1 << 31] = 3.0, 4.0, 12.0
    plan = gp.grad_plan([g])
    norm, scale = gp.grpo_grad_norm(plan, 6.5)
    assert norm.item() == 13.0
    gp.grpo_grad_clip(plan, scale)
    assert g[0].item() == 1.5 and g[-1].item() == 2.0 and g[1 << 31].item() == 6.0


def test_shared_memory_is_refused():
    x = torch.zeros(100, device="cuda")
    with pytest.raises(gp.GrpoError, match="overlap"):
        gp.grad_plan([x, x])
    with pytest.raises(gp.GrpoError, match="overlap"):
        gp.grad_plan([x[:60], x[50:]])
    plan = gp.grad_plan([x[:50], x[50:]])
    assert plan.holds([x[:50], x[50:]]) and not plan.holds([x[:50]]) and not plan.holds([x[:50], None])
    assert not plan.holds([x[:50], x[50:].clone()])


def test_captured_with_the_optimizer():
    """Norm, factor and AdamW's step replayed against the same calls made eagerly."""
    params, grads = tensors("f5000 f300", 1), tensors("f5000 f300", 2, scale=1.0)
    m, v = gp.adamw_moments(params)
    plan, gplan = gp.adamw_plan(params, grads, m, v), gp.grad_plan(grads)
    state = [*params, *m, *v]
    start = [t.clone() for t in state]

    def once():
        norm, scale = gp.grpo_grad_norm(gplan, 0.5)
        gp.grpo_adamw(plan, 1, lr=1e-2, grad_scale=scale)
        return norm, scale
    wants = []
    for k in range(4):
        grads[0].mul_(2.0 ** k)
        norm, scale = once()
        wants.append([norm.clone(), scale.clone(), *(t.clone() for t in state)])
        grads[0].div_(2.0 ** k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, scale = once()
    for t, s in zip(state, start):
        t.copy_(s)
    for k in range(4):
        grads[0].mul_(2.0 ** k)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([norm, scale, *state], wants[k]):
            assert torch.equal(a, b)
        grads[0].div_(2.0 ** k)


def test_two_calls_on_two_streams():
    grads = tensors("f900000 b70000 f3")
    plan = gp.grad_plan(grads)
    want = gp.grpo_grad_norm(plan, 1.0)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for s in sides:
            with torch.cuda.stream(s):
                got.append(gp.grpo_grad_norm(plan, 1.0))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
