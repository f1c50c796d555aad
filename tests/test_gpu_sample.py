"""Sampling on the GPU against a plain evaluation in float64.  Tokens are equal; a
log-probability is off by its float32 rounding (2^-24 of itself) and by the float64 sums
behind it (below 1e-11)."""
import math

import pytest
import torch

import grpo_policy_loss_amd as gp
from tests import plain_ops

pytestmark = pytest.mark.gpu


def logits(B, V, t=torch.float32, seed=0, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, V, generator=g) * 2.5
    few = max(1, min(9, V // 4))
    x.scatter_add_(1, torch.randint(0, V, (B, few), generator=g), 12 * torch.rand(B, few, generator=g) * torch.rand(B, 1, generator=g))
    if masked:
        off = torch.rand(B, V, generator=g) < masked
        off[:, V // 2] = False
        x[off] = float("-inf")
    return x.to(t), torch.rand(B, generator=g)


def check(x, u, got, **params):
    token, lp = (v.cpu() for v in got)
    for b in range(x.shape[0]):
        row = {k: (v[b].item() if torch.is_tensor(v) else v) for k, v in params.items()}
        want, want_lp = plain_ops.sample(x[b], u[b].item(), **row)
        assert token[b].item() == want, (b, token[b].item(), want, row)
        if want < 0:
            assert lp[b].isnan()
        else:
            assert abs(lp[b].item() - want_lp) <= 2.0 ** -24 * abs(want_lp) + 1e-11


def run(x, u, T=1.0, k=0, p=1.0, min_p=0.0):
    dev = lambda v: v.cuda() if torch.is_tensor(v) else v  # noqa: E731
    return gp.grpo_sample(x.cuda(), u.cuda(), temperature=dev(T), top_k=dev(k), top_p=dev(p), min_p=dev(min_p))


PARAMS = [dict(), dict(T=0.6), dict(k=1), dict(k=7), dict(p=0.9), dict(p=0.05), dict(min_p=0.1),
          dict(k=50, p=0.95), dict(T=0.7, k=40, p=0.8, min_p=0.02), dict(T=1.7, k=3000, p=0.99),
          dict(p=0.999, min_p=1e-6), dict(T=5.0, p=0.7), dict(T=0.01, k=5)]


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 5, 64, 511, 513, 4096, 10007, 151936])
@pytest.mark.parametrize("params", PARAMS, ids=str)
def test_tokens(V, t, params):
    x, u = logits(4, V, t, seed=V, masked=0.02 if V > 4 else 0)
    check(x, u, run(x, u, **params), **params)


def test_parameters_of_each_row():
    B, V = 40, 5003
    x, u = logits(B, V, masked=0.3)
    g = torch.Generator().manual_seed(5)
    params = dict(T=0.2 + torch.rand(B, generator=g), k=torch.randint(0, 60, (B,), generator=g, dtype=torch.int32),
                  p=torch.rand(B, generator=g), min_p=torch.rand(B, generator=g) * 0.1)
    params["k"][3], params["p"][4], params["min_p"][5], params["T"][6] = -1, 1.5, -0.5, 0.0   # off
    params["min_p"][7] = 3.0                                                             # counts as 1
    params["k"][8] = V + 9
    check(x, u, run(x, u, **params), **params)
    params["p"][9] = params["min_p"][9] = float("nan")                                     # off
    got = run(x, u, **params)
    params["p"][9] = params["min_p"][9] = 0.0
    check(x, u, got, **params)


@pytest.mark.parametrize("params", [dict(), dict(k=300), dict(p=0.5), dict(p=0.30001, k=700), dict(k=1), dict(min_p=1.0)], ids=str)
@pytest.mark.parametrize("V", [1000, 40000])
def test_equal_logits_go_by_index(V, params):
    x = torch.full((6, V), 1.25)
    x[1] = -0.0
    x[1, ::2] = 0.0                        # minus zero equals zero
    x[2, 17:] = -3.0
    x[3] = torch.arange(V).remainder(3).float()
    x[4] = float("-inf")
    x[4, V - 3:] = 0.5
    x[5, V // 2:] = 1.25 + 2.0 ** -20
    u = torch.tensor([0.0, 0.5, 0.25, 0.75, 0.99, 0.123])
    check(x, u, run(x, u, **params), **params)


@pytest.mark.parametrize("params", [dict(), dict(k=5), dict(p=0.9), dict(min_p=0.3)], ids=str)
def test_rows_without_a_distribution(params):
    x, u = logits(6, 3001)
    x[1, 7] = float("nan")
    x[2, 3000] = float("inf")
    x[3] = float("-inf")
    x[4, :] = float("-inf")
    x[4, 1234] = -50.0                     # one token left
    got = run(x, u, **params)
    check(x, u, got, **params)
    assert got[0].tolist()[1:5] == [-1, -1, -1, 1234] and got[1][4] == 0


def test_device_temperatures_out_of_range():
    x, u = logits(5, 300)
    T = torch.tensor([-1.0, float("nan"), float("inf"), 1e-30, 1e30])
    check(x, u, run(x, u, T=T), T=T)


def test_temperatures_near_zero_and_large_top_k():
    x, u = logits(3, 900)
    for T in (1e-300, 1e-310, 5e-324):
        token, lp = run(x, u, T=T)
        assert token.tolist() == x.argmax(1).tolist() and not lp.any()
    check(x, u, run(x, u, k=2**32 + 5))
    with pytest.raises(gp.GrpoError, match="top_k"):
        run(x, u, k=-2**32 + 5)


def test_bounds_of_u():
    x, _ = logits(6, 2000, masked=0.5)
    x[:, :5] = x[:, -5:] = float("-inf")
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, -3.0, 7.0, 0.5])
    for params in (dict(), dict(k=20), dict(p=0.9)):
        got = run(x, u, **params)
        check(x, u, got, **params)
        assert got[0][1] == got[0][1] and (x.gather(1, got[0].cpu().long()[:, None]) > float("-inf")).all()


def test_the_largest_u_reaches_the_last_token_that_weighs_enough():
    """Of two tokens with weights 1 and w: (1 - 2^-24)(1 + w) is above 1, the first one's mass, for
    w = 2^-20, and below it for w = 2^-30."""
    x = torch.full((4, 2000), float("-inf"))
    x[:, 3] = 0.0
    x[:, 1990] = torch.tensor([2.0 ** -20, 2.0 ** -30] * 2).log()
    u = torch.full((4,), 1.0 - 2.0 ** -24)
    for params in (dict(), dict(k=20), dict(p=0.9999999), dict(min_p=2.0 ** -40)):
        got = run(x, u, **params)
        assert got[0].tolist() == [1990, 3, 1990, 3]
        check(x, u, got, **params)


def test_far_apart_logits():
    """Weights far below the largest one: none of them is drawn, none disturbs."""
    x = torch.full((3, 4000), -1e30)
    x[0, 5], x[0, 6] = 3.0, 2.0
    x[1, ::7] = 3e38
    x[2] = torch.linspace(-3e38, 3e38, 4000)
    u = torch.tensor([0.9, 0.5, 0.99])
    for params in (dict(), dict(k=3), dict(p=0.99), dict(k=2000, p=0.5), dict(T=1e-3)):
        check(x, u, run(x, u, **params), **params)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e30, "lowest"])
@pytest.mark.parametrize("V", [50, 4000, 70001])
def test_tokens_without_weight_are_not_drawn(V, mask, t):
    """Finite masks, in front of the drawable tokens and behind them, and the bounds of u: where u
    is 0 the first token of any weight is drawn, where it is 1 the last."""
    g = torch.Generator().manual_seed(V)
    x = torch.full((7, V), torch.finfo(t).min if mask == "lowest" else mask)
    for b in range(7):
        at = torch.randperm(V - 20, generator=g)[:b + 1] + 10     # never the first or last ten
        x[b, at] = 2 * torch.randn(b + 1, generator=g)
    x = x.to(t)
    u = torch.tensor([0.0, 1.0, 0.0, 1.0 - 2.0 ** -24, -1.0, 3.0, 0.0])
    off = torch.ones(7)
    for params in (dict(), dict(T=0.5), dict(T=off * 0.5), dict(p=off), dict(p=0.9), dict(k=5)):
        check(x, u, run(x, u, **params), **params)


def test_bounds_of_u_at_temperatures_near_zero():
    x, _ = logits(6, 5000)
    u = torch.tensor([0.0, 1.0, 0.0, 1.0 - 2.0 ** -24, -1.0, 0.5])
    check(x, u, run(x, u, T=1e-3), T=1e-3)      # where weights of e^-428 and e^-600 are left
    for T in (1e-30, 1e-300, torch.full((6,), 1e-30)):
        token, lp = run(x, u, T=T)
        assert token.tolist() == x.argmax(1).tolist() and not lp.any()


def test_rows_that_lie_apart_and_any_alignment():
    for t in (torch.float32, torch.bfloat16):
        x, u = logits(7, 1999, t)
        wide = torch.full((7, 2101), 99.0, dtype=t, device="cuda")
        wide[:, 1:2000] = x.cuda()
        for params in (dict(), dict(k=30, p=0.9)):
            got = gp.grpo_sample(wide[:, 1:2000], u.cuda(), top_k=params.get("k", 0), top_p=params.get("p", 1.0))
            check(x, u, got, **params)
    x, u = logits(1, 50)
    got = gp.grpo_sample(x.cuda(), u.cuda())
    check(x, u, got)


def test_largest_vocabulary_and_row_offsets_beyond_32_bits():
    V = 1 << 20
    x, u = logits(2, V)
    for params in (dict(), dict(k=100, p=0.9), dict(p=0.95)):
        check(x, u, run(x, u, **params), **params)
    # two rows 2^31 + 64 elements apart
    far = torch.empty((1 << 31) + 64 + 1000, dtype=torch.bfloat16, device="cuda")
    x, u = logits(2, 1000, torch.bfloat16)
    rows = far.as_strided((2, 1000), ((1 << 31) + 64, 1))
    rows.copy_(x)
    check(x, u, gp.grpo_sample(rows, u.cuda(), top_k=20), k=20)


def test_many_rows():
    x, u = logits(3000, 37)
    check(x, u, run(x, u, k=5, p=0.9), k=5, p=0.9)
    x, u = logits(66000, 9)                 # more than one batch of rows
    token, lp = (v.cpu() for v in run(x, u, k=4))
    some = torch.arange(0, 66000, 997)
    some[-1] = 65999
    check(x[some], u[some], (token[some], lp[some]), k=4)
    x, u = logits(1100, 4100)
    params = dict(p=torch.linspace(0.3, 1.0, 1100), min_p=torch.linspace(0, 1e-3, 1100))
    token, lp = (v.cpu() for v in run(x, u, **params))
    some = torch.tensor([0, 1, 511, 1022, 1023, 1024, 1025, 1099])
    check(x[some], u[some], (token[some], lp[some]), **{k: v[some] for k, v in params.items()})


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 2, 63, 1000, 2047, 2048, 2049])
def test_every_size_of_the_candidates(k, t):
    for V in (4095, 4096, 4097, 70001):
        for p in (1.0, 0.97):
            x, u = logits(3, V, t, seed=k)
            x[1] = x[1].sort(descending=True).values     # all candidates side by side
            check(x, u, run(x, u, k=k, p=p), k=k, p=p)


@pytest.mark.parametrize("V", [5003, 40000, 270000])
@pytest.mark.parametrize("params", [dict(k=4000), dict(k=4000, min_p=0.01), dict(k=4000, p=0.9), dict(k=1500), dict(k=2049, T=3.0)], ids=str)
def test_rows_with_fewer_tokens_than_k(V, params):
    x, u = logits(5, V)
    for b, left in enumerate((1, 2, 300, 1400, 2040)):
        off = torch.ones(V, dtype=torch.bool)
        off[torch.randperm(V, generator=torch.Generator().manual_seed(b))[:left]] = False
        x[b, off] = float("-inf")
    check(x, u, run(x, u, **params), **params)
    rows = dict(params, k=torch.full((5,), params["k"], dtype=torch.int32))
    check(x, u, run(x, u, **rows), **rows)


@pytest.mark.parametrize("p", [0.01, 0.5, 0.9, 0.9999999])
@pytest.mark.parametrize("scale", [0.0, 0.01, 1.0, 8.0])
def test_nucleus_of_flat_and_peaked_rows(scale, p):
    for t in (torch.float32, torch.bfloat16):
        g = torch.Generator().manual_seed(11)
        x = (torch.randn(5, 50021, generator=g) * scale + 3).to(t)
        x[1, 100:] = float("-inf")
        x[2, ::2] = x[2, 0]
        u = torch.rand(5, generator=g)
        check(x, u, run(x, u, p=p, min_p=1e-4), p=p, min_p=1e-4)


def test_log_probability_is_the_loss_s():
    """lp is what the loss gives for the drawn token at the same temperature."""
    g = torch.Generator(device="cuda").manual_seed(0)
    H, W = torch.randn(64, 32, generator=g, device="cuda"), torch.randn(500, 32, generator=g, device="cuda") * 0.2
    token, lp = gp.grpo_sample(gp.grpo_gemm_nt(H, W), torch.rand(64, generator=g, device="cuda"), temperature=0.75)
    got = gp.grpo_ref_logprobs(H, W, token, opts={"temperature": 0.75})
    assert (lp - got).abs().max() <= 1e-5 * lp.abs().max()


def test_repeatable_and_on_two_streams_at_once():
    x, u = logits(64, 20011)
    x, u = x.cuda(), u.cuda()
    want = gp.grpo_sample(x, u, top_k=500, top_p=0.95)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(gp.grpo_sample(x, u, top_k=500, top_p=0.95))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def test_captured_graphs_with_one_workspace():
    x, u = logits(8, 20011)
    x, u = x.cuda(), u.cuda()
    k = torch.full((8,), 40, dtype=torch.int32, device="cuda")
    ws = torch.full((gp.lib().grpo_sample_workspace_bytes(8, 20011),), 255, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for params in (dict(top_k=k, top_p=0.9), dict()):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append((gp.grpo_sample(x, u, workspace=ws, **params), params))
    for seed in (3, 4, 5, 6):
        nx, nu = logits(8, 20011, seed=seed)
        x.copy_(nx)
        u.copy_(nu)
        k.fill_(seed * 10)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        ws.fill_(seed)
        for got, params in outs:
            want = gp.grpo_sample(x, u, **params)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        check(nx, nu, outs[0][0], k=seed * 10, p=0.9)


def test_out_tensors_and_refusals():
    x, u = logits(4, 100)
    token, lp = torch.full((6,), -7, dtype=torch.int32, device="cuda"), torch.full((6,), 5.0, device="cuda")
    gp.grpo_sample(x.cuda(), u.cuda(), out=(token[1:5], lp[1:5]))
    check(x, u, (token[1:5], lp[1:5]))
    assert token[0] == token[5] == -7 and lp[0] == lp[5] == 5
    with pytest.raises(gp.GrpoError, match="top_p"):
        gp.grpo_sample(x.cuda(), u.cuda(), top_p=1.01)
    with pytest.raises(gp.GrpoError, match="temperature"):
        gp.grpo_sample(x.cuda(), u.cuda(), temperature=math.inf)
    with pytest.raises(ValueError, match="on the GPU"):
        gp.grpo_sample(x, u.cuda())
