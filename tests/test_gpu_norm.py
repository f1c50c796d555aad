"""Norm forward and backward on the GPU against the formulas in float64.

Tolerances count roundings of u = 2^-24 (float32 arithmetic) and of half the element
type's eps for each stored element.  A float32 sum over a row passes at most
K = 64 + cols / 1024 additions per term (32 in a lane, then lanes, waves and the
passes of a long row), a sum over the rows at most KR = 128 + rows / 64."""
import pytest
import torch

import grpo_policy_loss_amd as gp
from tests import plain_ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
KINDS = {"layer": gp.NORM_LAYER, "rms": gp.NORM_RMS}


def inputs(rows, cols, t, seed=0, offset=0):
    """Rows of different size with a mean, `offset` elements into their buffers."""
    g = torch.Generator().manual_seed(seed)
    def rnd(*shape):
        return torch.randn(*shape, generator=g)
    def place(v):
        flat = torch.empty(v.numel() + offset, dtype=t, device="cuda")
        flat[offset:] = v.to(t).flatten().cuda()
        return flat[offset:].view(v.shape)
    x = rnd(rows, cols) * (0.2 + rnd(rows, 1).abs()) + rnd(rows, 1)
    return dict(x=place(x), w=place(1 + 0.2 * rnd(cols)), b=place(rnd(cols)),
                dy=place(rnd(rows, cols)))


def check_fwd(i, y, mean, rstd, bias, layer):
    rows, cols = i["x"].shape
    K = 64 + cols / 1024
    x, w, b = (i[k].cpu() for k in ("x", "w", "b"))
    want, mu, r = plain_ops.norm_fwd(x, w, b if bias else None, EPS, layer)
    ut = torch.finfo(x.dtype).eps / 2
    size = x.double().abs().mean(1) if layer else torch.zeros(rows, dtype=torch.float64)
    if layer:
        assert ((mean.cpu().double() - mu).abs() <= K * U * size + 1e-300).all()
    else:
        assert mean is None
    # the centred sum's relative error and the mean's shift of every centred value
    shift = K * U * size * r
    rel = 2 * K * U + shift
    assert ((rstd.cpu().double() - r).abs() <= r * rel).all()
    wide = w.double().abs()[None, :]
    tol = ut * want.abs() + (want.abs() + (b.double().abs() if bias else 0)) * (rel[:, None] + 4 * U) * 2 \
        + (shift[:, None] + 2 * U * x.double().abs() * r[:, None]) * wide
    assert ((y.cpu().double() - want).abs() <= tol + 1e-30).all()


def check_bwd(i, mean, rstd, dx, dw, db, layer, bias, dw0=0.0):
    rows, cols = i["x"].shape
    K, KR = 64 + cols / 1024, 128 + rows / 64
    x, w, dy = (i[k].cpu() for k in ("x", "w", "dy"))
    mu = mean.cpu() if layer else None
    want, want_w, want_b = plain_ops.norm_bwd(dy, x, w, mu, rstd.cpu(), layer)
    ut = torch.finfo(x.dtype).eps / 2
    r = rstd.cpu().double()[:, None]
    xh = (x.double() - (mu.double()[:, None] if layer else 0)) * r
    g = (dy.double() * w.double()).abs()
    size = g + xh.abs() * (g * xh.abs()).mean(1, keepdim=True) + (g.mean(1, keepdim=True) if layer else 0)
    tol = ut * want.abs() + (K + 8) * U * r * size
    assert ((dx.cpu().double() - want).abs() <= tol + 1e-30).all()
    tol_w = KR * U * ((dy.double() * xh).abs().sum(0) + abs(dw0))
    assert ((dw.cpu().double() - dw0 - want_w).abs() <= tol_w + 1e-30).all()
    if bias:
        assert ((db.cpu().double() - want_b).abs() <= KR * U * dy.double().abs().sum(0) + 1e-30).all()
    else:
        assert db is None


COLS = [1, 2, 7, 16, 33, 128, 129, 511, 512, 1000, 1537, 2048, 2880, 4096, 4097, 8192, 16384, 16387,
        40000]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_both_directions(cols, t, kind):
    for rows in (1, 5, 1300 if cols <= 4097 else 70):
        for bias in (False, True):
            i = inputs(rows, cols, t, seed=rows)
            y, mean, rstd = gp.grpo_norm_fwd(i["x"], i["w"], i["b"] if bias else None, EPS, KINDS[kind])
            check_fwd(i, y, mean, rstd, bias, kind == "layer")
            dx, dw, db = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, KINDS[kind], bias)
            check_bwd(i, mean, rstd, dx, dw, db, kind == "layer", bias)


# more rows than the grid takes at once: the forward's 2048 blocks of 64, 16, 4 or 1 rows (by
# the lanes of a row), the backward's 256 to 1024, and the last turn not full
@pytest.mark.parametrize("rows,cols", [(140003, 7), (33333, 100), (9001, 500), (9001, 900), (5003, 1537),
                                       (5003, 2880), (2300, 4096), (2100, 8192), (2100, 16384), (2100, 16387)])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_blocks_that_take_several_turns_of_rows(rows, cols, t):
    for kind in ("layer", "rms") if cols <= 1537 else ("layer",) if t == torch.float32 else ("rms",):
        i = inputs(rows, cols, t, seed=cols)
        bias = kind == "layer"
        y, mean, rstd = gp.grpo_norm_fwd(i["x"], i["w"], i["b"] if bias else None, EPS, KINDS[kind])
        check_fwd(i, y, mean, rstd, bias, bias)
        dx, dw, db = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, KINDS[kind], bias)
        check_bwd(i, mean, rstd, dx, dw, db, bias, bias)


@pytest.mark.parametrize("rows,cols", [(1041000, 2064), (131100, 16400)])
def test_offsets_beyond_32_bits(rows, cols):
    """Rows from 2^31 elements on, whose gradient alone is not zero."""
    assert (rows - 20) * cols > 1 << 31
    last = 16
    i = inputs(last, cols, torch.bfloat16)
    x, dy = (torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[:, ::3] = 1.0
    x[-last:], dy[-last:] = i["x"], i["dy"]
    y, mean, rstd = gp.grpo_norm_fwd(x, i["w"], i["b"], EPS, gp.NORM_LAYER)
    check_fwd(i, y[-last:], mean[-last:], rstd[-last:], True, True)
    assert torch.equal(y[0], y[rows - last - 1])
    dx, dw, db = gp.grpo_norm_bwd(dy, x, i["w"], mean, rstd, gp.NORM_LAYER, True)
    check_bwd(i, mean[-last:], rstd[-last:], dx[-last:], dw, db, True, True)
    assert not dx[:-last].any()


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [24, 1536, 20000])
def test_any_element_alignment(t, cols):
    i = inputs(37, cols, t, offset=1)
    y, mean, rstd = gp.grpo_norm_fwd(i["x"], i["w"], i["b"], EPS, gp.NORM_LAYER)
    check_fwd(i, y, mean, rstd, True, True)
    check_bwd(i, mean, rstd, *gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, gp.NORM_LAYER, True),
              True, True)


def test_a_mean_far_above_the_deviation():
    i = inputs(9, 4096, torch.float32)
    i["x"] += 1000.0
    y, mean, rstd = gp.grpo_norm_fwd(i["x"], i["w"], None, EPS, gp.NORM_LAYER)
    check_fwd(i, y, mean, rstd, False, True)


def test_gradients_are_accumulated_and_bitwise_repeatable():
    i = inputs(3000, 1537, torch.bfloat16)
    _, mean, rstd = gp.grpo_norm_fwd(i["x"], i["w"], i["b"], EPS, gp.NORM_LAYER)
    runs = [gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, gp.NORM_LAYER, True) for _ in range(3)]
    for a in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(a, runs[0]))
    dw, db = torch.full((1537,), 3.0, device="cuda"), torch.full((1537,), -2.0, device="cuda")
    ws = torch.full((gp.lib().grpo_norm_workspace_bytes(3000, 1537, 1),), 255, dtype=torch.uint8, device="cuda")
    dx = torch.full_like(i["x"], float("nan"))
    out = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, gp.NORM_LAYER, dX=dx, dweight=dw, dbias=db,
                           workspace=ws)
    assert out[0] is dx and out[1] is dw and out[2] is db
    assert torch.equal(dx, runs[0][0])
    assert torch.equal(dw, 3.0 + runs[0][1]) and torch.equal(db, -2.0 + runs[0][2])
    # one accumulator given: the other starts at zero
    dw = torch.full((1537,), 3.0, device="cuda")
    out = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, gp.NORM_LAYER, bias=True, dweight=dw)
    assert torch.equal(dw, 3.0 + runs[0][1]) and torch.equal(out[2], runs[0][2])


def test_nan_and_infinite_values_stay_in_their_row():
    for kind in KINDS.values():
        i = inputs(40, 600, torch.float32)
        clean, cm, cr = gp.grpo_norm_fwd(i["x"], i["w"], None, EPS, kind)
        dclean, _, _ = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], cm, cr, kind)
        i["x"][7, 3], i["x"][21, 599] = float("nan"), float("inf")
        y, mean, rstd = gp.grpo_norm_fwd(i["x"], i["w"], None, EPS, kind)
        dx, _, _ = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, kind)
        ok = torch.ones(40, dtype=torch.bool, device="cuda")
        ok[7] = ok[21] = False
        assert torch.equal(y[ok], clean[ok]) and torch.equal(dx[ok], dclean[ok])
        assert y[7].isnan().all() and y[21, 599].isnan() and dx[7].isnan().all()


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [3, 50, 100, 300, 1000, 1537, 3000, 5000, 12000, 16387])
def test_a_mean_whose_normalised_value_leaves_float32(cols, t):
    """Every element is its row's mean, 2^121 with rstd 2^8: no real column leaves float32's
    range, but (0 - mean) rstd would, where lanes lie behind the row's end."""
    i = inputs(5, cols, t)
    i["x"].fill_(2.0 ** 121)
    mean, rstd = torch.full((5,), 2.0 ** 121, device="cuda"), torch.full((5,), 256.0, device="cuda")
    for bias in (False, True):
        dx, dw, db = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, gp.NORM_LAYER, bias)
        check_bwd(i, mean, rstd, dx, dw, db, True, bias)


def test_rows_of_zeros_and_constants():
    x = torch.zeros(3, 256, device="cuda")
    x[1] = 5.0
    w, b = torch.full((256,), 2.0, device="cuda"), torch.full((256,), 0.5, device="cuda")
    y, mean, rstd = gp.grpo_norm_fwd(x, w, b, EPS, gp.NORM_LAYER)
    assert (y == 0.5).all() and mean.tolist() == [0.0, 5.0, 0.0]
    y, _, rstd = gp.grpo_norm_fwd(x, w, None, EPS, gp.NORM_RMS)
    assert (y[0] == 0).all() and torch.allclose(y[1], torch.full_like(y[1], 2.0), atol=1e-5)
    assert abs(rstd[0].item() - EPS ** -0.5) < 1e-4


def test_gradients_against_differences():
    """The gradient of sum(y c), against central differences of the float64 forward:
    the difference's own error is h^2 times a third derivative (values here are of
    order one, h = 1e-4) plus 2^-52 / h, below 1e-7; the float32 gradient is off by at
    most (K + 8) U times a few values of order one, 1e-5."""
    for kind, k in KINDS.items():
        g = torch.Generator().manual_seed(3)
        x, w, b, c = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((4, 24), (24,), (24,), (4, 24)))
        x, w, b, c = (v.float() for v in (x, w, b, c))
        leaves = [v.cuda().requires_grad_() for v in (x, w, b)]
        (gp.grpo_norm(*leaves, EPS, k) * c.cuda()).sum().backward()
        def f(*a):
            return (plain_ops.norm_fwd(*a, EPS, kind == "layer")[0] * c.double()).sum()
        h = 1e-4
        for n, leaf in enumerate(leaves):
            args = [v.double() for v in (x, w, b)]
            for j in range(0, args[n].numel(), 5):
                at = []
                for sign in (h, -h):
                    moved = [v.clone() for v in args]
                    moved[n].view(-1)[j] += sign
                    at.append(f(*moved))
                want = ((at[0] - at[1]) / (2 * h)).item()
                got = leaf.grad.view(-1)[j].item()
                assert abs(got - want) <= 1e-5 * (1 + abs(want)), (kind, n, j, got, want)


def test_autograd_takes_broadcast_gradients_and_skips_what_is_not_needed():
    i = inputs(70, 513, torch.bfloat16)
    x, w = i["x"].clone().requires_grad_(), i["w"].clone().requires_grad_()
    gp.grpo_norm(x, w, None, EPS).sum().backward()      # an expanded gradient of ones
    one = torch.ones_like(i["x"])
    _, _, rstd = gp.grpo_norm_fwd(i["x"], i["w"], None, EPS)
    dx, dw, _ = gp.grpo_norm_bwd(one, i["x"], i["w"], None, rstd)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw.bfloat16())
    y = gp.grpo_norm(i["x"], w.detach().requires_grad_(), i["b"], EPS, gp.NORM_LAYER)
    y.backward(i["dy"])
    w2 = i["w"].clone().view(1, -1).requires_grad_()     # a weight of another shape
    gp.grpo_norm(i["x"], w2, None, EPS).backward(i["dy"])
    assert w2.grad.shape == (1, 513)
    x = i["x"].clone().requires_grad_()
    gp.grpo_norm(x.t().contiguous().t().contiguous(), i["w"], None, EPS).backward(i["dy"].t().contiguous().t())
    assert x.grad.isfinite().all()


def test_another_stream_and_a_captured_graph():
    i = inputs(513, 1536, torch.bfloat16)
    _, mean, rstd = gp.grpo_norm_fwd(i["x"], i["w"], i["b"], EPS, gp.NORM_LAYER)
    want = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, gp.NORM_LAYER, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], mean, rstd, gp.NORM_LAYER, True)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, m2, r2 = gp.grpo_norm_fwd(i["x"], i["w"], i["b"], EPS, gp.NORM_LAYER)
        out = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], m2, r2, gp.NORM_LAYER, True)
    for seed in (5, 6, 7):
        new = inputs(513, 1536, torch.bfloat16, seed=seed)
        for k in ("x", "dy"):
            i[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        ey, em, er = gp.grpo_norm_fwd(i["x"], i["w"], i["b"], EPS, gp.NORM_LAYER)
        eager = gp.grpo_norm_bwd(i["dy"], i["x"], i["w"], em, er, gp.NORM_LAYER, True)
        assert torch.equal(y, ey) and all(torch.equal(a, b) for a, b in zip(out, eager))


def test_a_captured_backward_of_autograd_is_refused(monkeypatch):
    i = inputs(8, 64, torch.float32)
    x = i["x"].clone().requires_grad_()
    y = gp.grpo_norm(x, i["w"], None, EPS)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="grpo_norm_bwd"):
        y.backward(i["dy"])
    monkeypatch.undo()
    gp.grpo_norm(x, i["w"], None, EPS).backward(i["dy"])
    assert x.grad.isfinite().all()


def test_refusals_on_the_gpu():
    i = inputs(8, 64, torch.float32)
    with pytest.raises(ValueError, match="contiguous"):
        gp.grpo_norm_fwd(i["x"].t(), torch.ones(8, device="cuda"))
    with pytest.raises(ValueError, match="on the GPU"):
        gp.grpo_norm_fwd(i["x"], i["w"].cpu())
    with pytest.raises(gp.GrpoError, match="eps"):
        gp.grpo_norm_fwd(i["x"], i["w"], eps=-1.0)
    with pytest.raises(gp.GrpoError, match="kind"):
        gp.grpo_norm_fwd(i["x"], i["w"], kind=5)
