"""Refusals of the log-probabilities with a gradient, the clipped policy loss and the preference
loss, on the host: the C ABI's argument checks (no call here gets past them) and the binding's
checks of types, shapes and devices."""
import ctypes
import os
import re

import pytest
import torch

gp = pytest.importorskip("grpo_policy_loss_amd")
from grpo_policy_loss_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libgrpo.so not built", allow_module_level=True)

L = _lib.lib()
FAKE = ctypes.c_void_p(0x1000)     # never dereferenced
FAKE2, FAKE3 = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)
BIG = (1 << 31) - 1


def logprobs_fwd(**kw):
    a = dict(H=FAKE, W=FAKE, y=FAKE, N=8, d=16, V=32, dt=1, chunk=8, opts=None, lp=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return L.grpo_logprobs_fwd(*a.values(), None)


def logprobs_bwd(**kw):
    a = dict(H=FAKE, W=FAKE, y=FAKE, lp=FAKE, lse=FAKE, g=FAKE, N=8, d=16, V=32, dt=1, chunk=8, opts=None, acc=0, dwt=0,
             dH=FAKE2, dW=FAKE3, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return L.grpo_logprobs_bwd(*a.values(), None)


SHAPES = [({"N": 0}, -1), ({"V": -1}, -1), ({"d": 12}, -3), ({"dt": 2}, -1), ({"dt": 0, "d": 6}, -3), ({"chunk": 0}, -1),
          ({"N": 1 << 31}, -3), ({"ws": None}, -2), ({"wsb": 64}, -2), ({"H": None}, -1), ({"W": None}, -1), ({"y": None}, -1),
          ({"lp": None}, -1), ({"lse": None}, -1), ({"H": 0x1008}, -1), ({"W": 0x1002}, -1), ({"ws": 0x1010}, -2)]


@pytest.mark.parametrize("kw,code", SHAPES)
def test_logprobs_forward_argument_errors(kw, code):
    assert logprobs_fwd(**kw) == code
    assert L.grpo_last_error()


@pytest.mark.parametrize("kw,code", SHAPES + [({"g": None}, -1), ({"dH": None, "dW": None}, -1), ({"acc": 2}, -1), ({"dwt": 2}, -1),
                                             ({"dwt": 1, "dt": 0}, -1), ({"dwt": 1, "acc": 1}, -1), ({"dwt": 1, "chunk": 7}, -1),
                                             ({"dH": 0x100004}, -1), ({"dW": 0x100008}, -1), ({"dH": FAKE}, -1), ({"dW": 0x10f0}, -1),
                                             ({"dW": 0x1000 - 2032}, -1), ({"dW": FAKE2}, -1), ({"dH": 0x200000 + 2032}, -1)])
def test_logprobs_backward_argument_errors(kw, code):
    assert logprobs_bwd(**kw) == code
    assert L.grpo_last_error()


def clip(fwd=True, opts=None, **kw):
    a = dict(lp=FAKE, old=None, ref=None, mask=FAKE, adv=FAKE)
    a.update(dict(B=4, L=8, opts=opts, loss=FAKE, stats=FAKE, weights=FAKE, ws=FAKE, wsb=1 << 20) if fwd else
             dict(weights=FAKE, g=None, B=4, L=8, opts=opts, out=FAKE))
    a.update(kw)
    if isinstance(a["opts"], dict):
        a["opts"] = ctypes.pointer(_lib.ClipOpts(**a["opts"]))
    return (L.grpo_clip_loss_fwd if fwd else L.grpo_clip_loss_bwd)(*a.values(), None)


NAN, INF = float("nan"), float("inf")
CLIP = [({k: None}, -1) for k in ("lp", "mask", "adv", "weights")] + \
    [({"B": 0}, -1), ({"L": -1}, -1), ({"B": 1 << 16, "L": 1 << 15}, -3), ({"B": 1 << 40, "L": 1 << 40}, -3)] + \
    [({"opts": o}, -1) for o in (
        {"clip_low": -0.1}, {"clip_low": NAN}, {"clip_high": INF}, {"clip_high": 1e39}, {"clip_dual": 1.0}, {"clip_dual": 0.5},
        {"clip_dual": NAN}, {"beta": NAN}, {"beta": INF}, {"beta": 0.1}, {"ratio": 2}, {"kl_estimator": 3}, {"aggregation": -1},
        {"adv_per_token": 2}, {"adv_per_token": 1, "ratio": 1})]


@pytest.mark.parametrize("kw,code", CLIP + [({"loss": None}, -1), ({"stats": None}, -1), ({"ws": None}, -2), ({"wsb": 16}, -2),
                                            ({"ws": ctypes.c_void_p(0x1010)}, -2)])
def test_clip_forward_argument_errors(kw, code):
    assert clip(**kw) == code
    assert L.grpo_last_error()


@pytest.mark.parametrize("kw,code", CLIP + [({"out": None}, -1)])
def test_clip_backward_argument_errors(kw, code):
    assert clip(False, **kw) == code
    assert L.grpo_last_error()


def pref(**kw):
    a = dict(lp=FAKE, ref=None, mask=FAKE, P=4, L=8, opts={}, loss=FAKE, rewards=FAKE, weights=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    if a["opts"] is not None:
        a["opts"] = ctypes.pointer(_lib.PrefOpts(**{"beta": 0.1, **a["opts"]}))
    return L.grpo_pref_loss_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,code", [({k: None}, -1) for k in ("lp", "mask", "loss", "rewards", "weights", "opts")] + [
    ({"P": 0}, -1), ({"L": 0}, -1), ({"P": 1 << 15, "L": 1 << 15}, -3), ({"P": 1 << 62, "L": 3}, -3), ({"ws": None}, -2),
    ({"wsb": 8}, -2), ({"ws": ctypes.c_void_p(0x1001)}, -2)] + [({"opts": o}, -1) for o in (
        {"beta": 0.0}, {"beta": -1.0}, {"beta": NAN}, {"beta": INF}, {"margin": INF}, {"nll_weight": -1.0}, {"nll_weight": NAN},
        {"kind": 3}, {"kind": -1}, {"label_smoothing": 1.0}, {"label_smoothing": -0.1}, {"label_smoothing": NAN},
        {"label_smoothing": 0.1, "kind": 1}, {"length_mean": 2})])
def test_pref_forward_argument_errors(kw, code):
    assert pref(**kw) == code
    assert L.grpo_last_error()


@pytest.mark.parametrize("at,value,code", [(0, None, -1), (1, None, -1), (5, None, -1), (3, 0, -1), (4, -2, -1), (4, BIG, -3)])
def test_pref_backward_argument_errors(at, value, code):
    a = [FAKE, FAKE, None, 4, 8, FAKE]
    a[at] = value
    assert L.grpo_pref_loss_bwd(*a, None) == code
    assert L.grpo_last_error()


def test_head_workspaces():
    """The loss's forward's, or no tokens x vocabulary beyond a slab of 1.25 GiB, or of 64 tokens; fp8 and bad shapes have
    none."""
    for op in (16, 17):
        assert L.grpo_workspace_bytes(op, 64, 64, 500, 2, 64) == 0 == L.grpo_workspace_bytes(op, 0, 64, 500, 1, 64)
        assert L.grpo_workspace_bytes(op, 64, 62, 500, 0, 64) == 0
    for dt in (0, 1):
        for n, w, v, chunk in ((1, 64, 2, 1), (64, 1536, 151936, 4096), (4096, 1536, 151936, 4096), (163840, 4096, 128256, 8192), (8192, 64, 100, 8192),
                               (1 << 24, 64, 100000, 1 << 20)):
            fwd, bwd = (L.grpo_workspace_bytes(op, n, w, v, dt, chunk) for op in (16, 17))
            c = min(n, chunk)
            assert fwd == L.grpo_workspace_bytes(1, n, w, v, dt, chunk) or dt == 0 and 0 < fwd <= 3 << 30
            assert 0 < bwd <= (5 << 28) + 256 * 4 * v + 64 * c * w + 16 * n + (64 << 20) + 4 * 1024 * 64 * 64 * 8, (n, w, v, dt, bwd)


def test_workspaces_are_bounded():
    """A few thousand partial results at most, or one a row where there are more rows of more than 1024 tokens."""
    for rows in (1, 3, 8, 1021, 4096, 5000, 100003, 1 << 20):
        for length in (1, 5, 64, 1023, 1024, 1025, 4097, 20480, 1 << 20, BIG):
            for f, per, size in ((L.grpo_clip_loss_workspace_bytes, 1, 48), (L.grpo_pref_loss_workspace_bytes, 2, 24)):
                need = f(rows, length)
                if rows * per * length > BIG:
                    assert need == 0
                else:
                    assert 256 <= need <= size * max(4096, rows * per) + 256
    for bad in ((0, 1), (1, 0), (-1, 5), (5, -1), (1 << 40, 1 << 40)):
        assert L.grpo_clip_loss_workspace_bytes(*bad) == 0 == L.grpo_pref_loss_workspace_bytes(*bad)


@pytest.mark.parametrize("name,struct", [("grpo_clip_opts", _lib.ClipOpts), ("grpo_pref_opts", _lib.PrefOpts)])
def test_opts_structs_match_the_header(name, struct):
    hdr = open(os.path.join(os.path.dirname(__file__), "..", "include", "grpo.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), hdr, re.S).group(1)
    decl = [ln.split(";")[0].split() for ln in body.splitlines() if ";" in ln]
    types = {"double": ctypes.c_double, "int32_t": ctypes.c_int32}
    assert list(struct._fields_) == [(n, types[t]) for t, n in decl]


# ---------------------------------------------------------------- the binding
N, B, S, d, V = 12, 3, 4, 16, 40


def _head():
    return dict(H=torch.zeros(N, d, dtype=torch.bfloat16), W=torch.zeros(V, d, dtype=torch.bfloat16),
                y=torch.zeros(N, dtype=torch.int32))


@pytest.mark.parametrize("over,err,what", [
    ({"H": torch.zeros(N, d, dtype=torch.float16)}, TypeError, "float16"), ({"H": torch.zeros(N * d)}, ValueError, "2-D"),
    ({"W": torch.zeros(V, d)}, TypeError, "W"), ({"W": torch.zeros(V, 8, dtype=torch.bfloat16)}, ValueError, "W"),
    ({"y": torch.zeros(N, dtype=torch.int64)}, TypeError, "y"), ({"y": torch.zeros(N + 1, dtype=torch.int32)}, ValueError, "y"),
    ({}, ValueError, "on the GPU")])
def test_binding_logprobs_refusals(over, err, what):
    a = {**_head(), **over}
    with pytest.raises(err, match=what):
        gp.grpo_logprobs_fwd(**a)
    with pytest.raises(err, match=what):
        gp.grpo_logprobs_bwd(**a, lp=torch.zeros(N), lse=torch.zeros(N), grad_lp=torch.zeros(N))
    with pytest.raises(err, match=what):
        gp.grpo_logprobs(**a)


@pytest.mark.parametrize("over,err,what", [
    ({"lp": torch.zeros(N, dtype=torch.float64)}, TypeError, "lp"), ({"lse": torch.zeros(2 * N)}, ValueError, "lse"),
    ({"H": torch.zeros(N, d), "W": torch.zeros(V, d)}, ValueError, "lse"),      # float32: 2 N
    ({"grad_lp": torch.zeros(N, dtype=torch.bfloat16)}, TypeError, "grad_lp"), ({"grad_lp": torch.zeros(1)}, ValueError, "grad_lp"),
    ({"dH": torch.zeros(N, d)}, TypeError, "dH"), ({"dW": torch.zeros(V, d, dtype=torch.bfloat16)}, TypeError, "dW"),
    ({"dW": torch.zeros(V, d + 1)}, ValueError, "dW"), ({"need_h": False, "need_w": False}, ValueError, "need")])
def test_binding_logprobs_backward_refusals(over, err, what):
    a = {**_head(), "lp": torch.zeros(N), "lse": torch.zeros(N), "grad_lp": torch.zeros(N), **over}
    with pytest.raises(err, match=what):
        gp.grpo_logprobs_bwd(**a)


def _tokens(n=N):
    return dict(lp=torch.zeros(n), mask=torch.ones(n, dtype=torch.uint8))


@pytest.mark.parametrize("over,err,what", [
    ({"lp": torch.zeros(N, dtype=torch.float64)}, TypeError, "lp"), ({"lp": torch.zeros(N + 1)}, ValueError, "lp"),
    ({"mask": torch.ones(N)}, TypeError, "mask"), ({"adv": torch.zeros(B + 1)}, ValueError, "adv"),
    ({"adv": torch.zeros(B, dtype=torch.float64)}, TypeError, "adv"), ({"old_lp": torch.zeros(N - 1)}, ValueError, "old_lp"),
    ({"ref_lp": torch.zeros(N, dtype=torch.bfloat16)}, TypeError, "ref_lp"), ({"B": 0}, ValueError, "positive"),
    ({"L": -4}, ValueError, "positive"), ({}, ValueError, "on the GPU")])
def test_binding_clip_refusals(over, err, what):
    a = {**_tokens(), "adv": torch.zeros(B), "B": B, "L": S, **over}
    with pytest.raises(err, match=what):
        gp.grpo_clip_loss_fwd(**a)
    with pytest.raises(err, match=what):
        gp.grpo_clip_loss(**a)
    with pytest.raises(err, match=what):
        gp.grpo_clip_loss_bwd(weights=torch.zeros(2 * B + 1), **a)


def test_binding_clip_buffers():
    a = {**_tokens(), "adv": torch.zeros(N), "B": B, "L": S}
    for over, err, what in (({"weights": torch.zeros(2 * B)}, ValueError, "weights"), ({"out": torch.zeros(N + 1)}, ValueError, "out"),
                            ({"grad_loss": torch.zeros(2)}, ValueError, "grad_loss"), ({"grad_loss": 1.0}, TypeError, "grad_loss")):
        with pytest.raises(err, match=what):
            gp.grpo_clip_loss_bwd(**{"weights": torch.zeros(2 * B + 1), **a, **over})
    with pytest.raises(ValueError, match="workspace"):
        gp.grpo_clip_loss_fwd(workspace=torch.zeros(8, dtype=torch.uint8), **a)
    with pytest.raises(TypeError, match="workspace"):
        gp.grpo_clip_loss_fwd(workspace=torch.zeros(4096), **a)


@pytest.mark.parametrize("over,err,what", [
    ({"lp": torch.zeros(N)}, ValueError, "lp"), ({"mask": torch.ones(16, dtype=torch.bool)}, TypeError, "mask"),
    ({"ref_lp": torch.zeros(15)}, ValueError, "ref_lp"), ({"P": 0}, ValueError, "positive"),
    ({"workspace": torch.zeros(8, dtype=torch.uint8)}, ValueError, "workspace"), ({}, ValueError, "on the GPU")])
def test_binding_pref_refusals(over, err, what):
    with pytest.raises(err, match=what):
        gp.grpo_pref_loss_fwd(**{**_tokens(16), "P": 2, "L": 4, **over})


@pytest.mark.parametrize("over,err,what", [
    ({"mask": torch.ones(15, dtype=torch.uint8)}, ValueError, "mask"), ({"weights": torch.zeros(3)}, ValueError, "weights"),
    ({"grad_loss": torch.zeros(1, dtype=torch.float64)}, TypeError, "grad_loss"), ({"out": torch.zeros(4)}, ValueError, "out"),
    ({"L": 0}, ValueError, "positive"), ({}, ValueError, "on the GPU")])
def test_binding_pref_backward_refusals(over, err, what):
    with pytest.raises(err, match=what):
        gp.grpo_pref_loss_bwd(**{"mask": torch.ones(16, dtype=torch.uint8), "weights": torch.zeros(4), "P": 2, "L": 4, **over})
