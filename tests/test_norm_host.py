"""The norm's refusals, on the host: the C ABI's argument checks (no call here gets
past them) and the binding's checks of types, shapes and devices."""
import ctypes
import os

import pytest
import torch

gp = pytest.importorskip("grpo_policy_loss_amd")
from grpo_policy_loss_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libgrpo.so not built", allow_module_level=True)

L = _lib.lib()
FAKE, OUT = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x2000)


def fwd(**kw):
    a = dict(X=FAKE, w=FAKE, b=None, rows=4, cols=8, dt=0, kind=0, eps=1e-5, Y=OUT, mean=FAKE,
             rstd=FAKE)
    a.update(kw)
    return L.grpo_norm_fwd(*a.values(), None)


def bwd(**kw):
    a = dict(dY=FAKE, X=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, rows=4, cols=8, dt=0, kind=0, acc=0, dX=OUT,
             dw=FAKE, db=None, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return L.grpo_norm_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    ({"X": None}, -1), ({"w": None}, -1), ({"Y": None}, -1), ({"rstd": None}, -1),
    ({"mean": None}, -1), ({"rows": 0}, -1), ({"cols": -1}, -1), ({"dt": 2}, -1), ({"dt": -1}, -1),
    ({"kind": 2}, -1), ({"eps": -1e-5}, -1), ({"eps": float("nan")}, -1),
    ({"eps": float("inf")}, -1), ({"Y": FAKE}, -1), ({"rows": 1 << 31}, -3), ({"cols": (1 << 24) + 1}, -3)])
def test_forward_argument_errors(kw, code):
    assert fwd(**kw) == code
    assert L.grpo_last_error()


@pytest.mark.parametrize("kw,code", [
    ({"dY": None}, -1), ({"X": None}, -1), ({"w": None}, -1), ({"mean": None}, -1),
    ({"rstd": None}, -1), ({"dX": None}, -1), ({"dw": None}, -1), ({"rows": -3}, -1),
    ({"dt": 7}, -1), ({"kind": -1}, -1), ({"acc": 2}, -1), ({"dX": FAKE}, -1), ({"X": OUT}, -1), ({"dY": OUT}, -1),
    ({"ws": None}, -2), ({"wsb": 16}, -2), ({"ws": ctypes.c_void_p(0x1010)}, -2),
    ({"cols": 1 << 25}, -3)])
def test_backward_argument_errors(kw, code):
    assert bwd(**kw) == code
    assert L.grpo_last_error()


def test_workspace_is_bounded():
    for dt in (0, 1):
        assert L.grpo_norm_workspace_bytes(0, 8, dt) == 0
        assert L.grpo_norm_workspace_bytes(8, 0, dt) == 0
        assert L.grpo_norm_workspace_bytes(8, 8, 2) == 0
        for rows in (1, 3, 1000, 1 << 20):
            for cols in (1, 31, 1537, 4096, 16384, 100003):
                ws = L.grpo_norm_workspace_bytes(rows, cols, dt)
                # at most 1024 partial rows of dw and of db, and no more than there are rows
                assert 8 * cols <= ws <= 8 * cols * min(rows, 1024) + 512
        # long rows: 128 MB at most, or one partial row of each
        assert L.grpo_norm_workspace_bytes(1 << 20, 1 << 20, dt) <= 1 << 27
        assert L.grpo_norm_workspace_bytes(1 << 20, 1 << 24, dt) == 1 << 27


def test_workspace_holds_the_partial_rows_of_either_form():
    """bfloat16 rows of 2049 to 4096 elements with bias leave one partial row for each row up to
    512, whatever the form without bias leaves."""
    for rows in (1, 2, 511, 512, 700, 1023, 1024, 5000):
        for cols in (2049, 2880, 3328, 3329, 4096):
            need = 2 * (-(-min(rows, 512) * cols * 4 // 256) * 256)
            assert L.grpo_norm_workspace_bytes(rows, cols, 1) >= need


def _args(t=torch.bfloat16):
    return dict(X=torch.zeros(6, 8, dtype=t), weight=torch.ones(8, dtype=t),
                bias=torch.zeros(8, dtype=t))


@pytest.mark.parametrize("over,err,what", [
    ({"X": torch.zeros(6, 8, dtype=torch.float16)}, TypeError, "float16"),
    ({"X": torch.zeros(2, 3, 8, dtype=torch.bfloat16)}, ValueError, "2-D"),
    ({"weight": torch.ones(8)}, TypeError, "weight"),
    ({"weight": torch.ones(7, dtype=torch.bfloat16)}, ValueError, "weight"),
    ({"bias": torch.ones(9, dtype=torch.bfloat16)}, ValueError, "bias"),
    ({"out": torch.zeros(6, 8)}, TypeError, "out"),
    ({"out": torch.zeros(5, 8, dtype=torch.bfloat16)}, ValueError, "out"),
    ({}, ValueError, "on the GPU")])
def test_binding_forward_refusals(over, err, what):
    with pytest.raises(err, match=what):
        gp.grpo_norm_fwd(**{**_args(), **over})


@pytest.mark.parametrize("over,err,what", [
    ({"dY": torch.zeros(6, 8)}, TypeError, "dY"),
    ({"dY": torch.zeros(6, 7, dtype=torch.bfloat16)}, ValueError, "dY"),
    ({"mean": None}, TypeError, "mean"),
    ({"mean": torch.zeros(5)}, ValueError, "mean"),
    ({"rstd": torch.zeros(6, dtype=torch.float64)}, TypeError, "rstd"),
    ({"dweight": torch.zeros(8, dtype=torch.bfloat16)}, TypeError, "dweight"),
    ({"dbias": torch.zeros(7)}, ValueError, "dbias"),
    ({"dX": torch.zeros(6, 9, dtype=torch.bfloat16)}, ValueError, "dX"),
    ({"workspace": torch.zeros(8, dtype=torch.uint8)}, ValueError, "workspace"),
    ({}, ValueError, "on the GPU")])
def test_binding_backward_refusals(over, err, what):
    a = dict(dY=torch.zeros(6, 8, dtype=torch.bfloat16), X=torch.zeros(6, 8, dtype=torch.bfloat16),
             weight=torch.ones(8, dtype=torch.bfloat16), mean=torch.zeros(6), rstd=torch.zeros(6),
             kind=gp.NORM_LAYER)
    with pytest.raises(err, match=what):
        gp.grpo_norm_bwd(**{**a, **over})
