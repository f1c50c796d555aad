"""The gradients' norm and factor, its workspace and the factor that clips lie apart from the gradients:
blocks write them, or the gradients, while others still read.  Refused on the host (no call here gets past
its checks)."""
import ctypes
import os

import pytest
import torch

gp = pytest.importorskip("grpo_policy_loss_amd")
from grpo_policy_loss_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libgrpo.so not built", allow_module_level=True)

L = _lib.lib()
F32, BF16 = 0, 1
ROWS = [(0x10000, 300, F32), (0x30000, 0, BF16), (0x50000, 100, BF16), (0x70000, 9000, F32)]
FAR = 0x900000


def image_of(rows):
    t = (_lib.GradTensor * len(rows))(*[_lib.GradTensor(a, n, dt, 0) for a, n, dt in rows])
    size = L.grpo_grad_plan_bytes(len(rows))
    image = (ctypes.c_uint8 * size)()
    assert L.grpo_grad_plan(t, len(rows), image, size) == 0
    return image


def norm(**kw):
    a = dict(image=image_of(ROWS), plan=FAR, kind=0, max_norm=1.0, norm=FAR + 0x10000, scale=FAR + 0x20000, ws=FAR + 0x30000,
             wsb=L.grpo_grad_norm_workspace_bytes())
    a.update(kw)
    return L.grpo_grad_norm(a["image"], *(v if k in ("kind", "max_norm", "wsb") else ctypes.c_void_p(v) for k, v in list(a.items())[1:]), None)


@pytest.mark.parametrize("name", ["norm", "scale", "ws"])
@pytest.mark.parametrize("row", [0, 2, 3])
@pytest.mark.parametrize("end", [False, True])
def test_results_and_workspace_in_a_gradient_are_refused(name, row, end):
    at, n, dt = ROWS[row]
    last = at + n * (4 if dt == F32 else 2) - 1
    assert norm(**{name: last // 256 * 256 if name == "ws" and end else last if end else at}) == -1
    assert b"overlap" in L.grpo_last_error()


def test_results_in_each_other_are_refused():
    for kw in (dict(norm=FAR + 0x20003), dict(scale=FAR + 0x30004), dict(norm=FAR + 0x30000 + L.grpo_grad_norm_workspace_bytes() - 1)):
        assert norm(**kw) == -1
        assert b"overlap" in L.grpo_last_error()


@pytest.mark.parametrize("at", [0x10000, 0x10000 + 1199, 0x10000 - 3, 0x50000 + 199, 0x70000 + 4 * 8999])
def test_a_factor_in_a_gradient_is_refused(at):
    assert L.grpo_grad_clip(image_of(ROWS), ctypes.c_void_p(FAR), ctypes.c_void_p(at), None) == -1
    assert b"part of a gradient" in L.grpo_last_error()


@pytest.mark.gpu
def test_a_factor_beside_a_gradient():
    buf = torch.full((301,), 2.0, device="cuda")
    buf[300] = 0.25
    plan = gp.grad_plan([buf[:300]])
    with pytest.raises(gp.GrpoError, match="part of a gradient"):
        gp.grpo_grad_clip(plan, buf[299:300])
    gp.grpo_grad_clip(plan, buf[300:])
    assert (buf[:300] == 0.5).all() and buf[300] == 0.25
