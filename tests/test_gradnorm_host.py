"""The gradient plan and the refusals of the gradients' norm and clipping, on the host."""
import ctypes
import os

import pytest
import torch

gp = pytest.importorskip("grpo_policy_loss_amd")
from grpo_policy_loss_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libgrpo.so not built", allow_module_level=True)

L = _lib.lib()
FAKE = ctypes.c_void_p(0x1000)     # never dereferenced
F32, BF16 = 0, 1


def image_of(rows):
    """(code, image) of a plan of (address, elements, dtype)."""
    t = (_lib.GradTensor * max(1, len(rows)))(*[_lib.GradTensor(a, n, dt, 0) for a, n, dt in rows])
    size = L.grpo_grad_plan_bytes(len(rows))
    image = (ctypes.c_uint8 * size)()
    return L.grpo_grad_plan(t, len(rows), image, size), image


def norm(image, **kw):
    a = dict(image=image, plan=FAKE, kind=0, max_norm=1.0, norm=FAKE, scale=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return L.grpo_grad_norm(*a.values(), None)


@pytest.mark.parametrize("rows,code", [
    ([(0x10000, 8, F32), (0x10020, 8, BF16)], 0),                  # side by side
    ([(0x10000, 8, F32), (0x1001c, 8, F32)], -1),                  # one element shared
    ([(0x10000, 8, F32), (0x10000, 8, F32)], -1),
    ([(0x10020, 8, BF16), (0x10000, 17, BF16)], -1),
    ([(0x10000, 0, F32), (0x10000, 8, F32), (0, 0, BF16)], 0),     # empty ones have no place
    ([(0, 8, F32)], -1), ([(0x10002, 8, F32)], -1), ([(0x10001, 8, BF16)], -1), ([(0x10002, 8, BF16)], 0),
    ([(0x10000, -1, F32)], -1), ([(0x10000, 8, 2)], -1), ([(0x10000, 0, 7)], -1), ([(0x10000, (1 << 48) + 1, F32)], -1),
    ([(1 << 50, 8192 * ((1 << 22) - 1), F32)], 0), ([(1 << 50, 8192 * ((1 << 22) - 1) + 1, F32)], -3), ([], 0)])
def test_plan(rows, code):
    assert image_of(rows)[0] == code
    assert (code == 0) == (L.grpo_last_error() == b"")


def test_plan_argument_errors():
    assert L.grpo_grad_plan_bytes(-1) == 0 == L.grpo_grad_plan_bytes((1 << 24) + 1)
    buf = (ctypes.c_uint8 * 4096)()
    t = (_lib.GradTensor * 1)(_lib.GradTensor(0x1000, 4, 0, 0))
    assert L.grpo_grad_plan(None, 1, buf, 4096) == -1
    assert L.grpo_grad_plan(t, 1, None, 4096) == -1
    assert L.grpo_grad_plan(t, -1, buf, 4096) == -1
    assert L.grpo_grad_plan(t, 1, buf, L.grpo_grad_plan_bytes(1) - 1) == -2


@pytest.mark.parametrize("kw,code", [
    ({"image": None}, -1), ({"plan": None}, -1), ({"plan": ctypes.c_void_p(0x1004)}, -1), ({"kind": 2}, -1), ({"kind": -1}, -1),
    ({"max_norm": -1.0}, -1), ({"max_norm": float("nan")}, -1), ({"max_norm": float("inf")}, -1), ({"max_norm": 1e39}, -1),
    ({"norm": None}, -1), ({"scale": None}, -1), ({"ws": None}, -2), ({"wsb": 128}, -2), ({"ws": ctypes.c_void_p(0x1008)}, -2)])
def test_norm_argument_errors(kw, code):
    image = image_of([(0x10000, 8, F32)])[1]
    assert norm(**{"image": image, **kw}) == code
    assert L.grpo_last_error()


def test_other_images_are_refused():
    blank = (ctypes.c_uint8 * 1024)()
    assert norm(blank) == -1 and L.grpo_grad_clip(blank, FAKE, FAKE, None) == -1
    size = L.grpo_adamw_plan_bytes(0)
    adamw = (ctypes.c_uint8 * size)()
    assert L.grpo_adamw_plan(None, 0, 0, 0, 32, adamw, size) == 0
    assert norm(adamw) == -1 and L.grpo_grad_clip(adamw, FAKE, FAKE, None) == -1
    opts = _lib.AdamWOpts(beta1=0.9, beta2=0.99, step=1)
    assert L.grpo_adamw(image_of([])[1], FAKE, ctypes.byref(opts), None) == -1
    image = image_of([(0x10000, 8, F32)])[1]
    assert L.grpo_grad_clip(image, FAKE, None, None) == -1
    assert L.grpo_grad_clip(image_of([])[1], None, FAKE, None) == 0      # nothing to clip launches nothing


def test_binding_refusals():
    with pytest.raises(ValueError, match="empty"):
        gp.grad_plan([])
    with pytest.raises(TypeError, match="float16"):
        gp.grad_plan([torch.zeros(3, dtype=torch.float16)])
    with pytest.raises(TypeError, match=r"grads\[1\]"):
        gp.grad_plan([torch.zeros(3), None])
    with pytest.raises(ValueError, match="on the GPU"):
        gp.grad_plan([torch.zeros(3)])
