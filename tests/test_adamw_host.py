"""AdamW's plan and refusals on the host: grpo_adamw_plan runs without a GPU (it reads
no device memory), grpo_adamw is called with arguments that it rejects."""
import ctypes
import os

import pytest
import torch

gp = pytest.importorskip("grpo_policy_loss_amd")
from grpo_policy_loss_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libgrpo.so not built", allow_module_level=True)

L = _lib.lib()
NAMES = [n for n, _ in _lib.AdamWTensor._fields_][:-1]


def tensor(at, n=1000, master=False, scales=True):
    """A tensor whose parts lie 2^20 bytes apart from address `at` on."""
    t = _lib.AdamWTensor(**{name: at + (i << 20) for i, name in enumerate(NAMES)})
    t.n = n
    if not master:
        t.master = None
    if not scales:
        t.exp_avg_scales = t.exp_avg_sq_scales = None
    return t


def plan(ts, pt=1, gt=0, bits=8, size=None):
    rows = (_lib.AdamWTensor * max(1, len(ts)))(*ts)
    need = L.grpo_adamw_plan_bytes(len(ts))
    image = (ctypes.c_uint8 * need)()
    return L.grpo_adamw_plan(rows, len(ts), pt, gt, bits, image, need if size is None else size), image


def test_a_plan_of_many_tensors():
    ts = [tensor((i + 1) << 24, n) for i, n in enumerate([1, 0, 4096, 4097, 7, 100003, 0])]
    code, image = plan(ts)
    assert code == 0
    header = ctypes.cast(image, ctypes.POINTER(ctypes.c_int64))
    assert header[1] == 7                                 # tensors
    assert header[2] == 1 + 0 + 2 + 3 + 1 + 49 + 0        # chunks of 2048
    big = [tensor(1 << 40, (1 << 26) - 5), tensor(1 << 24, 5)]
    for i, name in enumerate(NAMES):
        if getattr(big[0], name):
            setattr(big[0], name, (1 << 40) + (i << 34))
    for bits, chunks in ((32, (1 << 14) + 1), (8, (1 << 15) + 1)):      # of 4096, of 2048
        code, image = plan(big, bits=bits)
        assert code == 0
        assert ctypes.cast(image, ctypes.POINTER(ctypes.c_int64))[2] == chunks
    assert plan([])[0] == 0
    assert plan([tensor(1 << 24, 0)])[0] == 0
    assert L.grpo_adamw_plan_bytes(-1) == 0


@pytest.mark.parametrize("change,word", [
    ({"param": None}, b"param"), ({"grad": None}, b"grad"), ({"exp_avg": None}, b"exp_avg"),
    ({"exp_avg_sq_scales": None}, b"scales"), ({"n": -1}, b"elements"),
    ({"param": (1 << 24) + 1}, b"aligned"), ({"grad": (1 << 25) + 2}, b"aligned"),
    ({"exp_avg_scales": (1 << 25) + 2}, b"aligned")])
def test_bad_tensors_are_refused(change, word):
    t = tensor(1 << 24)
    for k, v in change.items():
        setattr(t, k, v)
    assert plan([tensor(1 << 30), t])[0] == -1
    assert word in L.grpo_last_error()


def test_masters_are_all_or_none_and_for_bfloat16():
    a, b = tensor(1 << 24, master=True), tensor(1 << 25, master=True)
    assert plan([a, b])[0] == 0
    assert plan([a, tensor(1 << 25)])[0] == -1
    assert plan([a, b], pt=0)[0] == -1
    assert b"master" in L.grpo_last_error()


def test_shared_memory_is_refused():
    assert plan([tensor(1 << 24), tensor(1 << 24)])[0] == -1
    assert b"overlap" in L.grpo_last_error()
    a, b = tensor(1 << 24), tensor(1 << 25)
    assert plan([a, b])[0] == 0
    b.param = a.param + 2 * 1000 - 2           # the last element of a's parameter
    assert plan([a, b])[0] == -1
    b.param = a.param + 2 * 1000               # just behind it
    assert plan([a, b])[0] == 0
    b.grad = a.grad                            # a gradient is only read
    assert plan([a, b])[0] == 0
    b.grad = a.exp_avg
    assert plan([a, b])[0] == -1
    a.grad = a.param                           # its own parameter as gradient
    assert plan([a])[0] == -1
    c = tensor(1 << 26, n=10)                  # inside a longer range that starts before it
    c.exp_avg = a.exp_avg_sq + 300
    a = tensor(1 << 24)
    assert plan([a, c])[0] == -1


@pytest.mark.parametrize("kw,code", [({"pt": 2}, -1), ({"gt": 3}, -1), ({"bits": 16}, -1),
                                     ({"size": 64}, -2)])
def test_bad_plans_are_refused(kw, code):
    assert plan([tensor(1 << 24)], **kw)[0] == code


def step(image, **kw):
    o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1)
    o.update(kw)
    return L.grpo_adamw(image, None, ctypes.byref(_lib.AdamWOpts(**o)), None)


@pytest.mark.parametrize("kw", [
    {"lr": -1.0}, {"lr": float("nan")}, {"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.5},
    {"beta2": float("nan")}, {"eps": -1e-8}, {"eps": float("inf")}, {"weight_decay": -1.0},
    {"lr": 1e39}, {"eps": 1e39}, {"weight_decay": 1e39}, {"step": 0}, {"step": -5}])
def test_bad_hyperparameters_are_refused(kw):
    assert step(plan([tensor(1 << 24)])[1], **kw) == -1
    assert L.grpo_last_error()


def test_a_step_needs_its_plan():
    assert step(plan([tensor(1 << 24)])[1]) == -1          # no device copy
    assert step((ctypes.c_uint8 * 4096)()) == -1           # not an image
    assert L.grpo_adamw(None, None, None, None) == -1
    assert step(plan([])[1]) == 0                          # nothing to do


def test_moment_values_refusals():
    one = ctypes.c_void_p(16)
    assert L.grpo_moment_values(one, one, -1, 0, one, None) == -1
    assert L.grpo_moment_values(one, one, 5, 2, one, None) == -1
    assert L.grpo_moment_values(None, one, 5, 0, one, None) == -1
    assert L.grpo_moment_values(one, one, 0, 0, one, None) == 0
    assert L.grpo_moment_values(one, one, 1 << 40, 1, one, None) == -3


def _lists(n=300, t=torch.bfloat16, g=torch.float32, bits=32):
    p = [torch.zeros(n, dtype=t)]
    m, v = gp.adamw_moments(p, bits)
    return dict(params=p, grads=[torch.zeros(n, dtype=g)], exp_avg=m, exp_avg_sq=v)


@pytest.mark.parametrize("over,err,what", [
    ({"params": []}, ValueError, "empty"),
    ({"grads": []}, ValueError, "grads"),
    ({"grads": [torch.zeros(299)]}, ValueError, "grads"),
    ({"grads": [torch.zeros(300, dtype=torch.float16)]}, TypeError, "float16"),
    ({"exp_avg": [torch.zeros(300, dtype=torch.bfloat16)]}, TypeError, "exp_avg"),
    ({"exp_avg_sq": [torch.zeros(301)]}, ValueError, "exp_avg_sq"),
    ({"exp_avg": [gp.Moment8(torch.zeros(300, dtype=torch.int8), torch.zeros(2))]}, TypeError, "moments"),
    ({"master": [torch.zeros(300, dtype=torch.bfloat16)]}, TypeError, "master"),
    ({"master": []}, ValueError, "master"),
    ({}, ValueError, "on the GPU")])
def test_binding_refusals(over, err, what):
    with pytest.raises(err, match=what):
        gp.adamw_plan(**{**_lists(), **over})


def test_moments():
    m, v = gp.adamw_moments([torch.zeros(3, 200), torch.zeros(7)], 8)
    assert m[0].codes.dtype == torch.int8 and v[0].codes.dtype == torch.uint8
    assert m[0].shape == (3, 200) and m[0].scales.numel() == 3 and v[1].scales.numel() == 1
    with pytest.raises(ValueError):
        gp.adamw_moments([torch.zeros(3)], 4)
    with pytest.raises(ValueError, match="scales"):
        gp.Moment8(torch.zeros(257, dtype=torch.int8), torch.zeros(1))
    with pytest.raises(TypeError, match="codes"):
        gp.Moment8(torch.zeros(257), torch.zeros(2))
    with pytest.raises(TypeError, match="exp_avg"):     # the codes of the other moment
        gp.adamw_plan([torch.zeros(3)], [torch.zeros(3)], [v[1]][:1], [m[1]])


@pytest.mark.parametrize("default", [torch.float64, torch.bfloat16])
def test_moments_do_not_go_by_the_default_type(default):
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        for bits in (8, 32):
            m, v = gp.adamw_moments([torch.zeros(300, dtype=torch.float32)], bits)
            for q in (m[0], v[0]):
                assert (q.scales if bits == 8 else q).dtype == torch.float32
    finally:
        torch.set_default_dtype(before)


def test_structs_match_the_header():
    hdr = open(os.path.join(os.path.dirname(__file__), "..", "include", "grpo.h")).read()
    for struct, cls in (("grpo_adamw_tensor", _lib.AdamWTensor), ("grpo_adamw_opts", _lib.AdamWOpts)):
        body = hdr[hdr.index("typedef struct %s {" % struct):hdr.index("} %s;" % struct)]
        names = [ln.split(";")[0].split()[-1].lstrip("*") for ln in body.splitlines()[1:] if ";" in ln]
        assert names == [n for n, _ in cls._fields_]
