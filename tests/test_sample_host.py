"""Sampling's refusals, on the host: no call here gets past the argument checks."""
import ctypes
import os
import re
from decimal import Decimal, localcontext

import pytest
import torch

gp = pytest.importorskip("grpo_policy_loss_amd")
from grpo_policy_loss_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libgrpo.so not built", allow_module_level=True)

L = _lib.lib()
FAKE = ctypes.c_void_p(0x1000)


def call(opts=None, **kw):
    a = dict(logits=FAKE, dt=0, B=4, V=100, stride=100, u=FAKE, opts=None, token=FAKE, lp=FAKE,
             ws=FAKE, wsb=1 << 30)
    a.update(kw)
    if opts is not None:
        a["opts"] = ctypes.byref(_lib.SampleOpts(**opts))
    return L.grpo_sample(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    ({"logits": None}, -1), ({"u": None}, -1), ({"token": None}, -1), ({"lp": None}, -1),
    ({"dt": 2}, -1), ({"B": 0}, -1), ({"V": 0}, -1), ({"stride": 99}, -1),
    ({"V": (1 << 20) + 1, "stride": 1 << 21}, -3), ({"B": (1 << 20) + 1}, -3),
    ({"ws": None}, -2), ({"wsb": 8}, -2), ({"ws": ctypes.c_void_p(0x1008)}, -2)])
def test_argument_errors(kw, code):
    assert call(**kw) == code
    assert L.grpo_last_error()


@pytest.mark.parametrize("opts", [
    {"temperature": -1.0}, {"temperature": float("nan")}, {"temperature": float("inf")},
    {"top_k": -1}, {"top_p": 1.5}, {"top_p": -0.1}, {"top_p": float("nan")}, {"min_p": 2.0},
    {"min_p": -1.0}, {"min_p": float("nan")}])
def test_bad_options_are_refused(opts):
    assert call(opts=opts) == -1
    assert L.grpo_last_error()


def test_workspace():
    assert L.grpo_sample_workspace_bytes(0, 5) == 0
    assert L.grpo_sample_workspace_bytes(5, 0) == 0
    assert L.grpo_sample_workspace_bytes(5, (1 << 20) + 1) == 0
    one = L.grpo_sample_workspace_bytes(1, 151936)
    assert 0 < one <= L.grpo_sample_workspace_bytes(256, 151936) <= 256 * one


def test_struct_matches_the_header():
    hdr = open(os.path.join(os.path.dirname(__file__), "..", "include", "grpo.h")).read()
    body = hdr[hdr.index("typedef struct grpo_sample_opts {"):hdr.index("} grpo_sample_opts;")]
    names = [ln.split(";")[0].split()[-1].lstrip("*") for ln in body.splitlines()[1:] if ";" in ln]
    assert names == [n for n, _ in _lib.SampleOpts._fields_]


def test_the_polynomial_of_two_to_a_fraction():
    """The source's own coefficients, in 40 digits: what its comment says of their error (the
    Horner steps in float64 add a few 2^-53 = 1.1e-16)."""
    path = os.path.join(os.path.dirname(_lib.__file__), "csrc", "sample.hip")
    body = open(path).read()
    body = body[body.index("double pow2_down(double t) {"):]
    body = body[body.index("double q = "):body.index("// n into the exponent")]
    coef = [float.fromhex(c) for c in re.findall(r"0x1\.[0-9a-f]+p-\d+", body)] + [1.0]
    assert len(coef) == 10 and "fma(q, f, 1.0)" in body
    with localcontext() as ctx:
        ctx.prec = 40

        def error(f):
            q = Decimal(0)
            for c in coef:
                q = q * f + Decimal(c)
            return q / Decimal(2) ** f - 1
        at = [error(Decimal(i) / 4000) for i in range(-2000, 2001)]
        assert max(abs(e) for e in at) < Decimal("1.6e-14") - 4 * Decimal(2) ** -53
        assert abs(at[0] - at[-1]) < Decimal("1e-16")     # no jump where one n meets the next


@pytest.mark.parametrize("over,err,what", [
    ({"logits": torch.zeros(10)}, ValueError, "2-D"),
    ({"logits": torch.zeros(4, 10, dtype=torch.float16)}, TypeError, "float16"),
    ({"logits": torch.zeros(10, 4).t()}, ValueError, "adjacent"),
    ({"logits": torch.zeros(1, 10).expand(4, 10)}, ValueError, "overlap"),
    ({"u": torch.zeros(3)}, ValueError, "u must"),
    ({"u": torch.zeros(4, dtype=torch.float64)}, TypeError, "u must"),
    ({"top_k": torch.zeros(4)}, TypeError, "top_k"),
    ({"top_p": torch.zeros(3)}, ValueError, "top_p"),
    ({"temperature": torch.zeros(4, dtype=torch.float64)}, TypeError, "temperature"),
    ({"out": (torch.zeros(4), torch.zeros(4))}, TypeError, "token"),
    ({"out": (torch.zeros(4, dtype=torch.int32), torch.zeros(3))}, ValueError, "lp"),
    ({"workspace": torch.zeros(8, dtype=torch.uint8)}, ValueError, "workspace"),
    ({}, ValueError, "on the GPU")])
def test_binding_refusals(over, err, what):
    with pytest.raises(err, match=what):
        gp.grpo_sample(**{**dict(logits=torch.zeros(4, 10), u=torch.zeros(4)), **over})
