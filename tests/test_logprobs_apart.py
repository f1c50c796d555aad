"""What the log-probabilities' calls write lies apart from everything that they read: later chunks read lse
and grad_lp again after the first one's gradients are written.  Refused on the host by ranges (no call here
gets past its checks)."""
import ctypes
import os

import pytest
import torch

gp = pytest.importorskip("grpo_policy_loss_amd")
from grpo_policy_loss_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libgrpo.so not built", allow_module_level=True)

L = _lib.lib()
STEP = 1 << 34          # between the addresses, none of which is read
FIXED = ("N", "d", "V", "dt", "chunk", "opts", "wsb", "acc", "dwt")
HEADS = {"f32 small": (8, 16, 32, 0), "f32 large": (4096, 1024, 24600, 0), "bf16 small": (8, 16, 32, 1), "bf16 large": (4096, 1536, 151936, 1)}


def calls(head):
    N, d, V, dt = HEADS[head]
    es, lse = (4, 8) if dt == 0 else (2, 4)
    common = dict(H=N * d * es, W=V * d * es, y=4 * N)
    fwd, bwd = (L.grpo_workspace_bytes(op, N, d, V, dt, N) for op in (16, 17))
    return {"grpo_logprobs_fwd": (common | dict(N=N, d=d, V=V, dt=dt, chunk=N, opts=None, lp=4 * N, lse=lse * N, ws=fwd, wsb=fwd), ("lp", "lse", "ws")),
            "grpo_logprobs_bwd": (common | dict(lp=4 * N, lse=lse * N, g=4 * N, N=N, d=d, V=V, dt=dt, chunk=N, opts=None, acc=0, dwt=0,
                                                dH=N * d * es, dW=4 * V * d, ws=bwd, wsb=bwd), ("dH", "dW", "ws"))}


def overlaps():
    for head in HEADS:
        for fn, (sizes, outs) in calls(head).items():
            for out in outs:
                for other in sizes:
                    if other != out and other not in FIXED:
                        for by in (0, (sizes[other] - 1) // 256 * 256, -((sizes[out] - 1) // 256 * 256)):
                            yield head, fn, out, other, by


@pytest.mark.parametrize("head,fn,out,other,by", overlaps())
def test_shared_memory_is_refused(head, fn, out, other, by):
    sizes = calls(head)[fn][0]
    a = {k: v if k in FIXED else ctypes.c_void_p(STEP * (i + 1)) for i, (k, v) in enumerate(sizes.items())}
    a[out] = ctypes.c_void_p(a[other].value + by)
    assert getattr(L, fn)(*a.values(), None) == -1
    assert b"overlap" in L.grpo_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_gradients_over_saved_values_are_refused(t):
    N, d, V = 40, 64, 300
    H, W = torch.randn(N, d, device="cuda").to(t), torch.randn(V, d, device="cuda").to(t)
    y = torch.zeros(N, dtype=torch.int32, device="cuda")
    lp, lse = gp.grpo_logprobs_fwd(H, W, y)
    buf = torch.zeros(N + N * d, device="cuda")
    g, dH = buf[:N].copy_(torch.randn(N)), buf[N - 32:].view(t)[:N * d].view(N, d)
    with pytest.raises(gp.GrpoError, match="overlap"):
        gp.grpo_logprobs_bwd(H, W, y, lp, lse, g, dH=dH)
    beside = buf[N:].view(t)[:N * d].view(N, d)
    got = gp.grpo_logprobs_bwd(H, W, y, lp, lse, g, dH=beside)[0]
    assert torch.equal(got, gp.grpo_logprobs_bwd(H, W, y, lp, lse, g.clone())[0])
