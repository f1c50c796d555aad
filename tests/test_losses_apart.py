"""What the losses over given log-probabilities write lies apart from what they read: a block writes
while others still read, so outputs that share memory with an input, or with another output, are refused
on the host (no call here gets past its checks), by ranges rather than by where they start."""
import ctypes
import os

import pytest
import torch

gp = pytest.importorskip("grpo_policy_loss_amd")
from grpo_policy_loss_amd import _lib  # noqa: E402

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libgrpo.so not built", allow_module_level=True)

L = _lib.lib()
B, S, N = 4, 8, 32
STEP = 0x100000     # between the addresses, none of which is read
CLIP_FWD = dict(lp=4 * N, old=4 * N, ref=4 * N, mask=N, adv=4 * B, B=B, L=S, opts=None, loss=4, stats=16, weights=4 * (2 * B + 1),
                ws=L.grpo_clip_loss_workspace_bytes(B, S), wsb=1 << 20)
CLIP_BWD = dict(lp=4 * N, old=4 * N, ref=4 * N, mask=N, adv=4 * B, weights=4 * (2 * B + 1), g=4, B=B, L=S, opts=None, out=4 * N)
PREF_FWD = dict(lp=4 * N, ref=4 * N, mask=N, P=B // 2, L=S, opts=None, loss=4, rewards=4 * B, weights=4 * B,
                ws=L.grpo_pref_loss_workspace_bytes(B // 2, S), wsb=1 << 20)
PREF_BWD = dict(mask=N, weights=4 * B, g=4, P=B // 2, L=S, out=4 * N)
CALLS = dict(grpo_clip_loss_fwd=(CLIP_FWD, ("loss", "stats", "weights", "ws")), grpo_clip_loss_bwd=(CLIP_BWD, ("out",)),
             grpo_pref_loss_fwd=(PREF_FWD, ("loss", "rewards", "weights", "ws")), grpo_pref_loss_bwd=(PREF_BWD, ("out",)))
SIZES = ("B", "P", "L", "opts", "wsb")


def overlaps():
    for fn, (sizes, outs) in CALLS.items():
        tensors = [k for k in sizes if k not in SIZES]
        for out in outs:
            for other in tensors:
                if other == out:
                    continue
                # the same place, the other's last byte, and the output's last byte
                for by in (0, sizes[other] - 1, 1 - sizes[out]):
                    if out != "ws" or by % 256 == 0:
                        yield fn, out, other, by


@pytest.mark.parametrize("fn,out,other,by", overlaps())
def test_shared_memory_is_refused(fn, out, other, by):
    sizes = CALLS[fn][0]
    a = {k: v if k in SIZES else STEP * (i + 1) for i, (k, v) in enumerate(sizes.items())}
    a[out] = a[other] + by
    if fn == "grpo_pref_loss_fwd":
        a["opts"] = ctypes.pointer(_lib.PrefOpts(beta=0.1))
    assert getattr(L, fn)(*a.values(), None) == -1
    assert b"overlap" in L.grpo_last_error()


def test_advantages_for_each_token_are_longer():
    a = {k: v if k in SIZES else STEP * (i + 1) for i, (k, v) in enumerate(CLIP_BWD.items())}
    a["opts"] = ctypes.pointer(_lib.ClipOpts(adv_per_token=1))
    a["out"] = a["adv"] + 4 * N - 1
    assert L.grpo_clip_loss_bwd(*a.values(), None) == -1
    assert b"overlap" in L.grpo_last_error()


@pytest.mark.gpu
def test_neighbours_in_one_buffer():
    """Side by side is apart; one element in common is not."""
    g = torch.Generator().manual_seed(1)
    n = 3 * 41
    buf = torch.full((3 * n + 1,), 7.0, device="cuda")
    lp, out = buf[:n], buf[n:2 * n]
    lp.copy_(-torch.rand(n, generator=g))
    mask, adv = (torch.rand(n, generator=g) < 0.7).to(torch.uint8).cuda(), torch.randn(3, generator=g).cuda()
    w = gp.grpo_clip_loss_fwd(lp, mask, adv, 3, 41)[2]
    want = gp.grpo_clip_loss_bwd(lp, mask, adv, w, 3, 41)
    assert torch.equal(gp.grpo_clip_loss_bwd(lp, mask, adv, w, 3, 41, out=out), want)
    assert torch.equal(lp.cpu(), -torch.rand(n, generator=torch.Generator().manual_seed(1))) and (buf[2 * n:] == 7).all()
    for shifted in (buf[:n], buf[1:n + 1], buf[n - 1:2 * n - 1]):
        with pytest.raises(gp.GrpoError, match="overlap"):
            gp.grpo_clip_loss_bwd(lp, mask, adv, w, 3, 41, out=shifted)
    pw = torch.randn(6, device="cuda")
    ones = torch.ones(6, dtype=torch.uint8, device="cuda")
    with pytest.raises(gp.GrpoError, match="overlap"):
        gp.grpo_pref_loss_bwd(ones, pw, 3, 1, out=pw)
    assert torch.equal(gp.grpo_pref_loss_bwd(ones, pw, 3, 1), pw)
