"""What the clipped loss's forward keeps for its backward is written in full, whatever the ratio and the mean:
for each sequence the factor of its terms and the slope of its ratio, and the weight of them all."""
import ctypes
import itertools
import math

import pytest
import torch

import grpo_policy_loss_amd as gp
from grpo_policy_loss_amd import _lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("B,L", [(1, 1), (5, 3), (3, 700), (2, 3000), (300, 1100), (4500, 9)])
@pytest.mark.parametrize("sequence,seq_mean,per_token", [c for c in itertools.product((False, True), repeat=3) if not (c[0] and c[2])])
def test_every_element_is_written(B, L, sequence, seq_mean, per_token):
    g = torch.Generator().manual_seed(B + L)
    lp = -torch.rand(B * L, generator=g)
    old = lp + 0.1 * torch.randn(B * L, generator=g)
    mask = (torch.rand(B, L, generator=g) < 0.6).to(torch.uint8)
    mask[B // 2] = 0
    adv = torch.randn(B * L if per_token else B, generator=g)
    dev = [t.cuda().flatten() for t in (lp, old, mask, adv)]
    weights = torch.full((2 * B + 1,), math.nan, device="cuda")
    out = torch.empty(5, device="cuda")
    need = _lib.lib().grpo_clip_loss_workspace_bytes(B, L)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    opts = ctypes.pointer(_lib.ClipOpts(ratio=int(sequence), aggregation=gp.AGG_SEQUENCE_MEAN if seq_mean else gp.AGG_TOKEN_MEAN,
                                        adv_per_token=int(per_token)))
    stream = torch.cuda.current_stream().cuda_stream
    assert _lib.lib().grpo_clip_loss_fwd(dev[0].data_ptr(), dev[1].data_ptr(), None, dev[2].data_ptr(), dev[3].data_ptr(), B, L, opts,
                                         out.data_ptr(), out[1:].data_ptr(), weights.data_ptr(), ws.data_ptr(), need, stream) == 0
    w = weights.cpu().double()
    n = mask.sum(1, dtype=torch.float64)
    factor = 1 / n.clamp(min=1) if seq_mean else torch.ones(B, dtype=torch.float64)
    slope = torch.zeros(B, dtype=torch.float64)
    if sequence:
        D = ((lp.double() - old.double()).view(B, L) * mask).sum(1) / n.clamp(min=1)
        slope = -adv.double() * D.exp()
    # each a float64 rounded once
    assert ((w[0:-1:2] - factor).abs() <= 2 * U * factor).all()
    assert ((w[1:-1:2] - slope).abs() <= 2 * U * slope.abs()).all()
    whole = 1 / B if seq_mean else 1 / max(1.0, n.sum().item())
    assert abs(w[-1].item() - whole) <= 2 * U * whole
