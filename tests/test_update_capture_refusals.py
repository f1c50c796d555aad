"""The autograd forms' backwards raise while their stream is captured, before any device work: a captured one that
reaches an eager graph of the same leaves would end the process.  Nothing is captured here; the stream only says
that it is."""
import types

import pytest
import torch

gp = pytest.importorskip("grpo_policy_loss_amd")
from grpo_policy_loss_amd import autograd  # noqa: E402

FORMS = {"grpo_norm": (autograd._GrpoNorm, 1), "grpo_logprobs": (autograd._GrpoLogprobs, 1), "grpo_clip_loss": (autograd._GrpoClipLoss, 2),
         "grpo_pref_loss": (autograd._GrpoPrefLoss, 2)}


@pytest.fixture
def capturing(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)


@pytest.mark.parametrize("name", list(FORMS))
def test_refused_before_anything_is_read(name, capturing):
    function, outputs = FORMS[name]
    with pytest.raises(RuntimeError, match=f"{name}'s backward cannot be captured: call {name}_bwd"):
        function.backward(types.SimpleNamespace(), *[None] * outputs)


def losses():
    d = lambda *s: torch.randn(*s, generator=torch.Generator().manual_seed(2)).cuda()  # noqa: E731
    H, W, lp = d(8, 64).requires_grad_(), d(100, 64).requires_grad_(), d(8).requires_grad_()
    mask, y = torch.ones(8, dtype=torch.uint8, device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda")
    yield "grpo_logprobs", (H, W), lambda: gp.grpo_logprobs(H, W, y).sum()
    yield "grpo_clip_loss", (lp,), lambda: gp.grpo_clip_loss(lp, mask, d(2), 2, 4)[0]
    yield "grpo_pref_loss", (lp,), lambda: gp.grpo_pref_loss(lp, mask, 1, 4)[0]


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(3))
def test_a_loss_s_backward_is_refused_and_works_afterwards(which, monkeypatch):
    name, leaves, loss_of = list(losses())[which]
    loss = loss_of()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match=f"{name}'s backward cannot be captured"):
        loss.backward(retain_graph=True)
    assert all(x.grad is None for x in leaves)
    monkeypatch.undo()
    loss.backward()
    assert all(x.grad.any() for x in leaves)
