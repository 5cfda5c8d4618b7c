"""The training-step operators together: one step's gradients of the example's
network against PyTorch autograd in float64 on the same (rounded) parameters,
and a short training run."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import distill_moe_student as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def _reference(p, tokens, expert, idx, teacher, weight, T, scale):
    q = {k: v.double().requires_grad_(k != "router") for k, v in p.items()}
    h0 = scale * q["table"][tokens]
    y = torch.zeros_like(h0)
    for e in range(q["up"].shape[0]):
        at = (expert == e).nonzero()[:, 0]
        y = y.index_add(0, at, torch.nn.functional.silu(h0[at] @ q["up"][e].T) @ q["down"][e].T)
    logq = torch.log_softmax((h0 + y) @ q["head"][0].T / T, 1)
    logp = torch.log_softmax(teacher.double() / T, 1)
    loss = T * T * weight.double() * (logp.exp() * (logp - logq.gather(1, idx.long()))).sum(1)
    loss.sum().backward()
    return loss.detach(), {k: v.grad for k, v in q.items() if v.grad is not None}


def test_gradients_of_one_step_match_autograd():
    """Every stage rounds its rows to bf16 (2^-9 of their size on average); six such
    roundings lie between the table and the loss and as many on the way back, and they
    are independent: 12^(1/2) 2^-8 of a gradient's norm is about 1.4e-2.  Twice that is allowed."""
    n, vocab, dim, hidden, experts, top, T = 300, 520, 64, 96, 5, 7, 2.0
    p = ex.init(vocab, dim, hidden, experts)
    w = ex.Workspace(p, n)
    places, logits = ex.teacher_of(vocab, top)
    tokens = torch.randint(vocab, (n,), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    weight = torch.rand(n, device="cuda") / n
    idx, teacher = places[tokens], logits[tokens]
    loss = ex.forward_backward(p, w, tokens, idx, teacher, weight, T).clone()
    expert = (w.h0.float() @ p["router"]).argmax(1)
    want_loss, want = _reference(p, tokens, expert, idx, teacher, weight, T, w.scale)
    assert float((loss.double() - want_loss).norm() / want_loss.norm()) < 2.8e-2
    for k, g in want.items():
        assert float((w.grads[k].double() - g).norm() / g.norm()) < 2.8e-2, k


def test_short_training_run_learns():
    losses = ex.train(steps=30, tokens=1024, vocab=512, dim=128, hidden=256, experts=4, top=8)
    assert losses[-1] < 0.5 * losses[0]
