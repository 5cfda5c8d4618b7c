"""Trains a small mixture-of-experts student on a teacher's top logits, with the
library's operators for everything but the pointwise parts:

    tokens -> embedding_lookup -> rows sorted by expert (embedding_lookup again, as
    a gather) -> expert_linear, SiLU, expert_linear -> residual -> head
    (expert_linear with one expert) -> distill_topk_loss_grad -> the gradients, in
    reverse -> muon_step_batched over the expert matrices and the head, with the
    embedding table as its AdamW tail

    python examples/distill_moe_student.py [--steps 60] [--tokens 4096]

Each token goes to the expert of its highest score under a fixed random router.
The data are synthetic: the teacher's top logits are a fixed function of the token.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_optimizers_gb300 as mo  # noqa: E402

BF16 = torch.bfloat16


def init(vocab, dim, hidden, experts, seed=0, device="cuda"):
    """Parameters: the table is float32 (AdamW), the matrices bf16 (Muon)."""
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    return {
        "table": rand(vocab, dim) / dim,
        "router": rand(dim, experts),
        "up": (rand(experts, hidden, dim) * dim ** -0.5).to(BF16),
        "down": (rand(experts, dim, hidden) * hidden ** -0.5).to(BF16),
        "head": (rand(1, vocab, dim) * dim ** -0.5).to(BF16),
    }


class Workspace:
    """Buffers for a batch of up to `n` tokens, allocated once."""

    def __init__(self, p, n):
        dev = p["table"].device
        vocab, dim = p["table"].shape
        experts, hidden, _ = p["up"].shape
        buf = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device=dev)  # noqa: E731
        self.scale = dim ** 0.5
        for name in ("h0", "xs", "ys", "h1", "dh1", "dys", "dxs", "back"):
            setattr(self, name, buf(n, dim))
        self.u, self.da = buf(n, hidden), buf(n, hidden)
        self.logits = buf(n, vocab)
        self.loss = buf(n, dtype=torch.float32)
        self.grads = {k: torch.empty(p[k].shape, device=dev) for k in ("table", "up", "down", "head")}
        self.whole = torch.tensor([0, n], dtype=torch.int32, device=dev)
        size = max(mo.expert_linear_workspace_bytes(n, hidden, dim, experts),
                   mo.expert_linear_workspace_bytes(n, dim, hidden, experts),
                   mo.expert_linear_workspace_bytes(n, vocab, dim, 1))
        self.ws = torch.zeros(size, dtype=torch.uint8, device=dev)
        self.sort_ws = torch.empty(mo.embedding_grad_workspace_bytes(n, vocab, dim), dtype=torch.uint8, device=dev)


def route(p, h0):
    """(order of the rows by expert, its inverse, each expert's first row)."""
    expert = (h0.float() @ p["router"]).argmax(1)
    order = torch.argsort(expert, stable=True)
    inverse = torch.empty_like(order).scatter_(0, order, torch.arange(len(order), device=order.device))
    edges = torch.arange(p["router"].shape[1] + 1, device=order.device)
    return order, inverse, torch.searchsorted(expert[order], edges).int()


def forward_backward(p, w, tokens, idx, teacher, weight, temperature):
    """Loss per token; the gradients are left in w.grads."""
    mo.embedding_lookup(p["table"], tokens, w.h0, scale=w.scale)
    order, inverse, offsets = route(p, w.h0)
    mo.embedding_lookup(w.h0, order, w.xs)
    mo.expert_linear(w.xs, p["up"], offsets, w.u, w.ws)
    act = torch.nn.functional.silu(w.u)
    mo.expert_linear(act, p["down"], offsets, w.ys, w.ws)
    mo.embedding_lookup(w.ys, inverse, w.back)
    torch.add(w.h0, w.back, out=w.h1)
    mo.expert_linear(w.h1, p["head"], w.whole, w.logits, w.ws)
    # loss, and the gradient in the logits' place
    mo.distill_topk_loss_grad(w.logits, idx, teacher, w.loss, w.logits, temperature=temperature, row_weight=weight)
    mo.expert_linear_wgrad(w.logits, w.h1, w.whole, w.grads["head"], w.ws)
    mo.expert_linear_dgrad(w.logits, p["head"], w.whole, w.dh1, w.ws)
    mo.embedding_lookup(w.dh1, order, w.dys)
    mo.expert_linear_wgrad(w.dys, act, offsets, w.grads["down"], w.ws)
    mo.expert_linear_dgrad(w.dys, p["down"], offsets, w.da, w.ws)
    s = torch.sigmoid(w.u.float())
    du = (w.da.float() * s * (1 + w.u.float() * (1 - s))).to(BF16)
    mo.expert_linear_wgrad(du, w.xs, offsets, w.grads["up"], w.ws)
    mo.expert_linear_dgrad(du, p["up"], offsets, w.dxs, w.ws)
    mo.embedding_lookup(w.dxs, inverse, w.back)
    mo.embedding_grad(w.dh1 + w.back, tokens, w.grads["table"], w.sort_ws, scale=w.scale)
    return w.loss


class Optimizer:
    """Muon over the expert matrices and the head, AdamW on the embedding table."""

    def __init__(self, p, w, lr=0.02, table_lr=3e-3):
        self.p, self.w, self.t, self.table_lr = p, w, 0, table_lr
        self.momentum = {k: torch.zeros_like(w.grads[k]) for k in ("up", "down", "head")}
        self.m, self.v = torch.zeros_like(p["table"]), torch.zeros_like(p["table"])
        self.cfg = mo.make_cfg(lr=lr, update_scale=0.2 * max(p["table"].shape) ** 0.5)
        self.mats = [mo.make_matrix(p[k][e], self.momentum[k][e], w.grads[k][e])
                     for k in ("up", "down", "head") for e in range(p[k].shape[0])]
        self.ws = torch.empty(mo.mo_workspace_bytes(self.mats, self.cfg), dtype=torch.uint8, device=p["table"].device)

    def step(self):
        self.t += 1
        tail = mo.make_tail(self.p["table"], self.w.grads["table"], self.m, self.v, self.t, lr=self.table_lr)
        mo.muon_step_batched(self.mats, self.cfg, self.ws, tail=tail)


def teacher_of(vocab, top, seed=1, device="cuda"):
    """The teacher's top entries for each token: (places, logits)."""
    g = torch.Generator(device=device).manual_seed(seed)
    places = torch.randint(vocab, (vocab, 1), generator=g, device=device) + torch.arange(top, device=device) * (vocab // top)
    return (places % vocab).int(), torch.randn((vocab, top), generator=g, device=device).mul(2).to(BF16)


def train(steps=60, tokens=4096, vocab=4000, dim=256, hidden=512, experts=8, top=16, temperature=2.0, log=None):
    """Mean loss before each step."""
    p = init(vocab, dim, hidden, experts)
    w = Workspace(p, tokens)
    opt = Optimizer(p, w)
    places, logits = teacher_of(vocab, top)
    weight = torch.full((tokens,), 1.0 / tokens, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    losses = []
    for step in range(steps):
        batch = torch.randint(vocab, (tokens,), generator=g, device="cuda")
        loss = forward_backward(p, w, batch, places[batch], logits[batch], weight, temperature)
        opt.step()
        losses.append(float(loss.sum()))
        if log is not None:
            log(f"step {step}: loss {losses[-1]:.4f}")
    assert mo.mo_check_device_status(w.ws) == 0 and mo.mo_check_device_status(opt.ws) == 0
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=4096)
    args = ap.parse_args()
    train(args.steps, args.tokens, log=print)
