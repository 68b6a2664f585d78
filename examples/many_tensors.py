"""Train a small next-token model whose parameters stay where torch put them.

    python examples/many_tensors.py [--steps 200] [--state-bits 8]

The parameters are bf16 tensors of a few hundred to a few ten thousand
elements with fp32 masters; one MultiAdamW step updates all of them: global
norm and clip, then AdamW with weight decay on the matrices only.  With
--state-bits 8, m and v take 2.06 bytes a parameter instead of 8.  Half way the
states go out as fp32 (a checkpoint's form) and into a second optimizer that
goes on.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from zero_partitioned_mixed_replica_gb300.engine import AdamW  # noqa: E402
from zero_partitioned_mixed_replica_gb300.multi import MultiAdamW  # noqa: E402

VOCAB, DIM, HIDDEN = 97, 64, 192


def parameters(gen):
    shapes = {"embed": (VOCAB, DIM), "in": (DIM, HIDDEN), "in_bias": (HIDDEN,), "out": (HIDDEN, DIM), "norm": (DIM,),
              "head": (DIM, VOCAB)}
    made = {n: torch.randn(s, generator=gen, device="cuda") * 0.05 for n, s in shapes.items()}
    made["norm"].fill_(1.0)
    made["in_bias"].zero_()
    return made


def loss_of(p, x, y):
    h = p["embed"][x].float()
    h = h + torch.relu(h @ p["in"].float() + p["in_bias"].float()) @ p["out"].float()
    h = h / (h.square().mean(-1, keepdim=True) + 1e-5).sqrt() * p["norm"].float()
    return torch.nn.functional.cross_entropy(h @ p["head"].float(), y)


def train(steps=200, state_bits=32, seed=0, batch=512, say=print):
    """Losses of a run whose optimizer is replaced half way by one with the same states."""
    gen = torch.Generator("cuda").manual_seed(seed)
    master = parameters(gen)
    names = list(master)
    model = {n: t.bfloat16().requires_grad_() for n, t in master.items()}
    grads = [torch.zeros_like(model[n]) for n in names]
    groups = [AdamW(lr=3e-3, weight_decay=0.05), AdamW(lr=3e-3, weight_decay=0.0)]

    def optimizer():
        return MultiAdamW([master[n] for n in names], grads, [model[n].detach() for n in names], state_bits=state_bits,
                          groups=groups, group_of_tensor=[int(master[n].ndim < 2) for n in names], max_norm=1.0, seed=seed)

    opt = optimizer()
    rule = torch.randperm(VOCAB, generator=gen, device="cuda")     # the next token is a function of this one
    losses = []
    for step in range(steps):
        if step == steps // 2:
            m, v = opt.states32()
            t = opt.read_state()["t"]
            opt = optimizer()
            opt.load_states(m, v)
            opt.resume_at(t)
        x = torch.randint(VOCAB, (batch,), generator=gen, device="cuda")
        loss = loss_of(model, x, rule[x])
        for g, n in zip(torch.autograd.grad(loss, [model[n] for n in names]), range(len(names))):
            grads[n].copy_(g)
        opt.step()
        losses.append(loss.detach())
    losses = [float(x) for x in losses]
    state = sum(t.numel() * t.element_size() for t in opt.m + opt.v + (opt.m_scale + opt.v_scale if state_bits == 8 else []))
    say("%d-bit states: %d bytes for %d parameters; loss %.3f -> %.3f; grad norm %.3f"
        % (state_bits, state, sum(opt.numels), losses[0], losses[-1], opt.read_state()["grad_norm"]))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--state-bits", type=int, default=8, choices=[8, 32])
    a = ap.parse_args()
    train(a.steps, a.state_bits)
