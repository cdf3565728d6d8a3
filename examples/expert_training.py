"""Training an expert layer with compressed gradients.

A two-matrix expert layer (each token goes to one of E experts) learns the
outputs of a fixed teacher layer.  W data-parallel workers, simulated on one
GPU, each take their own tokens:

    rows sorted by expert -> experts_forward -> relu -> experts_forward -> loss
    -> experts_grad_weight, straight into the worker's packed gradient buffer
       (one layer of the compression step per expert matrix),
       experts_grad_input for the layer below
    -> clip_grad_norm: each worker's gradient to the same global norm
    -> PowerSGD.step_momentum: rank-r compression with error feedback, the mean
       over the workers, and the momentum update of the float32 parameters

    python examples/expert_training.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from rank_gradient_compression_layer_gb300 import (GradientLayout, PowerSGD, build, experts_forward,  # noqa: E402
                                                   experts_grad_input, experts_grad_weight, experts_sync)

EXPERTS, WIDTH, HIDDEN, TOKENS, WORKERS, RANK = 8, 256, 512, 2048, 2, 4


def sort_by_expert(expert: torch.Tensor):
    """(order, offsets): tokens in the experts' order, and where each expert's rows start."""
    order = torch.argsort(expert, stable=True)
    counts = torch.bincount(expert, minlength=EXPERTS)
    offsets = torch.zeros(EXPERTS + 1, dtype=torch.int32, device=expert.device)
    offsets[1:] = counts.cumsum(0)
    return order, offsets


def layer(x, up, down, offsets):
    """Both products of the layer; (hidden before and after relu, output)."""
    h = experts_forward(x, up, offsets)
    a = torch.relu(h)
    return h, a, experts_forward(a, down, offsets)


def train(steps: int = 30, lr: float = 1.0, beta: float = 0.5, max_norm: float = 4.0, verbose: bool = True):
    g = torch.Generator("cuda").manual_seed(0)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    shapes = [(HIDDEN, WIDTH)] * EXPERTS + [(WIDTH, HIDDEN)] * EXPERTS
    layout = GradientLayout(shapes)
    params = torch.zeros(layout.total, device="cuda")
    momentum = torch.zeros_like(params)
    up, down = layout.experts_view(params, 0, EXPERTS), layout.experts_view(params, EXPERTS, EXPERTS)
    up.copy_(normal(*up.shape, scale=WIDTH ** -0.5))
    down.copy_(normal(*down.shape, scale=HIDDEN ** -0.5))
    teacher = normal(*up.shape, scale=WIDTH ** -0.5), normal(*down.shape, scale=HIDDEN ** -0.5)
    router = normal(WIDTH, EXPERTS)
    grads = [torch.zeros_like(params) for _ in range(WORKERS)]
    ctx = PowerSGD(shapes, RANK, WORKERS, seed=1)
    losses = []
    for step in range(steps):
        w1, w2 = up.bfloat16(), down.bfloat16()
        loss = 0.0
        for w in range(WORKERS):
            x = normal(TOKENS, WIDTH)
            order, offsets = sort_by_expert((x @ router).argmax(1))
            x = x[order]
            target = layer(x, *teacher, offsets)[2]
            h, a, y = layer(x, w1, w2, offsets)
            diff = y.float() - target.float()
            loss += float(diff.square().mean()) / WORKERS
            dy = (diff * (2.0 / TOKENS)).bfloat16()
            experts_grad_weight(dy, a, offsets, out=layout.experts_view(grads[w], EXPERTS, EXPERTS))
            dh = experts_grad_input(dy, w2, offsets) * (h > 0)
            experts_grad_weight(dh, x, offsets, out=layout.experts_view(grads[w], 0, EXPERTS))
        norms = ctx.clip_grad_norm(grads, max_norm)
        ctx.step_momentum(grads, params, momentum, lr, beta)
        losses.append(loss)
        if verbose and step % 5 == 0:
            print(f"step {step:3d}  loss {loss:.4f}  gradient norms {[round(v, 3) for v in norms.tolist()]}", flush=True)
    experts_sync()
    ctx.sync()
    ctx.close()
    return losses


if __name__ == "__main__":
    build()
    history = train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
    print(f"loss {history[0]:.4f} -> {history[-1]:.4f}")
