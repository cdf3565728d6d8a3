"""Training a small language model with compressed gradients.

A model that predicts the next token: an embedding, a residual block whose
branch is a layer of experts, and a linear layer over the vocabulary.  W
data-parallel workers, simulated on one GPU, each take their own tokens:

    embedding -> rms_norm -> experts_forward -> relu -> experts_forward
    -> rms_norm of the residual stream, to which it adds the branch with dropout
    -> dropout -> linear_cross_entropy_grad: the loss, the rows' gradient, and
       the vocabulary's matrix and bias gradients, straight into the worker's
       packed gradient buffer
    -> the same backwards: dropout, rms_norm_grad, experts_grad_weight and
       experts_grad_input, all into that buffer
    -> clip_grad_norm, then PowerSGD.step_momentum: compression, the mean over the
       workers, and the momentum update of the float32 parameters

    python examples/language_training.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from rank_gradient_compression_layer_gb300 import (GradientLayout, PowerSGD, build, dropout, dropout_state,  # noqa: E402
                                                   experts_forward, experts_grad_input, experts_grad_weight, experts_sync,
                                                   linear_cross_entropy_grad, rms_norm, rms_norm_grad)

WORDS, WIDTH, HIDDEN, EXPERTS, TOKENS, WORKERS, RANK, DROP = 1003, 128, 256, 4, 1024, 2, 4, 0.1
BRANCH, HEAD = 1, 2  # the places that drop: their masks differ

# one layer of the packed buffer each, matrices and vectors (0 columns)
SHAPES = ([(HIDDEN, WIDTH)] * EXPERTS + [(WIDTH, HIDDEN)] * EXPERTS + [(WORDS, WIDTH)] * 2
          + [(WIDTH, 0), (WIDTH, 0), (WORDS, 0)])


def parts(layout: GradientLayout, buf: torch.Tensor) -> dict:
    """The parameters, or their gradients, in a packed buffer."""
    e = EXPERTS
    last = [layout.layer_view(buf, i) for i in range(2 * e, len(SHAPES))]
    return {"up": layout.experts_view(buf, 0, e), "down": layout.experts_view(buf, e, e), "embedding": last[0],
            "head": last[1], "norm1": last[2], "norm2": last[3], "bias": last[4]}


def sort_by_expert(tokens: torch.Tensor):
    """(order, offsets): token t goes to expert t % EXPERTS."""
    expert = tokens % EXPERTS
    order = torch.argsort(expert, stable=True)
    offsets = torch.zeros(EXPERTS + 1, dtype=torch.int32, device=tokens.device)
    offsets[1:] = torch.bincount(expert, minlength=EXPERTS).cumsum(0)
    return order, offsets


def gradients(p: dict, tokens: torch.Tensor, target: torch.Tensor, state: torch.Tensor, out: dict) -> torch.Tensor:
    """One worker's loss; its gradients go into the views of `out`.  `p`: the
    parameters in bfloat16 (the norms' and the bias's may be float32)."""
    order, offsets = sort_by_expert(tokens)
    tokens, target = tokens[order], target[order]
    x = p["embedding"][tokens]
    n1, r1 = rms_norm(x, p["norm1"])
    h = experts_forward(n1, p["up"], offsets)
    a = torch.relu(h)
    branch = experts_forward(a, p["down"], offsets)
    n2, r2 = rms_norm(branch, p["norm2"], residual=r1, p=DROP, state=state, site=BRANCH)
    z = dropout(n2, DROP, state, site=HEAD)
    loss, dz, _, _ = linear_cross_entropy_grad(z, p["head"], target, bias=p["bias"], weight_grad=out["head"],
                                               bias_grad=out["bias"])
    dn2 = dropout(dz, DROP, state, site=HEAD)
    dbranch, dr1, _ = rms_norm_grad(dn2, r2, p["norm2"], p=DROP, state=state, site=BRANCH, weight_grad=out["norm2"])
    experts_grad_weight(dbranch, a, offsets, out=out["down"])
    dh = experts_grad_input(dbranch, p["down"], offsets) * (h > 0)
    experts_grad_weight(dh, n1, offsets, out=out["up"])
    dn1 = experts_grad_input(dh, p["up"], offsets)
    dx, _, _ = rms_norm_grad(dn1, r1, p["norm1"], dr=dr1, weight_grad=out["norm1"])
    out["embedding"].zero_().index_add_(0, tokens, dx.float())
    return loss


def in_half(p: dict) -> dict:
    """What the products take: matrices in bfloat16."""
    return {k: v.bfloat16() if v.dim() > 1 else v.contiguous() for k, v in p.items()}


def first_parameters(layout: GradientLayout, g: torch.Generator) -> torch.Tensor:
    params = torch.zeros(layout.total, device="cuda")
    for name, v in parts(layout, params).items():
        if name.startswith("norm"):
            v.fill_(1.0)
        elif v.dim() > 1:
            v.copy_(torch.randn(v.shape, generator=g, device="cuda") * v.shape[-1] ** -0.5)
    return params


def train(steps: int = 30, lr: float = 0.3, beta: float = 0.5, max_norm: float = 1.0, verbose: bool = True):
    g = torch.Generator("cuda").manual_seed(0)
    layout = GradientLayout(SHAPES)
    params = first_parameters(layout, g)
    momentum = torch.zeros_like(params)
    grads = [torch.zeros_like(params) for _ in range(WORKERS)]
    following = torch.randperm(WORDS, generator=g, device="cuda")  # the language: each word's next one
    states = [dropout_state(seed) for seed in range(WORKERS)]
    ctx = PowerSGD(SHAPES, RANK, WORKERS, seed=1)
    losses = []
    for step in range(steps):
        p = in_half(parts(layout, params))
        loss = 0.0
        for w in range(WORKERS):
            tokens = torch.randint(0, WORDS, (TOKENS,), generator=g, device="cuda")
            loss = loss + gradients(p, tokens, following[tokens], states[w], parts(layout, grads[w])) / WORKERS
            states[w][1] += 1  # the next step's masks
        norms = ctx.clip_grad_norm(grads, max_norm)
        ctx.step_momentum(grads, params, momentum, lr, beta)
        losses.append(float(loss))
        if verbose and step % 5 == 0:
            print(f"step {step:3d}  loss {losses[-1]:.4f}  gradient norms {[round(v, 3) for v in norms.tolist()]}", flush=True)
    experts_sync()
    ctx.sync()
    ctx.close()
    return losses


if __name__ == "__main__":
    build()
    history = train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
    print(f"loss {history[0]:.4f} -> {history[-1]:.4f}")
