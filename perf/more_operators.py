"""The cases in which the loss over a vocabulary, dropout and the root-mean-square norm are measured.

Three operators that stand between the embedding and the compression step of a language model's training:

* the softmax cross entropy of a linear layer over a large vocabulary, whose logits are never kept, and its gradients
  in the rows, the matrix and the bias;
* dropout whose mask comes from a counter-based generator (Philox 4x32 with 10 rounds) and is never stored;
* the root-mean-square norm of a residual stream to which a branch, with dropout, is added in the same pass, and its
  gradients.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the framework's operators.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
IGNORED = -100

# the work of the largest listed case of each operator; a drawn case stays within it
MOST_MACS = 16384 * 65536 * 2048
MOST_LOGITS = 16384 * 65536
MOST_MATRIX = 65536 * 2048
MOST_DROPPED = 32768 * 8192
MOST_NORMED = 32768 * 2048


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # The loss of one token, as in scoring a text word by word: the LSTM set's 33278 x 650 matrix is read once.
        {"name": "loss_one_token", "op": "loss", "dtype": "bf16", "rows": 1, "vocab": 33278, "width": 650, "bias": True,
         "ignored": 0.0, "scale": 1.0},
        # An evaluation batch of the LSTM set, 10 sequences of 35 words: between reading the matrix and arithmetic.
        {"name": "loss_evaluation", "op": "loss", "dtype": "bf16", "rows": 350, "vocab": 33278, "width": 650, "bias": True,
         "ignored": 0.0, "scale": 1.0},
        # A training batch of the LSTM set, 64 sequences of 35 words: rows of 650, whose gradients are dense.
        {"name": "loss_train_lstm", "op": "train", "dtype": "bf16", "rows": 2240, "vocab": 33278, "width": 650,
         "bias": True, "ignored": 0.0, "scale": 1.0},
        # Odd sizes in every dimension, padded sequences, float16 with a loss scale.
        {"name": "loss_train_odd", "op": "train", "dtype": "f16", "rows": 1001, "vocab": 5003, "width": 651, "bias": False,
         "ignored": 0.3, "scale": 1024.0},
        # A training batch of the transformer set's width over a large vocabulary: bound by arithmetic.
        {"name": "loss_train_large", "op": "train", "dtype": "bf16", "rows": 16384, "vocab": 65536, "width": 2048,
         "bias": False, "ignored": 0.1, "scale": 1.0},
        # Dropout behind a recurrent layer of the LSTM set, 20 sequences of 35 steps: latency.
        {"name": "dropout_lstm", "op": "dropout", "dtype": "f32", "rows": 700, "width": 650, "p": 0.65},
        # Dropout on the hidden values of a training batch of the transformer set: bound by memory.
        {"name": "dropout_hidden", "op": "dropout", "dtype": "bf16", "rows": 32768, "width": 8192, "p": 0.1},
        # One row of a residual stream: latency.
        {"name": "norm_one_row", "op": "norm", "dtype": "bf16", "rows": 1, "width": 2048, "residual": True, "p": 0.0},
        # The norm in front of a layer of the transformer set, with the branch's dropout and addition.
        {"name": "norm_train", "op": "norm", "dtype": "bf16", "rows": 32768, "width": 2048, "residual": True, "p": 0.1},
        # Its gradients.
        {"name": "norm_grad_train", "op": "norm_grad", "dtype": "bf16", "rows": 32768, "width": 2048, "residual": True,
         "p": 0.1},
        # Gradients of rows that do not start on 16-byte boundaries, no dropout.
        {"name": "norm_grad_odd", "op": "norm_grad", "dtype": "f16", "rows": 5003, "width": 651, "residual": True,
         "p": 0.0},
        # The gradients in float32, without a residual stream.
        {"name": "norm_grad_float32", "op": "norm_grad", "dtype": "f32", "rows": 8192, "width": 1500, "residual": False,
         "p": 0.0},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.random()
    if kind < 0.45:
        while True:
            rows, vocab, width = log(1, 32768), log(256, 131072), log(64, 4096)
            if rng.random() < 0.7:  # whole 16-byte rows
                width = max(64, width // 8 * 8)
            if rows * vocab * width <= MOST_MACS and rows * vocab <= MOST_LOGITS and vocab * width <= MOST_MATRIX:
                break
        dtype = rng.choice(("bf16", "bf16", "f16"))
        return {"op": rng.choice(("loss", "train", "train")), "dtype": dtype, "rows": rows, "vocab": vocab, "width": width,
                "bias": rng.random() < 0.5, "ignored": rng.choice((0.0, round(rng.uniform(0.0, 0.9), 2))),
                "scale": 1024.0 if dtype == "f16" else 1.0}
    dtype = rng.choice(("bf16", "f16", "f32"))
    if kind < 0.65:
        while True:
            rows, width = log(1, 32768), log(8, 8192)
            if rows * width <= MOST_DROPPED // 2:
                break
        return {"op": "dropout", "dtype": dtype, "rows": rows, "width": width, "p": round(rng.uniform(0.02, 0.9), 3)}
    while True:
        rows, width = log(1, 32768), log(32, 16384)
        if rng.random() < 0.7:
            width = max(32, width // 8 * 8)
        if rows * width <= MOST_NORMED // (2 if dtype == "f32" else 1):
            break
    return {"op": rng.choice(("norm", "norm_grad")), "dtype": dtype, "rows": rows, "width": width,
            "residual": rng.random() < 0.7, "p": rng.choice((0.0, round(rng.uniform(0.02, 0.5), 3)))}


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    T, H = case["rows"], case["width"]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    state = dict(case)
    if case["op"] in ("loss", "train"):
        V = case["vocab"]
        # frequent words are the first ones; a row of a trained model leans towards its target
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        target = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
        state["w"] = normal(V, H, scale=1.5 * H ** -0.5)
        state["x"] = normal(T, H).add_(state["w"][target], alpha=2.0)
        if case["bias"]:
            state["b"] = normal(V, scale=0.5)
        drop = torch.rand(T, generator=g, device="cuda") < case["ignored"]
        drop[:1] = False
        state["target"] = torch.where(drop, IGNORED, target)
        return state
    # where the generator stands: seed and step
    state["state"] = torch.tensor([seed * 0x9E3779B1 + 12345, seed % 1000], dtype=torch.int64, device="cuda")
    state["x"] = normal(T, H)
    if case["op"] == "dropout":
        return state
    state["w"] = normal(H, scale=0.1).add_(1.0)
    if case["op"] == "norm":
        if case["residual"]:
            state["res"] = normal(T, H, scale=2.0)
    else:
        state["r"] = state.pop("x").mul_(2.0)
        state["dy"] = normal(T, H, scale=1e-2)
        if case["residual"]:
            state["dr"] = normal(T, H, scale=1e-2)
    return state


# ------------------------------------------------------------ plain forms --

def plain_loss(s):
    valid = s["target"] != IGNORED
    count = valid.sum()
    target = torch.where(valid, s["target"], 0)
    x, w = s["x"].float(), s["w"].float()
    logits = x @ w.T
    if s["bias"]:
        logits += s["b"].float()
    top = logits.amax(1, keepdim=True)
    mine = logits.gather(1, target[:, None]) - top
    p = logits.sub_(top).exp_()
    total = p.sum(1, keepdim=True)
    losses = torch.where(valid, (total.log() - mine)[:, 0], 0.0)
    if s["op"] == "loss":
        return losses
    loss = losses.sum() / count
    g = torch.where(valid, s["scale"] / count, 0.0)[:, None]
    p.div_(total).scatter_add_(1, target[:, None], torch.full_like(g, -1.0)).mul_(g)
    out = {"loss": loss, "dx": (p @ w).to(s["x"].dtype), "dw": (p.T @ x).to(s["w"].dtype)}
    if s["bias"]:
        out["db"] = p.sum(0).to(s["b"].dtype)
    return out


def plain_bits(state, n):
    """16 random bits for each of n values: value i takes half i % 8 of Philox's words for counter i // 8."""
    low = 0xFFFFFFFF
    group = torch.arange(-(-n // 8), device="cuda")
    c = [group & low, group >> 32, (state[1] & low).expand_as(group), ((state[1] >> 32) & low).expand_as(group)]
    k0, k1 = state[0] & low, (state[0] >> 32) & low

    def product(m, v):  # high and low word of a 32 by 32 bit product
        return ((m * (v >> 16) + ((m * (v & 0xFFFF)) >> 16)) >> 16) & low, (m * v) & low

    for _ in range(10):
        h0, l0 = product(0xD2511F53, c[0])
        h1, l1 = product(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]


def plain_drop(s, x):
    """x in 32 bits with dropout."""
    cut = round(s["p"] * 65536)
    kept = plain_bits(s["state"], x.numel()).view_as(x) >= cut
    return torch.where(kept, x * (65536.0 / (65536 - cut)), 0.0)


def plain_norm(s):
    x, dt = s["x"].float(), s["x"].dtype
    if s["p"]:
        x = plain_drop(s, x)
    if s["residual"]:
        x = x + s["res"].float()
    r = x.to(dt)
    f = r.float()
    rstd = (f.square().mean(1, keepdim=True) + EPS).rsqrt()
    return {"y": (f * rstd * s["w"].float()).to(dt), "r": r}


def plain_norm_grad(s):
    r, dy, dt = s["r"].float(), s["dy"].float(), s["r"].dtype
    rstd = (r.square().mean(1, keepdim=True) + EPS).rsqrt()
    n = r * rstd
    g = dy * s["w"].float()
    dr = rstd * (g - n * (g * n).mean(1, keepdim=True))
    if s["residual"]:
        dr = dr + s["dr"].float()
    return {"dr": dr.to(dt), "dx": (plain_drop(s, dr) if s["p"] else dr).to(dt), "dw": (dy * n).sum(0)}


# -------------------------------------------------------------------- run --

def run(s):
    op = s["op"]
    if not own:
        if op in ("loss", "train"):
            return plain_loss(s)
        if op == "dropout":
            return plain_drop(s, s["x"].float()).to(s["x"].dtype)
        return plain_norm(s) if op == "norm" else plain_norm_grad(s)
    import rank_gradient_compression_layer_gb300 as G
    if op == "loss":
        return G.linear_cross_entropy(s["x"], s["w"], s["target"], bias=s.get("b"), reduction="none")
    if op == "train":
        loss, dx, dw, db = G.linear_cross_entropy_grad(s["x"], s["w"], s["target"], bias=s.get("b"), scale=s["scale"])
        out = {"loss": loss, "dx": dx, "dw": dw}
        if s["bias"]:
            out["db"] = db
        return out
    if op == "dropout":
        return G.dropout(s["x"], s["p"], s["state"])
    if op == "norm":
        y, r = G.rms_norm(s["x"], s["w"], residual=s.get("res"), eps=EPS, p=s["p"], state=s["state"])
        return {"y": y, "r": r}
    dx, dr, dw = G.rms_norm_grad(s["dy"], s["r"], s["w"], dr=s.get("dr"), eps=EPS, p=s["p"], state=s["state"])
    return {"dr": dr, "dx": dx, "dw": dw}


# ------------------------------------------------------------------- work --

def work(case):
    T, H = case["rows"], case["width"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("loss", "train"):
        V = case["vocab"]
        once = (T * H + V * H + V * case["bias"]) * size
        train = case["op"] == "train"
        return {"bytes": once * (2 if train else 1) + (8 if train else 12) * T, "flops": (6.0 if train else 2.0) * T * V * H}
    if case["op"] == "dropout":
        return {"bytes": 2 * T * H * size, "flops": T * H}
    if case["op"] == "norm":  # x, the residual stream in, and out where it changes, y
        rows = 2 + case["residual"] + bool(case["residual"] or case["p"])
        return {"bytes": (rows * T * H + H) * size, "flops": 4.0 * T * H}
    rows = 3 + case["residual"] + bool(case["p"])
    return {"bytes": (rows * T * H + H) * size + 4 * H, "flops": 10.0 * T * H}


# ------------------------------------------------------------------ exact --

def exact_kept(case, state):
    """Which values are kept, from the generator's definition in unsigned 64-bit numbers on the host."""
    n = case["rows"] * case["width"]
    seed, step = (np.uint64(int(v) & 0xFFFFFFFFFFFFFFFF) for v in state.tolist())
    word, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    key = [int(seed & word), int(seed >> half)]
    a = np.arange((n + 7) // 8, dtype=np.uint64)
    b, c, d = a >> half, np.full_like(a, step & word), np.full_like(a, step >> half)
    a = a & word
    for r in range(10):
        k0, k1 = ((k + r * w) & 0xFFFFFFFF for k, w in zip(key, (0x9E3779B9, 0xBB67AE85)))
        p, q = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, d = (q >> half) ^ b ^ np.uint64(k0), q & word, (p >> half) ^ d ^ np.uint64(k1), p & word
    bits = np.empty((a.size, 8), dtype=np.int32)
    for j, w in enumerate((a, b, c, d)):
        bits[:, 2 * j], bits[:, 2 * j + 1] = w & np.uint64(0xFFFF), w >> np.uint64(16)
    cut = round(case["p"] * 65536)
    return torch.from_numpy(bits.reshape(-1)[:n] >= cut).view(case["rows"], case["width"]).cuda(), 65536 / (65536 - cut)


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    T, H = case["rows"], case["width"]
    if case["op"] in ("loss", "train"):
        if 6.0 * T * case["vocab"] * H > 4e12:
            return None
        valid = s["target"] >= 0
        x, w = s["x"][valid].double(), s["w"].double()
        y = s["target"][valid]
        a = torch.addmm(s["b"].double(), x, w.T) if case["bias"] else x @ w.T
        logp = a - torch.logsumexp(a, 1, keepdim=True)
        n = x.shape[0]
        losses = torch.zeros(T, device="cuda", dtype=torch.float64)
        losses[valid] = -logp[torch.arange(n, device="cuda"), y]
        if case["op"] == "loss":
            return losses
        loss = losses.sum() / n
        d = logp.exp()
        d[torch.arange(n, device="cuda"), y] = torch.expm1(logp[torch.arange(n, device="cuda"), y])
        d *= case["scale"] / n
        dx = torch.zeros(T, H, device="cuda", dtype=torch.float64)
        dx[valid] = d @ w
        out = {"loss": loss, "dx": dx, "dw": d.T @ x}
        if case["bias"]:
            out["db"] = d.sum(0)
        return out
    if T * H > 1 << 27:
        return None
    kept, times = exact_kept(case, s["state"]) if case["p"] else (None, 1.0)

    def drop(t):
        return t * times * kept if case["p"] else t

    if case["op"] == "dropout":
        return drop(s["x"].double())
    w = s["w"].double()
    if case["op"] == "norm":
        r = drop(s["x"].double())
        if case["residual"]:
            r = r + s["res"].double()
        return {"y": r / torch.sqrt((r * r).mean(1, keepdim=True) + EPS) * w, "r": r}
    r, dy = s["r"].double(), s["dy"].double()
    size = torch.sqrt((r * r).mean(1, keepdim=True) + EPS)
    n = r / size
    dr = (dy * w - n * (dy * w * n).mean(1, keepdim=True)) / size
    if case["residual"]:
        dr = dr + s["dr"].double()
    return {"dr": dr, "dx": drop(dr), "dw": (dy * n).sum(0)}
