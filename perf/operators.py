"""The cases in which the expert products and the gradient norm and clipping are measured.

Two families that stand next to each other in a training step of a model with expert layers:

* the matrix products grouped by expert (rows sorted by expert, ragged group sizes): the forward product, the input
  gradient, and the weight gradient, whose float32 matrices are what the compression step takes;
* the global norm of a set of gradients and clipping by it, over lists of tensors and over the packed buffers of
  several workers.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the framework's operators.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PRODUCTS = ("forward", "grad_input", "grad_weight")
NORMS = ("norm", "clip")

# sizes of the largest listed case of each family; a drawn case stays within them
MOST_MACS = 32768 * 8192 * 2048
MOST_WEIGHTS = 8 * 8192 * 2048
MOST_ROW_VALUES = 32768 * 10240
MOST_GRADIENTS = 24 * (4 * 2048 * 2048 + 2 * 2048 * 8192)


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # One token of a sparse model, sent to 8 of 64 experts: latency, and the weights of 8 experts.
        {"name": "forward_one_token", "op": "forward", "dtype": "bf16", "rows": 8, "experts": 64, "empty": 0,
         "skew": 0.0, "n": 1024, "k": 2048},
        # A short batch over many small experts, unevenly loaded and some without rows: bound by the weights.
        {"name": "forward_many_experts", "op": "forward", "dtype": "f16", "rows": 4099, "experts": 64, "empty": 5,
         "skew": 0.8, "n": 1024, "k": 2048},
        # A training batch through 8 large experts (the transformer set's 2048 x 8192 matrices): bound by arithmetic.
        {"name": "forward_training", "op": "forward", "dtype": "bf16", "rows": 32768, "experts": 8, "empty": 0,
         "skew": 0.3, "n": 8192, "k": 2048},
        # The LSTM set's hidden size 650, whose rows are not 16-byte aligned, and odd group sizes.
        {"name": "forward_hidden_650", "op": "forward", "dtype": "bf16", "rows": 5003, "experts": 13, "empty": 2,
         "skew": 0.5, "n": 2600, "k": 650},
        # The input gradient of the training batch.
        {"name": "grad_input_training", "op": "grad_input", "dtype": "bf16", "rows": 32768, "experts": 8, "empty": 0,
         "skew": 0.3, "n": 8192, "k": 2048},
        # Few rows and odd sizes in every dimension.
        {"name": "grad_input_odd", "op": "grad_input", "dtype": "f16", "rows": 1001, "experts": 5, "empty": 1,
         "skew": 1.0, "n": 1365, "k": 651},
        # The weight gradient of the training batch: float32 matrices for the compression step.
        {"name": "grad_weight_training", "op": "grad_weight", "dtype": "bf16", "rows": 32768, "experts": 8,
         "empty": 0, "skew": 0.3, "n": 8192, "k": 2048},
        # The weight gradient of many experts with few rows each: bound by writing the matrices.
        {"name": "grad_weight_many_experts", "op": "grad_weight", "dtype": "bf16", "rows": 4099, "experts": 64,
         "empty": 5, "skew": 0.8, "n": 1024, "k": 2048},
        # The norm of one 256 x 128 gradient: latency.
        {"name": "norm_256x128", "op": "norm", "dtype": "f32", "set": "list", "tensors": 1, "total": 32768,
         "workers": 1},
        # The norms of four workers' packed gradients of the LSTM set, whose rows of 650 are padded to 652.
        {"name": "norm_lstm_packed", "op": "norm", "dtype": "f32", "set": "lstm", "tensors": 0, "total": 0,
         "workers": 4},
        # Clipping four workers' packed gradients of the ResNet-18 set, right before the compression step.
        {"name": "clip_resnet18_packed", "op": "clip", "dtype": "f32", "set": "resnet18", "tensors": 0, "total": 0,
         "workers": 4},
        # Clipping the 144 bfloat16 gradients of the 1.2 billion parameter transformer set.
        {"name": "clip_transformer", "op": "clip", "dtype": "bf16", "set": "transformer", "tensors": 0, "total": 0,
         "workers": 1},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.6:
        experts = log(1, 64)
        while True:
            rows, n, k = log(1, 32768), log(64, 8192), log(64, 8192)
            if rng.random() < 0.7:  # whole 16-byte rows
                n, k = max(64, n // 8 * 8), max(64, k // 8 * 8)
            if (rows * n * k <= MOST_MACS and experts * n * k <= MOST_WEIGHTS and rows * (n + k) <= MOST_ROW_VALUES):
                break
        return {"op": rng.choice(PRODUCTS), "dtype": rng.choice(("bf16", "f16")), "rows": rows, "experts": experts,
                "empty": rng.randrange(0, (experts + 1) // 2), "skew": round(rng.uniform(0.0, 1.2), 2), "n": n, "k": k}
    op = rng.choice(NORMS)
    if rng.random() < 0.25:
        return {"op": op, "dtype": "f32", "set": rng.choice(("lstm", "resnet18")), "tensors": 0, "total": 0,
                "workers": rng.randrange(1, 9)}
    dtype = rng.choice(("f32", "bf16", "f16"))
    total = log(1000, MOST_GRADIENTS // (2 if dtype == "f32" else 1))
    return {"op": op, "dtype": dtype, "set": "list", "tensors": log(1, 300), "total": total, "workers": 1}


# ------------------------------------------------------------------ sizes --

def group_sizes(case):
    """Rows of each expert, largest first: shares that fall as a power of the rank, and `empty` experts without rows."""
    E, T = case["experts"], case["rows"]
    used = E - case["empty"]
    share = np.arange(1, used + 1, dtype=np.float64) ** -case["skew"]
    want = T * share / share.sum()
    got = np.floor(want).astype(np.int64)
    for i in np.argsort(-(want - got), kind="stable")[:T - int(got.sum())]:
        got[i] += 1
    return np.concatenate([got, np.zeros(E - used, dtype=np.int64)])


def layer_shapes(name):
    """(rows, columns) of the gradients of the framework's own training sets; 0 columns for a vector."""
    if name == "transformer":
        return ([(2048, 2048)] * 4 + [(2048, 8192)] * 2) * 24
    if name == "lstm":
        vectors = [(2600, 0)] * 6 + [(33278, 0)]
        return [(33278, 650)] + [(2600, 650)] * 6 + vectors
    width = [64] * 5 + [128] * 5 + [256] * 5 + [512] * 5
    return ([(64, 27)] + [(64, 576)] * 4 + [(128, 576)] + [(128, 1152)] * 3 + [(128, 64)] + [(256, 1152)]
            + [(256, 2304)] * 3 + [(256, 128)] + [(512, 2304)] + [(512, 4608)] * 3 + [(512, 256)] + [(10, 512)]
            + [(c, 0) for c in width for _ in range(2)] + [(10, 0)])


def shapes_of(case):
    """The gradients' shapes: a set's, or `tensors` vectors of very different lengths that make `total` values."""
    if case["set"] != "list":
        return layer_shapes(case["set"])
    share = np.arange(1, case["tensors"] + 1, dtype=np.float64) ** -1.5
    sizes = np.floor(case["total"] * share / share.sum()).astype(np.int64)
    sizes[0] += case["total"] - int(sizes.sum())
    return [(int(s), 0) for s in sizes]


def packed(case):
    return case["set"] in ("lstm", "resnet18")


def packed_layout(shapes):
    """Per layer (offset, row stride), and the length: rows padded to four values, layers on four-value boundaries."""
    at, where = 0, []
    for n, m in shapes:
        ld = -(-m // 4) * 4
        where.append((at, ld))
        at += n * ld if m else -(-n // 4) * 4
    return where, at


def packed_views(buf, shapes):
    where, _ = packed_layout(shapes)
    return [buf[o:o + n * ld].view(n, ld)[:, :m] if m else buf[o:o + n] for (n, m), (o, ld) in zip(shapes, where)]


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt).mul_(scale)

    if case["op"] in PRODUCTS:
        sizes = np.random.RandomState(seed % 2 ** 32).permutation(group_sizes(case))
        T, N, K = case["rows"], case["n"], case["k"]
        offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda()
        state = {"op": case["op"], "offsets": offsets, "most": int(sizes.max())}
        if case["op"] != "grad_input":
            state["x"] = normal(T, K)
        if case["op"] != "forward":
            state["dy"] = normal(T, N)
        if case["op"] != "grad_weight":
            state["w"] = normal(case["experts"], N, K, scale=K ** -0.5)
        return state

    shapes = shapes_of(case)
    state = {"op": case["op"], "packed": packed(case), "shapes": shapes}
    if packed(case):
        _, total = packed_layout(shapes)
        bufs = [torch.zeros(total, device="cuda", dtype=dt) for _ in range(case["workers"])]
        for buf in bufs:
            for v in packed_views(buf, shapes):
                v.copy_(normal(*v.shape, scale=1e-3))
        state["grads"] = bufs
        state["out"] = [torch.zeros_like(b) for b in bufs]
        if own:
            from rank_gradient_compression_layer_gb300 import GradientLayout
            state["layout"] = GradientLayout(shapes)
    else:
        shapes = [s if s[1] else (s[0],) for s in shapes]
        state["grads"] = [normal(*s, scale=1e-3) for s in shapes]
        state["flat"] = torch.empty(sum(t.numel() for t in state["grads"]), device="cuda", dtype=dt)
        parts = state["flat"].split([t.numel() for t in state["grads"]])
        state["out"] = [p.view(t.shape) for p, t in zip(parts, state["grads"])]
    state["max_norm"] = 1.0
    return state


# ------------------------------------------------------------ plain forms --

def expert_of_row(offsets, rows):
    return torch.bucketize(torch.arange(rows, device="cuda", dtype=torch.int32), offsets[1:], right=True)


def grouped(t, offsets, expert, most):
    """Rows sorted by expert -> (experts, most, columns) in 32 bits, zeros behind each group; and the rows' places."""
    place = torch.arange(t.shape[0], device="cuda") - offsets[expert].long()
    out = torch.zeros(offsets.numel() - 1, most, t.shape[1], device="cuda")
    out[expert, place] = t.float()
    return out, place


def plain_product(s):
    rows = (s["dy"] if "dy" in s else s["x"])
    expert = expert_of_row(s["offsets"], rows.shape[0])
    if s["op"] == "grad_weight":
        dy, _ = grouped(s["dy"], s["offsets"], expert, s["most"])
        x, _ = grouped(s["x"], s["offsets"], expert, s["most"])
        return torch.bmm(dy.transpose(1, 2), x)
    g, place = grouped(rows, s["offsets"], expert, s["most"])
    w = s["w"].float()
    out = torch.bmm(g, w if s["op"] == "grad_input" else w.transpose(1, 2))
    return out[expert, place].to(rows.dtype)


def plain_norm(tensors):
    return torch.stack([t.float().square().sum() for t in tensors]).sum().sqrt()


def plain_scale(tensors, out, norm, max_norm):
    c = (max_norm / (norm + 1e-6)).clamp(max=1.0)
    return [o.copy_(t.float() * c) for t, o in zip(tensors, out)]


def plain_gradients(s):
    sets = [packed_views(b, s["shapes"]) for b in s["grads"]] if s["packed"] else [s["grads"]]
    norms = torch.stack([plain_norm(v) for v in sets])
    if s["op"] == "norm":
        return norms
    outs = [packed_views(b, s["shapes"]) for b in s["out"]] if s["packed"] else [s["out"]]
    _ = [plain_scale(v, o, c, s["max_norm"]) for v, o, c in zip(sets, outs, norms)]
    return {"norm": norms, "clipped": s["out"] if s["packed"] else s["flat"]}


# -------------------------------------------------------------------- run --

def run(s):
    if not own:
        return plain_product(s) if s["op"] in PRODUCTS else plain_gradients(s)
    import rank_gradient_compression_layer_gb300 as G
    if s["op"] == "forward":
        return G.experts_forward(s["x"], s["w"], s["offsets"])
    if s["op"] == "grad_input":
        return G.experts_grad_input(s["dy"], s["w"], s["offsets"])
    if s["op"] == "grad_weight":
        return G.experts_grad_weight(s["dy"], s["x"], s["offsets"])
    if s["packed"]:
        if s["op"] == "norm":
            return s["layout"].grad_norm(s["grads"])
        return {"norm": s["layout"].clip_grad_norm(s["grads"], s["max_norm"], out=s["out"]), "clipped": s["out"]}
    if s["op"] == "norm":
        return G.grad_norm(s["grads"]).view(1)
    return {"norm": G.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"]).view(1), "clipped": s["flat"]}


# ------------------------------------------------------------------- work --

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] in PRODUCTS:
        T, N, K, E = case["rows"], case["n"], case["k"], case["experts"]
        if case["op"] == "grad_weight":
            moved = T * (N + K) * size + E * N * K * 4
        else:
            moved = T * (N + K) * size + int((group_sizes(case) > 0).sum()) * N * K * size
        return {"bytes": moved, "flops": 2.0 * T * N * K}
    values = sum(n * (m or 1) for n, m in shapes_of(case)) * case["workers"]
    return {"bytes": values * size * (2 if case["op"] == "clip" else 1), "flops": values * (3.0 if case["op"] == "clip" else 2.0)}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """The definitions in 64 bits, one expert and one tensor at a time."""
    s = prepare(case, seed)
    if case["op"] in PRODUCTS:
        ends = s["offsets"].tolist()
        T, N, K, E = case["rows"], case["n"], case["k"], case["experts"]
        if case["op"] == "grad_weight":
            out = torch.zeros(E, N, K, device="cuda", dtype=torch.float64)
        else:
            out = torch.zeros(T, N if case["op"] == "forward" else K, device="cuda", dtype=torch.float64)
        for e in range(E):
            a, b = ends[e], ends[e + 1]
            if a == b:
                continue
            if case["op"] == "forward":
                out[a:b] = s["x"][a:b].double() @ s["w"][e].double().T
            elif case["op"] == "grad_input":
                out[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
            else:
                out[e] = s["dy"][a:b].double().T @ s["x"][a:b].double()
        return out
    norms, clipped = [], []
    for w in range(case["workers"]):
        values = [s["grads"][w]] if packed(case) else s["grads"]  # the padding holds zeros
        total = 0.0
        for t in values:
            total += float(t.double().pow(2).sum())
        norms.append(math.sqrt(total))
        if case["op"] == "clip":
            c = min(1.0, s["max_norm"] / (norms[-1] + 1e-6))
            clipped.append(torch.cat([t.reshape(-1).double() * c for t in values]))
    norm = torch.tensor(norms, dtype=torch.float64)
    if case["op"] == "norm":
        return norm
    return {"norm": norm, "clipped": clipped if packed(case) else clipped[0]}
