"""The cross entropy over a vocabulary and its gradients against their definition in 64 bits.

Tolerances, from the arithmetic.  A logit is a float32 sum of H exact products,
each addition rounded or truncated, and one FMA: off by at most
    D = (H + 8) 2^-23 sum |x w| + 2^-21 (|l| + |b|)   (in units of log 2 and back).
A sum of exponentials is off by R of itself: 2^-22 for ex2 and its argument's
rounding (|argument| 2^-24 ln 2, under 2^-18 for the arguments below 90 that
count), and an addition's 2^-24 for each of the at most 64 + V / 256 + 16 on a
value's way.  So a loss is off by 2 D + R + 2^-21 of itself, a probability by
rho = 2 D + R + 2^-21 of itself, and d = p - [v = y] is then rounded once: u |d|
with u = 2^-8 (bfloat16) or 2^-11 (float16, and 2^-25 / 16384 below its normal
range; nothing below 2^-126 is told from 0).  A gradient sums n such terms (n 2^-23 of their magnitudes), and is
rounded to its type.  Rows of unequal weights round weight times x once more.

bfloat16 calls of over 3e9 multiplications hold exp(l - l_y) instead of a
probability: that is off by rho of itself, and so is the factor 1 / (1 + S) by
which it becomes one; for dW and db the factor is rounded with x, as a row's
weight is.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# bfloat16 and float32 reach down to 2^-126; an exponential or a sum below that becomes 0, off by all of itself
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def inputs(rows, vocab, width, dtype=torch.bfloat16, bias=None, ignored=0.0, seed=0, spread=1.5):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    w = (normal(vocab, width) * spread * width ** -0.5).to(dtype)
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    x = (normal(rows, width) + w[target].float()).to(dtype)
    b = None if bias is None else normal(vocab).to(bias)
    drop = torch.rand(rows, generator=g, device="cuda") < ignored
    return x, w, torch.where(drop, -100, target), b


def definition(x, w, target, b, weight, dw_type=None, db_type=None, part_of=None):
    """Losses and gradients in 64 bits with the rows' weights, and how far off each may be.  `part_of`: the rows are some of
    so many, and their share of dw and db is meant, before the final rounding."""
    X, W = x.double(), w.double()
    keep = target != -100
    y = torch.where(keep, target, 0).long()
    V, H, T = w.shape[0], w.shape[1], x.shape[0]
    rows = torch.arange(T, device="cuda")
    l = X @ W.T
    D = (H + 8) * 2.0 ** -23 * (X.abs() @ W.abs().T) + 2.0 ** -21 * l.abs()
    if b is not None:
        l = l + b.double()
        D = D + 2.0 ** -21 * b.double().abs()
    D = torch.where(torch.isfinite(D), D, 0.0).amax(1)
    lse = torch.logsumexp(l, 1)
    logp = l - lse[:, None]
    loss = torch.where(keep, -logp[rows, y], 0.0)
    R = 2.0 ** -22 + 2.0 ** -18 + (80 + V / 256) * 2.0 ** -24
    out = {"losses": (loss, 2 * D + R + 2.0 ** -21 * loss.abs())}
    p = logp.exp()
    d = p.clone()
    d[rows, y] = torch.expm1(logp[rows, y])
    g = torch.where(keep, weight.double(), 0.0)
    u = ROUND[x.dtype]
    unequal = u if float((g[keep] - g[keep].mean()).abs().max() if bool(keep.any()) else 0.0) > 0 else 0.0
    rho = 2 * D + R + 2.0 ** -21
    n = part_of or T
    if x.dtype is torch.bfloat16 and float(n) * V * H > 3e9:
        rho, unequal = 2 * rho, u
    err = p * rho[:, None] + u * d.abs() + max(TINY[x.dtype] / 16384, 2.0 ** -126)
    ga = g.abs()[:, None]

    def final(v, e, dtype):
        return v, e + ROUND[dtype] * (v.abs() + e) + TINY[dtype]
    dx = g[:, None] * (d @ W)
    out["dx"] = final(dx, ga * (err @ W.abs() + (V + 16) * 2.0 ** -23 * (d.abs() @ W.abs())), x.dtype)
    dw = (g[:, None] * d).T @ X
    e = (ga * (err + unequal * d.abs())).T @ X.abs() + (n + 16) * 2.0 ** -23 * ((ga * d.abs()).T @ X.abs())
    out["dw"] = (dw, e) if part_of else final(dw, e, dw_type or w.dtype)
    if b is not None:
        db = (g[:, None] * d).sum(0)
        e = (ga * (err + unequal * d.abs())).sum(0) + (n + 16) * 2.0 ** -23 * (ga * d.abs()).sum(0)
        out["db"] = (db, e) if part_of else final(db, e, db_type or b.dtype)
    return out


def near(name, got, want):
    v, tol = want
    assert got.shape == v.shape, name
    assert bool(torch.isfinite(got).all()), name
    off = (got.double() - v).abs() - tol
    assert not bool((off > 0).any()), (name, int((off > 0).sum()), (off > 0).nonzero()[0].tolist(), float(off.max()))


def check_all(G, x, w, target, b, scale=1.0, reduction="mean"):
    count = int((target != -100).sum())
    one = scale / max(count, 1) if reduction == "mean" else scale
    want = definition(x, w, target, b, torch.full((x.shape[0],), one, device="cuda"))
    near("losses", G.linear_cross_entropy(x, w, target, bias=b, reduction="none"), want["losses"])
    loss, dx, dw, db = G.linear_cross_entropy_grad(x, w, target, bias=b, scale=scale, reduction=reduction)
    v, tol = want["losses"]
    over = max(count, 1) if reduction == "mean" else 1
    if count or reduction == "sum":
        near("loss", loss, (v.sum() / over, tol.sum() / over + 2.0 ** -22 * v.abs().sum() / over))
    else:
        assert math.isnan(float(loss))
    near("dx", dx, want["dx"])
    near("dw", dw, want["dw"])
    if b is not None:
        near("db", db, want["db"])


@pytest.mark.parametrize("rows", [1, 2, 31, 33, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("vocab", [256, 1000])
def test_rows(G, rows, vocab):
    check_all(G, *inputs(rows, vocab, 128, seed=rows))


@pytest.mark.parametrize("vocab", [1, 2, 31, 32, 33, 63, 64, 65, 255, 257, 5003, 33278])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_vocab(G, vocab, dtype):
    check_all(G, *inputs(300, vocab, 72, dtype, bias=dtype, seed=vocab))


@pytest.mark.parametrize("width", [1, 2, 8, 15, 16, 17, 63, 64, 65, 129, 255, 256, 257, 512, 650, 651, 2048])
@pytest.mark.parametrize("bias", [None, torch.bfloat16, torch.float32], ids=str)
def test_width(G, width, bias):
    check_all(G, *inputs(150, 700, width, bias=bias, ignored=0.2, seed=width))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("reduction,scale", [("mean", 1.0), ("mean", 1024.0), ("sum", 1.0), ("sum", -0.37)])
def test_reductions(G, dtype, reduction, scale):
    check_all(G, *inputs(513, 1300, 200, dtype, bias=dtype, ignored=0.4, seed=5), scale=scale, reduction=reduction)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("spread", [0.0, 8.0, 40.0])
def test_flat_and_peaked_rows(G, dtype, spread):
    # at 40 the target or another word takes a row whole, and losses reach hundreds
    check_all(G, *inputs(300, 900, 64, dtype, seed=9, spread=spread))


def test_many_tiles(G):
    check_all(G, *inputs(2240, 12000, 650, bias=torch.bfloat16, seed=11))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=str)
def test_rows_in_chunks(G, kind):
    # a chunk's buffers have 4 GiB: two chunks, the last one shorter
    T, V = 420001, 5003
    x, w, target, b = inputs(T, V, 64, bias=torch.bfloat16, ignored=0.1, seed=13)
    dw, db = torch.empty(V, 64, device="cuda", dtype=kind), torch.empty(V, device="cuda", dtype=kind)
    loss, dx, _, _ = G.linear_cross_entropy_grad(x, w, target, bias=b, reduction="sum", weight_grad=dw, bias_grad=db)
    sums = {"dw": [0.0, 0.0], "db": [0.0, 0.0], "losses": [0.0, 0.0]}
    for s in range(0, T, 60000):
        part = slice(s, min(s + 60000, T))
        n = part.stop - s
        want = definition(x[part], w, target[part], b, torch.ones(n, device="cuda"), part_of=T)
        near("dx", dx[part], want["dx"])
        for name, both in sums.items():
            for i in (0, 1):
                both[i] = both[i] + (want[name][i].sum() if name == "losses" else want[name][i])
    for name, got in (("dw", dw), ("db", db)):
        v, e = sums[name]
        near(name, got, (v, e + ROUND[kind] * (v.abs() + e) + TINY[kind]))
    v, e = sums["losses"]
    assert abs(float(loss) - float(v)) <= float(e) + 2.0 ** -22 * float(v)


def test_strided_operands_and_results(G):
    x, w, target, b = inputs(300, 700, 130, bias=torch.float32, ignored=0.2, seed=17)
    wide_x, wide_w = torch.full((300, 141), 7.0, device="cuda").bfloat16(), torch.full((700, 152), 7.0, device="cuda").bfloat16()
    wide_x[:, 3:133], wide_w[:, 8:138] = x, w
    want = G.linear_cross_entropy_grad(x, w, target, bias=b)
    layout = G.GradientLayout([(5, 7), (700, 130), (700, 0)])
    buf = torch.full((layout.total,), 3.0, device="cuda")
    got = G.linear_cross_entropy_grad(wide_x[:, 3:133], wide_w[:, 8:138], target.int(), bias=b,
                                      weight_grad=layout.layer_view(buf, 1), bias_grad=layout.layer_view(buf, 2))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    untouched = buf.clone()
    layout.layer_view(untouched, 1).fill_(3.0), layout.layer_view(untouched, 2).fill_(3.0)
    assert bool((untouched == 3.0).all())  # padding and the layer in front
    weight = torch.full((300,), 1.0 / int((target != -100).sum()), device="cuda")
    for kind, (dw, db) in ((torch.float32, got[2:]), (torch.bfloat16, want[2:])):
        right = definition(x, w, target, b, weight, kind, torch.float32)
        near("dw", dw, right["dw"]), near("db", db, right["db"])


def test_rows_repeated_by_a_stride_of_zero(G):
    x, w, target, b = inputs(40, 300, 64, seed=18)
    one = x[:1].expand(40, 64)
    a, c = G.linear_cross_entropy_grad(one, w, target), G.linear_cross_entropy_grad(one.contiguous(), w, target)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], c[:3]))


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("width", [128, 130])
def test_accumulate(G, kind, width):
    x, w, target, b = inputs(300, 500, width, bias=torch.bfloat16, seed=19)
    one, two = torch.full((500, width), 2.0, device="cuda", dtype=kind), torch.full((500,), -1.0, device="cuda", dtype=kind)
    _, _, dw, db = G.linear_cross_entropy_grad(x, w, target, bias=b, weight_grad=one.clone(), bias_grad=two.clone())
    G.linear_cross_entropy_grad(x, w, target, bias=b, weight_grad=one, bias_grad=two, accumulate=True)
    # the sums are the same float32 values, here rounded after the addition: two roundings of values up to 4 apart
    for got, start, add in ((one, 2.0, dw), (two, -1.0, db)):
        assert float((got.double() - (start + add.double())).abs().max()) <= 2 * ROUND[kind] * 4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_autograd(G, dtype, reduction):
    x, w, target, b = inputs(400, 600, 96, dtype, bias=dtype, ignored=0.3, seed=21)
    x, w, b = (t.requires_grad_() for t in (x, w, b))
    g = torch.Generator("cuda").manual_seed(1)
    loss = G.linear_cross_entropy(x, w, target, bias=b, reduction=reduction)
    up = torch.randn(loss.shape, generator=g, device="cuda") * 8
    loss.backward(up)
    weight = up if reduction == "none" else (up / int((target != -100).sum()) if reduction == "mean" else up).expand(400)
    want = definition(x.detach(), w.detach(), target, b.detach(), weight)
    for name, t in (("dx", x), ("dw", w), ("db", b)):
        near(name, t.grad, want[name])


def test_autograd_of_some_operands(G):
    x, w, target, b = inputs(100, 300, 64, bias=torch.float32, seed=22)
    full = G.linear_cross_entropy_grad(x, w, target, bias=b)[1:]
    for i, name in enumerate(("x", "w", "b")):
        t = {"x": x, "w": w, "b": b}[name].detach().clone().requires_grad_()
        args = {"x": x, "w": w, "b": b, name: t}
        G.linear_cross_entropy(args["x"], args["w"], target, bias=args["b"]).backward()
        assert torch.equal(t.grad, full[i])
    y = G.linear_cross_entropy(x.detach().requires_grad_(), w, target)
    g, = torch.autograd.grad(y, [y.grad_fn.next_functions[0][0].variable], create_graph=True)
    assert not g.requires_grad or pytest.raises(RuntimeError, g.sum().backward)


def test_gradient_against_differences(G):
    # d loss / d x along a direction, from losses of bfloat16 rows that the direction leaves exact
    x, w, target, _ = inputs(64, 500, 64, seed=23)
    x = (x.float() * 8).round() / 8
    step = torch.zeros_like(x)
    step[:, 5] = 0.125
    f = lambda v: G.linear_cross_entropy(v.bfloat16(), w, target, reduction="none").double()
    slope = (f(x + step) - f(x - step)) / 0.25
    dx = G.linear_cross_entropy_grad(x.bfloat16(), w, target, reduction="sum")[1].double()[:, 5]
    # a third derivative of a softmax is below 2 max|w|^3: h^2 / 6 of it, float32 losses, bfloat16 d and dx
    most = float(w[:, 5].abs().max())
    tol = 0.125 ** 2 / 6 * 2 * most ** 3 + 2.0 ** -18 / 0.125 + 2.0 ** -8 * 3 * most
    assert float((slope - dx).abs().max()) <= tol


def test_ignored_rows_may_hold_anything(G):
    x, w, target, b = inputs(300, 700, 136, bias=torch.bfloat16, ignored=0.5, seed=24)
    target[0], target[1] = -100, 3
    want = G.linear_cross_entropy_grad(x, w, target, bias=b)
    gone = target == -100
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min):
        y = x.clone()
        y[gone] = bad
        got = G.linear_cross_entropy_grad(y, w, target, bias=b)
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        assert bool((got[1][gone] == 0).all())
        losses = G.linear_cross_entropy(y, w, target, bias=b, reduction="none")
        assert bool((losses[gone] == 0).all()) and bool(torch.isfinite(losses).all())


def test_every_row_ignored(G):
    x, w, target, b = inputs(70, 300, 64, bias=torch.bfloat16, seed=25)
    target.fill_(-1)
    loss, dx, dw, db = G.linear_cross_entropy_grad(x, w, target, bias=b, ignore_index=-1)
    assert math.isnan(float(loss))
    assert not dx.any() and not dw.any() and not db.any()
    assert float(G.linear_cross_entropy(x, w, target, ignore_index=-1, reduction="sum")) == 0.0


def test_words_with_a_bias_of_minus_infinity(G):
    x, w, target, b = inputs(90, 300, 64, bias=torch.float32, seed=26)
    target %= 100
    b[100:] = -float("inf")
    want = definition(x, w[:100], target, b[:100], torch.full((90,), 1.0 / 90, device="cuda"))
    loss, dx, dw, db = G.linear_cross_entropy_grad(x, w, target, bias=b)
    near("dx", dx, want["dx"]), near("dw", dw[:100], want["dw"]), near("db", db[:100], want["db"])
    assert not dw[100:].any() and not db[100:].any()
    target[7] = 200  # impossible: an infinite loss
    assert float(G.linear_cross_entropy(x, w, target, bias=b, reduction="none")[7]) == float("inf")


def test_targets_outside_the_vocabulary_give_nan(G):
    x, w, target, _ = inputs(90, 300, 64, seed=27)
    for bad in (300, -1, 2 ** 31 + 5, -2 ** 40):
        t = target.clone()
        t[50] = bad
        losses = G.linear_cross_entropy(x, w, t, reduction="none")
        assert bool(torch.isnan(losses[50])) and int(torch.isnan(losses).sum()) == 1
        loss, dx, dw, _ = G.linear_cross_entropy_grad(x, w, t)
        assert math.isnan(float(loss)) and bool(torch.isnan(dw).all()) and bool(torch.isnan(dx[50]).all())
        assert bool(torch.isfinite(dx[:50]).all())


def test_nan_and_infinity_reach_the_loss(G):
    x, w, target, _ = inputs(90, 300, 64, seed=28)
    x[3, 4] = float("nan")
    losses = G.linear_cross_entropy(x, w, target, reduction="none")
    assert torch.isnan(losses).nonzero().flatten().tolist() == [3]
    assert bool(torch.isnan(G.linear_cross_entropy_grad(x, w, target)[1][3]).all())


def test_no_rows(G):
    w = torch.randn(300, 64, device="cuda").bfloat16()
    x, t, b = w[:0], torch.empty(0, dtype=torch.int64, device="cuda"), torch.zeros(300, device="cuda")
    assert G.linear_cross_entropy(x, w, t, reduction="none").shape == (0,)
    assert float(G.linear_cross_entropy(x, w, t, reduction="sum")) == 0.0
    assert math.isnan(float(G.linear_cross_entropy(x, w, t)))
    loss, dx, dw, db = G.linear_cross_entropy_grad(x, w, t, bias=b, reduction="sum")
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    keep = torch.ones(300, 64, device="cuda")
    G.linear_cross_entropy_grad(x, w, t, reduction="sum", weight_grad=keep, accumulate=True)
    assert bool((keep == 1).all())


def test_the_same_call_twice_gives_the_same_bits(G):
    args = inputs(700, 5003, 650, bias=torch.bfloat16, ignored=0.1, seed=29)
    a, b = (G.linear_cross_entropy_grad(*args[:3], bias=args[3]) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_and_replayed(G):
    x, w, target, b = inputs(300, 1000, 130, bias=torch.bfloat16, ignored=0.2, seed=30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.linear_cross_entropy_grad(x, w, target, bias=b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = G.linear_cross_entropy_grad(x, w, target, bias=b)
        losses = G.linear_cross_entropy(x, w, target, bias=b, reduction="none")
    for seed in (31, 32):
        new = inputs(300, 1000, 130, bias=torch.bfloat16, ignored=0.2, seed=seed)
        for t, n in zip((x, w, target, b), new):
            t.copy_(n)
        graph.replay()
        want = G.linear_cross_entropy_grad(*new[:3], bias=new[3])
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.equal(losses, G.linear_cross_entropy(*new[:3], bias=new[3], reduction="none"))


def test_two_streams_at_once(G):
    sets = [inputs(600, 3001, 200, bias=torch.bfloat16, seed=s) for s in (33, 34)]
    want = [G.linear_cross_entropy_grad(*s[:3], bias=s[3]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(G.linear_cross_entropy_grad(*sets[i][:3], bias=sets[i][3]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(g, want[i]))


def test_refusals(G):
    x, w, target, b = inputs(20, 50, 32, bias=torch.bfloat16, seed=35)
    f, g = G.linear_cross_entropy, G.linear_cross_entropy_grad
    for error, call in ((TypeError, lambda: f(x.float(), w.float(), target)), (TypeError, lambda: f(x, w.half(), target)),
                        (TypeError, lambda: f(x, w, target.float())), (TypeError, lambda: f(x, w, target, bias=b.half())),
                        (ValueError, lambda: f(x, w[:, :31], target)), (ValueError, lambda: f(x, w, target[:19])),
                        (ValueError, lambda: f(x, w, target, bias=b[:49])), (ValueError, lambda: f(x.cpu(), w, target)),
                        (ValueError, lambda: f(x, w, target, reduction="max")), (ValueError, lambda: f(x.t(), w, target)),
                        (ValueError, lambda: f(x, w, target.repeat_interleave(2)[::2])),
                        (ValueError, lambda: g(x, w, target, reduction="none")),
                        (ValueError, lambda: g(x, w, target, accumulate=True)),
                        (ValueError, lambda: g(x, w, target, bias_grad=b)),
                        (ValueError, lambda: g(x, w, target, weight_grad=torch.empty(50, 31, device="cuda"))),
                        (TypeError, lambda: g(x, w, target, weight_grad=w.half())),
                        (G.PsgdError, lambda: g(x, w, target, scale=float("nan")))):
        with pytest.raises(error):
            call()


# bfloat16 calls of over 3e9 multiplications take statistics and exponentials from one product

def test_one_product(G):
    check_all(G, *inputs(2300, 20001, 136, bias=torch.bfloat16, ignored=0.2, seed=36))
    check_all(G, *inputs(5001, 2049, 640, ignored=0.2, seed=37), reduction="sum", scale=3.0)


@pytest.mark.parametrize("bad", [[0], [255, 256], [2047], list(range(0, 2048, 7))], ids=["first", "edge", "last", "many"])
def test_rows_out_of_the_exponentials_range(G, bad):
    # losses of about 45 to 700: their 256 rows are computed another way, the others as before
    x, w, target, b = inputs(2048, 8001, 400, bias=torch.float32, ignored=0.1, seed=38)
    x, w = x.float(), w.float()
    w[:, 0] = 0.0
    w[17, 0], target[target == 17], target[bad[0]] = 1.0, 18, 18
    x[:, 0] = 0.0
    x[bad, 0] = torch.linspace(45, 700, len(bad), device="cuda").bfloat16().float()
    check_all(G, x.bfloat16(), w.bfloat16(), target, b, reduction="sum")


def test_weighted_rows_in_one_product(G):
    x, w, target, b = inputs(2048, 8001, 400, bias=torch.bfloat16, ignored=0.1, seed=39)
    x, w, b = (t.requires_grad_() for t in (x, w, b))
    up = torch.randn(2048, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 8
    G.linear_cross_entropy(x, w, target, bias=b, reduction="none").backward(up)
    want = definition(x.detach(), w.detach(), target, b.detach(), up)
    for name, t in (("dx", x), ("dw", w), ("db", b)):
        near(name, t.grad, want[name])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9])
@pytest.mark.parametrize("width", [1, 2, 7, 64, 200, 650, 651, 1400, 1416, 11300])
def test_few_rows(G, dtype, rows, width):
    for vocab, bias, ignored in ((1, None, 0.0), (3, dtype, 0.0), (1000, torch.float32, 0.4), (5003, dtype, 0.0)):
        x, w, target, b = inputs(rows, vocab, width, dtype, bias=bias, ignored=ignored, seed=rows + width)
        want, tol = definition(x, w, target, b, torch.ones(rows, device="cuda"))["losses"]
        losses = G.linear_cross_entropy(x, w, target, bias=b, reduction="none")
        near("losses", losses, (want, tol))
        near("sum", G.linear_cross_entropy(x, w, target.int(), bias=b, reduction="sum"), (want.sum(), tol.sum() + 2.0 ** -22 * want.abs().sum()))
        count = int((target != -100).sum())
        mean = G.linear_cross_entropy(x, w, target, bias=b)
        assert math.isnan(float(mean)) if not count else abs(float(mean) - float(want.sum()) / count) <= float(
            tol.sum() + 2.0 ** -22 * want.abs().sum()) / count
    t = target.clone()
    t[-1] = 5003
    assert torch.isnan(G.linear_cross_entropy(x, w, t, bias=b, reduction="none")).nonzero().flatten().tolist() == [rows - 1]


@pytest.mark.parametrize("dtype,rows", [(torch.bfloat16, 300), (torch.bfloat16, 4096), (torch.float16, 300)], ids=str)
def test_what_was_abandoned_is_nan_and_told_of(G, dtype, rows):
    # nothing is loaded, and the waits run out after 50 ms each; 4096 rows are over 3e9 multiplications
    x, w, target, b = inputs(rows, 6000, 256, dtype, bias=dtype, seed=40)
    buf, half = torch.ones(6000, 256, device="cuda"), torch.ones(6000, 256, device="cuda", dtype=dtype)
    bg = torch.ones(6000, device="cuda")
    want = G.linear_cross_entropy_grad(x, w, target, bias=b)
    G.experts_sync()
    for call in (lambda: G.linear_cross_entropy_grad(x, w, target, bias=b, weight_grad=buf, bias_grad=bg),
                 lambda: G.linear_cross_entropy_grad(x, w, target, bias=b, weight_grad=half),
                 lambda: (G.linear_cross_entropy(x, w, target, bias=b, reduction="none"),)):
        assert G.lib().psgd_experts_set_wait(50, 1) == 0
        try:
            got = call()
            torch.cuda.current_stream().synchronize()
        finally:
            assert G.lib().psgd_experts_set_wait(0, 0) == 0
        for t in got:
            assert bool(torch.isnan(t).all())
        with pytest.raises(G.PsgdError) as e:
            G.experts_sync()
        assert e.value.code == G.PSGD_ERR_TIMEOUT
    again = G.linear_cross_entropy_grad(x, w, target, bias=b)
    G.experts_sync()
    assert all(torch.equal(p, q) for p, q in zip(want, again))


def test_a_padding_word_is_ignored(G):
    x, w, target, b = inputs(120, 300, 64, bias=torch.bfloat16, ignored=0.3, seed=41)
    padded = torch.where(target == -100, 0, torch.where(target == 0, 1, target))
    want = definition(x, w, torch.where(padded == 0, -100, padded), b, torch.full((120,), 1.0, device="cuda"))
    loss, dx, dw, db = G.linear_cross_entropy_grad(x, w, padded, bias=b, ignore_index=0, reduction="sum")
    near("dx", dx, want["dx"]), near("dw", dw, want["dw"]), near("db", db, want["db"])
    near("losses", G.linear_cross_entropy(x, w, padded, bias=b, ignore_index=0, reduction="none"), want["losses"])


@pytest.mark.parametrize("rows", [1, 24])
def test_a_matrix_past_32_bit_offsets(G, rows):
    # 2.2e9 values of w and dw: the last words against their definition, given the rows' logarithms of the sums
    V, H, end = 1 << 20, 2056, 1000
    g = torch.Generator("cuda").manual_seed(5)
    w = torch.empty(V, H, device="cuda", dtype=torch.bfloat16).normal_(0.0, 0.02, generator=g)
    x = torch.randn(rows, H, generator=g, device="cuda").bfloat16()
    target = torch.randint(V - end, V, (rows,), generator=g, device="cuda")
    losses = G.linear_cross_entropy(x, w, target, reduction="none").double()
    X, tail = x.double(), w[-end:].double()
    l = X @ tail.T
    y = target - (V - end)
    at = torch.arange(rows, device="cuda")
    # the whole sum, a share of the words at a time
    top = torch.full((rows,), -float("inf"), device="cuda", dtype=torch.float64)
    for s in range(0, V, 1 << 17):
        top = torch.logaddexp(top, torch.logsumexp(X @ w[s:s + (1 << 17)].double().T, 1))
    D = (H + 8) * 2.0 ** -23 * (X.abs() @ tail.abs().T).amax(1) * 2
    assert bool(((losses - (top - l[at, y])).abs() <= 2 * D + 2.0 ** -17 + 2.0 ** -21 * losses.abs()).all())
    if rows == 1:
        return
    dw = torch.empty(V, H, device="cuda", dtype=torch.bfloat16)
    _, dx, _, _ = G.linear_cross_entropy_grad(x, w, target, reduction="sum", weight_grad=dw)
    d = (l - top[:, None]).exp()
    d[at, y] -= 1.0
    want = d.T @ X
    # rounded: the probability (or its row's factor) twice, the result once; a probability is off by 2 rho
    tol = (d.abs() * (2 * 2.0 ** -8 + 4 * D[:, None] + 2.0 ** -16)).T @ X.abs() + 2.0 ** -8 * want.abs() + 2.0 ** -126
    assert bool(((dw[-end:].double() - want).abs() <= tol * 1.01).all())
    assert bool(torch.isfinite(dx).all())
