"""The expert products against their definition in 64 bits.

Tolerance, from the arithmetic: the operands are exact, a product of two of
them is exact in float32, and a float32 sum of D terms in any order, each
addition rounded or truncated, is off by at most (D + 8) 2^-23 sum |a b|
(8 additions for joining partial sums).  The result is rounded once more:
2^-8 (bfloat16), 2^-11 (float16, and 2^-25 below its normal range), 2^-24
(float32) of itself.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def offsets_of(sizes, first=0):
    return torch.from_numpy(np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)).cuda()


def rand(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def definition(op, rows, other, offsets, k=None):
    """(result, sum of absolute products, terms) in float64; rows of no expert are 0."""
    off = [min(max(int(v), 0), rows.shape[0]) for v in offsets.tolist()]
    for i in range(1, len(off)):
        off[i] = max(off[i], off[i - 1])
    a, b = rows.double(), other.double()
    E = len(off) - 1
    if op == "grad_weight":
        shape = (E, a.shape[1], b.shape[1])
    else:
        shape = (a.shape[0], b.shape[1] if op == "forward" else b.shape[2])
    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for e in range(E):
        s, t = off[e], off[e + 1]
        if s == t:
            continue
        if op == "forward":
            out[s:t], mag[s:t] = a[s:t] @ b[e].T, a[s:t].abs() @ b[e].abs().T
        elif op == "grad_input":
            out[s:t], mag[s:t] = a[s:t] @ b[e], a[s:t].abs() @ b[e].abs()
        else:
            out[e], mag[e] = a[s:t].T @ b[s:t], a[s:t].abs().T @ b[s:t].abs()
    if op == "grad_weight":
        terms = max(off[i + 1] - off[i] for i in range(E))
    else:
        terms = b.shape[2] if op == "forward" else b.shape[1]
    return out, mag, terms


def check(got, want):
    out, mag, terms = want
    u = ROUND[got.dtype]
    tol = u * out.abs() + (1 + u) * (terms + 8) * 2.0 ** -23 * mag + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    err = (got.double() - out).abs()
    assert got.shape == out.shape
    assert bool(torch.isfinite(got).all())
    bad = err > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist(), float((err - tol).max()))


def run(G, op, rows, other, offsets, out=None):
    f = {"forward": G.experts_forward, "grad_input": G.experts_grad_input, "grad_weight": G.experts_grad_weight}[op]
    return f(rows, other, offsets, out=out)


def operands(op, T, E, n, k, dtype, seed=0):
    rows = rand(seed, T, k if op == "forward" else n, dtype=dtype)
    if op == "grad_weight":
        return rows, rand(seed + 1, T, k, dtype=dtype)
    return rows, rand(seed + 1, E, n, k, dtype=dtype)


OPS = ("forward", "grad_input", "grad_weight")
GROUPS = [[1], [0], [0, 1, 0], [2, 0, 1, 5], [15, 16, 17], [31, 32, 33, 0, 1], [63, 64, 65], [127, 128, 129],
          [255, 256, 257, 0], [300, 0, 513, 1], [1000]]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("sizes", GROUPS, ids=str)
@pytest.mark.parametrize("nk", [(64, 64), (256, 128), (328, 264), (8, 520)], ids=str)
def test_group_sizes(G, op, sizes, nk):
    n, k = nk
    off = offsets_of(sizes)
    rows, other = operands(op, sum(sizes), len(sizes), n, k, torch.bfloat16)
    check(run(G, op, rows, other, off), definition(op, rows, other, off))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("nk", [(1, 1), (1, 200), (7, 9), (65, 33), (130, 650), (255, 257), (1365, 651), (72, 1048),
                                (1024, 96)], ids=str)
def test_sides(G, op, dtype, nk):
    n, k = nk
    sizes = [37, 0, 130, 1, 64]
    off = offsets_of(sizes)
    rows, other = operands(op, sum(sizes), len(sizes), n, k, dtype, seed=3)
    check(run(G, op, rows, other, off), definition(op, rows, other, off))


@pytest.mark.parametrize("op", OPS)
def test_many_tiles(G, op):
    sizes = [700, 0, 1301, 256, 64, 2, 511]
    off = offsets_of(sizes)
    rows, other = operands(op, sum(sizes), len(sizes), 1288, 776, torch.bfloat16, seed=5)
    check(run(G, op, rows, other, off), definition(op, rows, other, off))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("experts", [64, 2048])
def test_many_experts(G, op, experts):
    rng = np.random.RandomState(1)
    sizes = rng.randint(0, 4, experts) * rng.randint(0, 2, experts)
    off = offsets_of(sizes)
    rows, other = operands(op, int(sizes.sum()), experts, 64, 72, torch.float16, seed=7)
    check(run(G, op, rows, other, off), definition(op, rows, other, off))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 31])
@pytest.mark.parametrize("nk", [(256, 512), (1024, 2048), (100, 300)], ids=str)
def test_few_rows_of_many_experts(G, op, rows, nk):
    # single tokens: every row another expert's, then all rows one expert's
    n, k = nk
    for sizes in ([1 if i % 2 else 0 for i in range(2 * rows)], [0, rows, 0]):
        off = offsets_of(sizes)
        r, o = operands(op, rows, len(sizes), n, k, torch.bfloat16, seed=9)
        check(run(G, op, r, o, off), definition(op, r, o, off))


@pytest.mark.parametrize("op", OPS)
def test_rows_of_no_expert(G, op):
    # 5 rows before the first expert, 40 behind the last: zero rows, and no part of any weight gradient
    sizes = [20, 0, 33]
    off = offsets_of(sizes, first=5)
    rows, other = operands(op, 5 + 53 + 40, 3, 264, 200, torch.bfloat16, seed=11)
    rows[:5] = float("nan")
    rows[58:] = float("inf")
    if op == "grad_weight":
        other[:5] = float("inf")
        other[58:] = float("nan")
    keep = rows.clone()
    keep[:5] = 0
    keep[58:] = 0
    other_keep = torch.nan_to_num(other, 0.0, 0.0, 0.0)
    check(run(G, op, rows, other, off), definition(op, keep, other_keep, off))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("sizes", [[17, 30, 5], [64, 1, 63], [3, 2, 4]], ids=str)
def test_one_experts_nan_stays_its_own(G, op, sizes):
    off = offsets_of(sizes)
    rows, other = operands(op, sum(sizes), 3, 136, 264, torch.bfloat16, seed=13)
    a, b = sizes[0], sizes[0] + sizes[1]
    rows[a:b] = float("nan")
    if op == "grad_weight":
        other[a:b] = float("inf")
    else:
        other[1] = float("nan")
    got = run(G, op, rows, other, off)
    zr, zo = rows.clone(), other.clone()
    zr[a:b] = 0
    if op == "grad_weight":
        zo[a:b] = 0
    else:
        zo[1] = 0
    out, mag, terms = definition(op, zr, zo, off)
    keep = torch.ones(got.shape[0], dtype=torch.bool, device="cuda")
    if op == "grad_weight":
        keep[1] = False
    else:
        keep[a:b] = False
    assert bool(torch.isnan(got[~keep]).all())
    check(got[keep], (out[keep], mag[keep], terms))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("case", ["strided", "misaligned", "broadcast"])
def test_layouts(G, op, case):
    sizes = [70, 0, 45]
    T, n, k = 115, 264, 200
    off = offsets_of(sizes)
    rows, other = operands(op, T, 3, n, k, torch.bfloat16, seed=15)

    def lay(t):
        if case == "strided":  # rows 24 values further apart, experts one row further
            big = torch.full((*t.shape[:-2], t.shape[-2] + 1, t.shape[-1] + 24), float("nan"), dtype=t.dtype, device="cuda")
            v = big[..., :t.shape[-2], :t.shape[-1]]
        elif case == "misaligned":  # one value behind a 16-byte boundary
            v = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        else:  # one row, or one matrix, for all
            return t[:1].expand(t.shape)
        v.copy_(t)
        return v
    rows, other = lay(rows), lay(other)
    want = definition(op, rows, other, off)
    check(run(G, op, rows, other, off), want)
    dt = torch.float32 if op == "grad_weight" else torch.bfloat16
    shape = want[0].shape
    big = torch.full((*shape[:-1], shape[-1] + 3), 7.0, dtype=dt, device="cuda")
    out = big[..., 1:1 + shape[-1]]
    assert run(G, op, rows, other, off, out=out) is out
    check(out, want)
    assert bool((big[..., 0] == 7).all()) and bool((big[..., 1 + shape[-1]:] == 7).all())


def test_weight_gradient_types_and_packed_buffer(G):
    sizes = [33, 0, 90]
    off = offsets_of(sizes)
    dy, x = operands("grad_weight", 123, 3, 70, 130, torch.bfloat16, seed=17)
    want = definition("grad_weight", dy, x, off)
    check(G.experts_grad_weight(dy, x, off, out=torch.empty(3, 70, 130, dtype=torch.bfloat16, device="cuda")), want)
    layout = G.GradientLayout([(9, 0)] + [(70, 130)] * 3 + [(5, 7)])
    buf = torch.full((layout.total,), 3.0, device="cuda")
    G.experts_grad_weight(dy, x, off, out=layout.experts_view(buf, 1, 3))
    for e in range(3):
        check(layout.layer_view(buf, 1 + e).contiguous()[None], (want[0][e:e + 1], want[1][e:e + 1], want[2]))
    assert bool((layout.layer_view(buf, 0) == 3).all()) and bool((layout.layer_view(buf, 4) == 3).all())


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("values", [[0, 50, 20, 90], [-7, 10, 200, 200], [30, 30, 10, 5]], ids=str)
def test_offsets_out_of_order_stay_inside(G, op, values):
    off = torch.tensor(values, dtype=torch.int32, device="cuda")
    rows, other = operands(op, 90, 3, 72, 104, torch.bfloat16, seed=19)
    check(run(G, op, rows, other, off), definition(op, rows, other, off))


@pytest.mark.parametrize("op", OPS)
def test_no_rows(G, op):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    rows, other = operands(op, 0, 3, 40, 24, torch.bfloat16)
    got = run(G, op, rows, other, off)
    assert got.shape == ((3, 40, 24) if op == "grad_weight" else (0, 40 if op == "forward" else 24))
    assert bool((got == 0).all())


@pytest.mark.parametrize("op", OPS)
def test_other_stream_and_repeatability(G, op):
    sizes = [100, 30, 0, 260]
    off = offsets_of(sizes)
    rows, other = operands(op, 390, 4, 520, 392, torch.bfloat16, seed=21)
    first = run(G, op, rows, other, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = [run(G, op, rows, other, off) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(first, a) for a in again)
    check(first, definition(op, rows, other, off))


def test_gradient_against_differences(G):
    # the product is linear in x and in w, so a difference of any length is the derivative times it
    sizes = [40, 0, 77]
    off = offsets_of(sizes)
    x, w = rand(1, 117, 96), rand(2, 3, 160, 96)
    g = rand(3, 117, 160)
    xv, wv = rand(4, 117, 96), rand(5, 3, 160, 96)
    xs, ws = (x.float() + xv.float()).bfloat16(), (w.float() + wv.float()).bfloat16()
    xv, wv = xs.double() - x.double(), ws.double() - w.double()  # the step that was taken

    def loss(x_, w_):
        y = G.experts_forward(x_, w_, off)
        return float((y.double() * g.double()).sum()), float((y.double() * g.double()).abs().sum())
    l0, m0 = loss(x, w)
    lx, mx = loss(xs, w)
    lw, mw = loss(x, ws)
    dx = G.experts_grad_input(g, w, off).double()
    dw = G.experts_grad_weight(g, x, off).double()
    # each y is off by at most 2^-8 of itself (and the float32 sums, far less), dx too
    tol = 2.0 ** -7.9
    assert abs((lx - l0) - float((dx * xv).sum())) <= tol * (mx + m0 + float((dx * xv).abs().sum()))
    assert abs((lw - l0) - float((dw * wv).sum())) <= tol * (mw + m0 + float((dw * wv).abs().sum()))


def test_linear_is_differentiable(G):
    sizes = [40, 0, 77]
    off = offsets_of(sizes)
    x, w, g = rand(1, 117, 96).requires_grad_(), rand(2, 3, 160, 96).requires_grad_(), rand(3, 117, 160)
    G.experts_linear(x, w, off).backward(g)
    check(x.grad, definition("grad_input", g, w.detach(), off))
    check(w.grad, definition("grad_weight", g, x.detach(), off))
    buf = torch.full((3, 160, 96), 5.0, device="cuda")
    x2 = x.detach().clone().requires_grad_()
    G.experts_linear(x2, w.detach(), off, weight_grad=buf).sum().backward()  # an expanded gradient
    check(buf, definition("grad_weight", torch.ones_like(g), x.detach(), off))


def test_refusals(G):
    off = offsets_of([3, 4])
    x, w = rand(1, 7, 16), rand(2, 2, 24, 16)
    ok = G.experts_forward(x, w, off)
    assert ok.shape == (7, 24)
    with pytest.raises(TypeError):
        G.experts_forward(x.float(), w.float(), off)
    with pytest.raises(TypeError):
        G.experts_forward(x, w.half(), off)
    with pytest.raises(TypeError):
        G.experts_forward(x, w, off.long())
    with pytest.raises(ValueError):
        G.experts_forward(x, w[:1], off)
    with pytest.raises(ValueError):
        G.experts_forward(x[:, :8], w, off)
    with pytest.raises(ValueError):
        G.experts_forward(rand(1, 16, 7).t(), w, off)
    with pytest.raises(ValueError):
        G.experts_forward(x, w, off.cpu())
    with pytest.raises(ValueError):
        G.experts_forward(x, w, off, out=torch.empty(7, 25, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        G.experts_forward(x, w, off, out=torch.empty(7, 24, device="cuda"))
    with pytest.raises(ValueError):
        G.experts_grad_input(x, w, off)
    with pytest.raises(ValueError):
        G.experts_grad_weight(x, x[:6], off)
    with pytest.raises(ValueError):
        G.experts_forward(x, w, torch.zeros(2050, dtype=torch.int32, device="cuda"))
    with pytest.raises(G.PsgdError):  # results that would overlap themselves
        G.experts_forward(x, w, off, out=torch.empty(1, 24, dtype=torch.bfloat16, device="cuda").expand(7, 24))


@pytest.mark.parametrize("op", ["forward", "grad_input"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("case", [([1], 64, 8192), ([5], 250, 4097), ([300, 0, 41], 256, 2048), ([0, 2], 1000, 3000),
                                  ([700], 120, 6000)], ids=str)
def test_long_contraction_of_few_tiles(G, op, dtype, case):
    # summed in parts; 3 rows of no expert behind the last
    sizes, side, depth = case
    off = offsets_of(sizes)
    n, k = (side, depth) if op == "forward" else (depth, side)
    rows, other = operands(op, sum(sizes) + 3, len(sizes), n, k, dtype, seed=23)
    got = run(G, op, rows, other, off)
    check(got, definition(op, rows, other, off))
    assert torch.equal(got, run(G, op, rows, other, off))


@pytest.mark.parametrize("sizes", [[5000], [3001, 0, 17, 1025, 64], [1, 2047, 4, 4100], [1025] * 5], ids=str)
@pytest.mark.parametrize("nk", [(256, 256), (250, 131), (512, 700), (8, 40)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_many_rows_of_small_weights(G, sizes, nk, dtype):
    # experts of many rows are cut into segments, the others are not
    n, k = nk
    off = offsets_of(sizes, first=2)
    dy, x = operands("grad_weight", sum(sizes) + 5, len(sizes), n, k, torch.bfloat16, seed=25)
    out = torch.empty(len(sizes), n, k, dtype=dtype, device="cuda")
    want = definition("grad_weight", dy, x, off)
    check(G.experts_grad_weight(dy, x, off, out=out), want)
    again = G.experts_grad_weight(dy, x, off, out=torch.empty_like(out))
    assert torch.equal(out, again)


def test_without_room_for_parts(G):
    # the C entry runs without a workspace too, the contraction then in one piece
    off = offsets_of([6])
    x, w = rand(27, 6, 4096), rand(28, 1, 128, 4096)
    y = torch.empty(6, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert G.lib().psgd_experts_forward(6, 1, 128, 4096, G.PSGD_BF16, x.data_ptr(), 4096, w.data_ptr(), 4096, 128 * 4096,
                                        off.data_ptr(), y.data_ptr(), 128, None, 0, s) == 0
    check(y, definition("forward", x, w, off))
    dy, x = rand(29, 6000, 64), rand(30, 6000, 72)
    off = offsets_of([6000])
    dw = torch.empty(1, 64, 72, device="cuda")
    assert G.lib().psgd_experts_grad_weight(6000, 1, 64, 72, G.PSGD_BF16, dy.data_ptr(), 64, x.data_ptr(), 72,
                                            off.data_ptr(), G.PSGD_F32, dw.data_ptr(), 72, 64 * 72, None, 0, s) == 0
    check(dw, definition("grad_weight", dy, x, off))


@pytest.mark.parametrize("op", OPS)
def test_a_wait_that_runs_out_is_reported(G, op):
    # nothing is loaded: every role's waits end after 50 ms, the kernel returns, the host hears of it
    off = offsets_of([300, 0, 41])
    rows, other = operands(op, 341, 3, 264, 200, torch.bfloat16, seed=31)
    G.experts_sync()
    assert G.lib().psgd_experts_set_wait(50, 1) == 0
    try:
        run(G, op, rows, other, off)
        with pytest.raises(G.PsgdError) as e:
            G.experts_sync()
        assert e.value.code == G.PSGD_ERR_TIMEOUT
    finally:
        assert G.lib().psgd_experts_set_wait(0, 0) == 0
    check(run(G, op, rows, other, off), definition(op, rows, other, off))
    G.experts_sync()
