"""The gradient norm and clipping against their definition in 64 bits.

Tolerance, from the arithmetic: a sum of squares is float32 over at most 8
chained multiply-adds and 2 additions (10 x 2^-24 of a sum without cancelling),
float64 after that; the square root halves it, and the norm is rounded once:
8 x 2^-24 bounds the norm.  The factor adds one rounding to that and the
product one: 10 x 2^-24, plus 2^-8 (bfloat16) or 2^-11 (float16, and 2^-25
below its normal range) where the result has fewer bits.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def norm_of(tensors):
    return math.sqrt(sum(float(t.double().pow(2).sum()) for t in tensors))


def near(got, want):
    assert got.dtype == torch.float32
    assert abs(float(got) - want) <= 8 * 2.0 ** -24 * want + 1e-45, (float(got), want)


def check_clipped(got, grads, want_norm, max_norm):
    c = min(1.0, max_norm / (want_norm + 1e-6))
    for o, g in zip(got, grads):
        want = g.double() * c
        tol = (10 * 2.0 ** -24 + ROUND[g.dtype] * 1.001) * want.abs() + (2.0 ** -25 if g.dtype == torch.float16 else 1e-45)
        assert o.shape == g.shape
        assert bool(((o.double() - want).abs() <= tol).all())


SIZES = [[1], [3], [4], [5], [7, 9], [4095], [4096], [4097], [8191, 1, 8193], [1000003], [17] * 300, [64, 0, 9, 0]]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_lists(G, dtype, sizes, max_norm):
    grads = [rand(i, s, dtype=dtype) for i, s in enumerate(sizes)]
    want = norm_of(grads)
    near(G.grad_norm(grads), want)
    keep = [g.clone() for g in grads]
    out = [torch.empty_like(g) for g in grads]
    near(G.clip_grad_norm(grads, max_norm, out=out), want)
    check_clipped(out, keep, want, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    near(G.clip_grad_norm(grads, max_norm), want)  # in place
    assert all(torch.equal(a, b) for a, b in zip(grads, out))


@pytest.mark.parametrize("count", [447, 448, 449, 1500])
def test_more_tensors_than_one_launch_takes(G, count):
    grads = [rand(i, 1 + i % 37) for i in range(count)]
    want = norm_of(grads)
    near(G.grad_norm(grads), want)
    keep = [g.clone() for g in grads]
    near(G.clip_grad_norm(grads, 1.0), want)
    check_clipped(grads, keep, want, 1.0)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_large(G, dtype):
    # several tiles for each block of threads
    grads = [rand(1, 3000, 5001, dtype=dtype), rand(2, 70001, dtype=dtype), rand(3, 2048, 2048, dtype=dtype)]
    want = norm_of(grads)
    near(G.grad_norm(grads), want)
    keep = [g.clone() for g in grads]
    near(G.clip_grad_norm(grads, 2.0), want)
    check_clipped(grads, keep, want, 2.0)


@pytest.mark.parametrize("value", [1e25, 3e19, 1e-25, 1e-30, 0.0])
def test_range(G, value):
    # squares that overflow or vanish in float32; the norm itself does not
    g = torch.full((5000,), value, device="cuda")
    g[::3] = 0
    want = norm_of([g])
    near(G.grad_norm([g]), want)
    keep = g.clone()
    near(G.clip_grad_norm([g], 1.0), want)
    check_clipped([g], [keep], want, 1.0)


def test_infinite_and_nan(G):
    g = rand(1, 9000)
    g[77] = float("inf")
    out = torch.empty_like(g)
    assert float(G.clip_grad_norm([g], 1.0, out=[out])) == math.inf
    assert math.isnan(float(out[77])) and int((out != 0).sum()) == 1
    g[5000] = float("nan")
    assert math.isnan(float(G.clip_grad_norm([g], 1.0, out=[out])))
    assert bool(torch.isnan(out).all())


def test_max_norm_zero(G):
    g = rand(1, 333)
    G.clip_grad_norm([g], 0.0)
    assert bool((g == 0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_strides_and_alignment(G, dtype):
    base = rand(1, 40, 130, dtype=dtype)
    flat = rand(2, 5000, dtype=dtype)
    chan = rand(3, 4, 6, 5, 7, dtype=dtype).to(memory_format=torch.channels_last)
    grads = [base[:, :100], base[3:20, 101:104], base.t()[105:130], flat[1:4999], chan, flat[4999:],
             rand(4, 6, 64, dtype=dtype)[:, 8:40]]
    want = norm_of(grads)
    near(G.grad_norm(grads), want)
    out = [torch.empty_like(g) for g in grads]
    near(G.clip_grad_norm(grads, 0.25, out=[o if i != 3 else torch.empty(5001, dtype=dtype, device="cuda")[2:5000]
                                            for i, o in enumerate(out)]), want)
    outs = [torch.empty_strided(g.shape, g.stride(), dtype=dtype, device="cuda") for g in grads]
    near(G.clip_grad_norm(grads, 0.25, out=outs), want)
    check_clipped(outs, grads, want, 0.25)
    wide = [torch.full((g.shape[0], 200), 9.0, dtype=dtype, device="cuda") for g in grads[:2]]
    near(G.clip_grad_norm(grads[:2], 0.25, out=[o[:, 5:5 + g.shape[1]] for o, g in zip(wide, grads)]), norm_of(grads[:2]))
    for o, g in zip(wide, grads):
        check_clipped([o[:, 5:5 + g.shape[1]]], [g], norm_of(grads[:2]), 0.25)
        assert bool((o[:, :5] == 9).all()) and bool((o[:, 5 + g.shape[1]:] == 9).all())


def test_gradients_and_outputs_with_other_gaps(G):
    # the same rows further apart, contiguous on either side, and the same order of permuted dimensions
    wide = rand(1, 4, 6, 10)[:, :, :7]
    pairs = [(wide, torch.empty(4, 6, 13, device="cuda")[:, :, 2:9]), (wide, torch.empty(4, 6, 7, device="cuda")),
             (rand(2, 4, 6, 7), torch.empty(4, 6, 9, device="cuda")[:, :, :7]),
             (rand(3, 9, 5).t(), torch.empty(9, 8, device="cuda")[:, 1:6].t()),
             (rand(4, 4, 7, 7)[:, :6], torch.empty(4, 9, 7, device="cuda")[:, 2:8])]
    grads, out = [p[0] for p in pairs], [p[1] for p in pairs]
    want = norm_of(grads)
    near(G.clip_grad_norm(grads, 0.5, out=out), want)
    check_clipped(out, grads, want, 0.5)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_views_of_a_flat_buffer(G, dtype, shift):
    # views that start anywhere, into views that start elsewhere, and in place
    sizes = [100003, 7, 65537, 1, 16384, 130, 33000]
    flat = rand(5, sum(sizes) + 5, dtype=dtype)
    other = torch.full((sum(sizes) + 5,), 9.0, dtype=dtype, device="cuda")
    grads = list(flat[1:1 + sum(sizes)].split(sizes))
    out = list(other[shift:shift + sum(sizes)].split(sizes))
    want = norm_of(grads)
    near(G.grad_norm(grads), want)
    near(G.clip_grad_norm(grads, 3.0, out=out), want)
    check_clipped(out, grads, want, 3.0)
    assert bool((other[:shift] == 9).all()) and bool((other[shift + sum(sizes):] == 9).all())
    keep = flat.clone()
    G.clip_grad_norm(grads, 3.0)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))
    assert float(flat[0]) == float(keep[0]) and torch.equal(flat[-4:], keep[-4:])


@pytest.mark.parametrize("shapes", [[(64, 27), (10, 0), (5, 6), (3, 4), (7, 0), (130, 651)], [(3, 1)], [(5, 0)],
                                    [(64, 32), (8, 0), (16, 4)], [(2000, 650), (2600, 0), (33, 1)],
                                    [(3, 5)] * 500], ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("workers", [1, 3, 64])
def test_packed(G, shapes, workers):
    layout = G.GradientLayout(shapes)
    bufs, sets = [], []
    for w in range(workers):
        buf = torch.full((layout.total,), float("nan"), device="cuda")  # padding must not count
        for i in range(len(shapes)):
            v = layout.layer_view(buf, i)
            v.copy_(rand(100 * w + i, *v.shape, scale=1.0 + w))
        bufs.append(buf)
        sets.append([layout.layer_view(buf, i) for i in range(len(shapes))])
    want = [norm_of(s) for s in sets]
    for got, n in zip(layout.grad_norm(bufs), want):
        near(got, n)
    out = [torch.full((layout.total,), 8.0, device="cuda") for _ in range(workers)]
    for got, n in zip(layout.clip_grad_norm(bufs, 1.5, out=out), want):
        near(got, n)
    for o, s, b, n in zip(out, sets, bufs, want):
        check_clipped([layout.layer_view(o, i) for i in range(len(shapes))], s, n, 1.5)
        pad = torch.isnan(b)
        assert bool((o[pad] == 8).all())
    layout.clip_grad_norm(bufs, 1.5)
    for o, b in zip(out, bufs):
        for i in range(len(shapes)):
            assert torch.equal(layout.layer_view(o, i), layout.layer_view(b, i))


def test_same_on_another_stream_and_every_time(G):
    grads = [rand(1, 1500, 777), rand(2, 5)]
    out = [torch.empty_like(g) for g in grads]
    first = G.clip_grad_norm(grads, 1.0, out=out).clone()
    keep = [o.clone() for o in out]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = [G.clip_grad_norm(grads, 1.0, out=out) for _ in range(4)]
    s.synchronize()
    assert all(torch.equal(first, a) for a in again)
    assert all(torch.equal(a, b) for a, b in zip(out, keep))


def test_context_clips_its_own_buffers(G):
    shapes = [(70, 45), (33, 0), (16, 64)]
    ctx = G.PowerSGD(shapes, 1, 2, seed=5)
    grads = [ctx.pack([rand(7 * w + i, *(s if s[1] else (s[0],))) for i, s in enumerate(shapes)]) for w in range(2)]
    keep = [g.clone() for g in grads]
    want = [norm_of([g]) for g in grads]
    for got, n in zip(ctx.grad_norm(grads), want):
        near(got, n)
    for got, n in zip(ctx.clip_grad_norm(grads, 2.0), want):
        near(got, n)
    for g, k, n in zip(grads, keep, want):
        check_clipped([g], [k], n, 2.0)
    ctx.step(grads, ctx.empty_buffer())
    ctx.sync()
    with pytest.raises(ValueError):
        ctx.clip_grad_norm(grads[:1], 1.0)
    ctx.close()


def test_refusals(G):
    g = rand(1, 8, 8)
    with pytest.raises(ValueError):
        G.grad_norm([])
    with pytest.raises(TypeError):
        G.grad_norm([g.double()])
    with pytest.raises(TypeError):
        G.grad_norm([g, g.half()])
    with pytest.raises(ValueError):
        G.grad_norm([g.cpu()])
    with pytest.raises(ValueError):
        G.grad_norm([rand(1, 4, 4, 4)[:, ::2, ::2]])
    with pytest.raises(ValueError):
        G.grad_norm([g[:1].expand(8, 8)])
    with pytest.raises(G.PsgdError):
        G.clip_grad_norm([g], -1.0)
    with pytest.raises(G.PsgdError):
        G.clip_grad_norm([g], float("nan"))
    with pytest.raises(ValueError):
        G.clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(ValueError):
        G.clip_grad_norm([g], 1.0, out=[rand(1, 8, 9)])
    with pytest.raises(ValueError):
        G.clip_grad_norm([g], 1.0, out=[rand(1, 8, 8).t()])
    with pytest.raises(ValueError):  # rows of 7 values 10 apart, and runs of 42 values 49 apart
        G.clip_grad_norm([rand(1, 4, 6, 10)[:, :, :7]], 1.0, out=[rand(1, 4, 7, 7)[:, :6]])
    with pytest.raises(TypeError):
        G.clip_grad_norm([g], 1.0, out=[g.half()])
    layout = G.GradientLayout([(4, 5)])
    with pytest.raises(ValueError):
        layout.grad_norm([rand(1, 10)])
    with pytest.raises(TypeError):
        layout.grad_norm([rand(1, 40).half()])
    with pytest.raises(G.PsgdError):
        layout.grad_norm([rand(1, 41)[1:]])
