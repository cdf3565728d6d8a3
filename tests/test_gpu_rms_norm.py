"""The root-mean-square norm of a residual stream and its gradients against their definition in 64 bits.

Tolerances, from the arithmetic, with u half a step of the type and e = 2^-24:
    r    u |r|, and 2 e (|x| / (1 - p) + |residual|) of the product and the sum
    s    its mean is a float32 sum of H squares, off by (H + 8) e of itself, its
         root by half of that; rsqrt and the rest 2^-21: rho = (H + 8) e / 2 + 2^-21
    y    |y| (rho + 4 e + u), from the r that was returned
    dr   rho |s dy w| for its first term; |r| s^3 (H + 8) e mean|dy w r| + 4 rho |r s^3 mean| for
         its second; 4 e of all magnitudes, and u |dr| (dx: of its own value, from the unrounded dr)
    dw   rho and (T + 16) e of sum |dy r s|
and the smallest numbers of the types.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_dropout import kept  # noqa: E402

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
E = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * scale).to(dtype)


def near(name, got, want, tol):
    assert got.shape == want.shape, name
    assert bool(torch.isfinite(got).all()), name
    off = (got.double() - want).abs() - tol - TINY[got.dtype]
    assert not bool((off > 0).any()), (name, int((off > 0).sum()), (off > 0).nonzero()[0].tolist(), float(off.max()))


def mask_of(shape, p, seed=7, step=3, site=2):
    if not p:
        return 1.0
    m, scale = kept(shape[0] * shape[1], p, seed, step, site)
    return m.view(shape).cuda() * scale


def check_forward(G, x, w, res, p=0.0, eps=1e-6):
    H = x.shape[1]
    y, r = G.rms_norm(x, w, residual=res, eps=eps, p=p, state=G.dropout_state(7, 3), site=2)
    d = x.double() * mask_of(x.shape, p)
    want = d if res is None else d + res.double()
    if res is None and not p:
        assert r is x
    else:
        near("r", r, want, ROUND[x.dtype] * want.abs() * (1 + E) + 2 * E * (d.abs() + (0 if res is None else res.double().abs())))
    R = r.double()
    s = (R.square().mean(1, keepdim=True) + eps).rsqrt()
    out = R * s * (1.0 if w is None else w.double())
    near("y", y, out, out.abs() * ((H + 8) * E / 2 + 2.0 ** -21 + 4 * E + ROUND[x.dtype]))


def definition(dy, r, w, dr, p=0.0, eps=1e-6, dw_type=torch.float32):
    """{name: (value, tolerance)}"""
    T, H = r.shape
    u = ROUND[r.dtype]
    R, D, W = r.double(), dy.double(), torch.ones(H, device="cuda", dtype=torch.float64) if w is None else w.double()
    s = (R.square().mean(1, keepdim=True) + eps).rsqrt()
    rho = (H + 8) * E / 2 + 2.0 ** -21
    first, dot = s * D * W, (D * W * R).mean(1, keepdim=True)
    second = R * s ** 3 * dot
    out = first - second
    tol = rho * first.abs() + R.abs() * s ** 3 * (H + 8) * E * (D * W * R).abs().mean(1, keepdim=True) + 4 * rho * second.abs()
    size = first.abs() + second.abs()
    if dr is not None:
        out, size = out + dr.double(), size + dr.double().abs()
    tol = tol + 4 * E * size
    m = mask_of(r.shape, p)
    dx = out * m
    dw = (D * R * s).sum(0)
    return {"dr": (out, tol + u * (out.abs() + tol)), "dx": (dx, tol * m + (u + E) * (dx.abs() + tol * m)),
            "dw": (dw, (rho + (T + 16) * E) * (D * R * s).abs().sum(0) + ROUND[dw_type] * dw.abs())}


def check_grad(G, dy, r, w, dr, p=0.0, eps=1e-6, **kw):
    dx, dres, dw = G.rms_norm_grad(dy, r, w, dr=dr, eps=eps, p=p, state=G.dropout_state(7, 3), site=2, **kw)
    want = definition(dy, r, w, dr, p, eps, torch.float32 if dw is None else dw.dtype)
    near("dr", dres, *want["dr"])
    near("dx", dx, *want["dx"])
    assert dw is None if w is None else near("dw", dw, *want["dw"]) is None


WIDTHS = [1, 2, 7, 8, 9, 15, 31, 64, 650, 651, 753, 754, 755, 760, 767, 768, 769, 776, 1000, 1500, 2048, 2305, 8191, 8440, 8448,
          8449, 8456, 12289, 16370, 16371, 16384, 16392, 23999, 24000]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_widths(G, width, dtype):
    x, res, w = rand(1, 21, width, dtype=dtype), rand(2, 21, width, dtype=dtype, scale=2.0), rand(3, width, dtype=dtype)
    dy, dr = rand(4, 21, width, dtype=dtype), rand(5, 21, width, dtype=dtype)
    for p in (0.0, 0.3):
        check_forward(G, x, w, res, p)
        check_grad(G, dy, x, w, dr, p)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 150, 153, 1300, 5003])
@pytest.mark.parametrize("width", [64, 651, 2048])
def test_rows(G, rows, width):
    x, w, dy = rand(1, rows, width, dtype=torch.bfloat16), rand(3, width), rand(4, rows, width, dtype=torch.bfloat16)
    check_forward(G, x, w, None)
    check_grad(G, dy, x, w, None)
    check_grad(G, dy, x, w, x, 0.1)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_without_weight_or_residual(G, dtype, p):
    x, dy = rand(1, 100, 650, dtype=dtype), rand(2, 100, 650, dtype=dtype)
    check_forward(G, x, None, None, p)
    check_forward(G, x, None, dy, p)
    check_grad(G, dy, x, None, None, p)


def test_strides_and_alignment(G):
    wide = rand(1, 50, 700, dtype=torch.bfloat16)
    w = rand(2, 640, dtype=torch.bfloat16)
    for x in (wide[:, :640], wide[:, 8:648], wide[:, 3:643], wide.reshape(-1)[5:5 + 50 * 640].view(50, 640),
              wide.t()[:640].t(), wide[:1, :640].expand(50, 640)):
        check_forward(G, x, w, None)
        check_forward(G, x, w, wide[:, 16:656], 0.2)
        check_grad(G, x, wide[:, 24:664], w, wide[:, 1:641], 0.2)
    big = rand(3, 20, 1304, dtype=torch.float16)
    x, w = big[:, :651], rand(4, 1302, dtype=torch.float16)[651:]
    check_forward(G, x, w, big[:, 653:1304])
    check_grad(G, big[:, 5:656], x, w, big[:, 653:1304])


def test_zero_rows_and_sizes_at_the_ends(G):
    w = rand(1, 64)
    zero = torch.zeros(3, 64, device="cuda")
    y, _ = G.rms_norm(zero, w, residual=zero)
    assert not y.any()
    check_grad(G, rand(2, 3, 64), zero, w, None)
    for scale in (1e-12, 1e12):
        check_forward(G, rand(3, 5, 64, scale=scale), w, None)
        check_grad(G, rand(2, 5, 64), rand(3, 5, 64, scale=scale), w, None)
    none = torch.empty(0, 64, device="cuda")
    assert G.rms_norm(none, w)[0].shape == (0, 64)
    dx, dr, dw = G.rms_norm_grad(none, none, w)
    assert dx.shape == (0, 64) and not dw.any()


def test_a_rows_nan_stays_in_it(G):
    x, w = rand(1, 9, 65, dtype=torch.bfloat16), rand(2, 65)
    want = G.rms_norm(x, w, residual=x)[0]
    x2 = x.clone()
    x2[4, 64] = float("nan")
    got = G.rms_norm(x2, w, residual=x)[0]
    assert bool(torch.isnan(got[4]).all())
    assert torch.equal(got[:4], want[:4]) and torch.equal(got[5:], want[5:])


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16], ids=str)
def test_weight_gradient_of_the_callers(G, kind):
    dy, r, w = rand(1, 300, 130, dtype=torch.bfloat16), rand(2, 300, 130, dtype=torch.bfloat16), rand(3, 130)
    layout = G.GradientLayout([(3, 5), (130, 0), (7, 0)])
    buf = torch.full((layout.total,), 2.0, device="cuda", dtype=kind)
    view = layout.layer_view(buf, 1)
    check_grad(G, dy, r, w, None, weight_grad=view)
    first = view.double()
    G.rms_norm_grad(dy, r, w, weight_grad=view, accumulate=True)
    assert float((view.double() - 2 * first).abs().max()) <= 4 * ROUND[kind] * float(first.abs().max())
    rest = buf.clone()
    layout.layer_view(rest, 1).fill_(2.0)
    assert bool((rest == 2.0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("residual", [True, False])
def test_autograd(G, dtype, p, residual):
    x, w = rand(1, 90, 130, dtype=dtype).requires_grad_(), rand(2, 130, dtype=dtype).requires_grad_()
    res = rand(3, 90, 130, dtype=dtype).requires_grad_() if residual else None
    dy, dr = rand(4, 90, 130, dtype=dtype), rand(5, 90, 130, dtype=dtype)
    state = G.dropout_state(7, 3)
    y, r = G.rms_norm(x, w, residual=res, p=p, state=state, site=2)
    state[1] += 5
    torch.autograd.backward((y, r), (dy, dr))
    fused = residual or p
    want = definition(dy, r.detach(), w.detach(), dr if fused else None, p, dw_type=dtype)
    if fused:
        near("dx", x.grad, *want["dx"])
    else:  # r is x: torch adds its gradient, rounded once more
        v, tol = want["dx"]
        near("dx", x.grad, v + dr.double(), tol + ROUND[dtype] * (v.abs() + dr.double().abs() + tol))
    if residual:
        near("dres", res.grad, *want["dr"])
    near("dw", w.grad, *want["dw"])


def test_autograd_of_one_result(G):
    x, res, w = (rand(i, 40, 72).requires_grad_() for i in (1, 2, 3))
    w = rand(3, 72).requires_grad_()
    y, r = G.rms_norm(x, w, residual=res, p=0.5, state=G.dropout_state(7, 3), site=2)
    gx, gres = torch.autograd.grad(r, (x, res), rand(4, 40, 72), retain_graph=True)
    near("dres", gres, rand(4, 40, 72).double(), 0.0)
    near("dx", gx, rand(4, 40, 72).double() * mask_of((40, 72), 0.5), 2.0 ** -23 * rand(4, 40, 72).double().abs())
    y.sum().backward()
    want = definition(torch.ones_like(y), r.detach(), w.detach(), None, 0.5)
    near("dx", x.grad, *want["dx"]), near("dw", w.grad, *want["dw"])


def test_gradient_against_differences(G):
    # float32 losses along one coordinate of every row: the slope's own error is h^2 and 2^-24 / h of the terms
    x, w, dy = rand(1, 30, 16), rand(2, 16), rand(3, 30, 16)
    h = torch.zeros_like(x)
    h[:, 3] = 2.0 ** -8
    f = lambda v: (G.rms_norm(v, w)[0].double() * dy.double()).sum(1)
    slope = (f(x + h) - f(x - h)) / 2.0 ** -7
    dx = G.rms_norm_grad(dy, x, w)[0].double()[:, 3]
    s = float((x.double().square().mean(1)).rsqrt().max())
    terms = float((dy * w).double().abs().sum(1).max())
    assert float((slope - dx).abs().max()) <= 2.0 ** -16 * 15 * s ** 3 * terms + 2.0 ** -21 * 2.0 ** 7 * terms * 3


def test_repeated_captured_and_on_two_streams(G):
    x, res, w = rand(1, 500, 648, dtype=torch.bfloat16), rand(2, 500, 648, dtype=torch.bfloat16), rand(3, 648)
    state = G.dropout_state(7, 3)

    def both(x, res):
        y, r = G.rms_norm(x, w, residual=res, p=0.1, state=state)
        return (y, r) + G.rms_norm_grad(y, r, w, dr=res, p=0.1, state=state)
    want = both(x, res)
    assert all(torch.equal(a, b) for a, b in zip(want, both(x, res)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(both(x, res))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(x, res)
        state[1] += 1
    state[1] = 10
    x.copy_(rand(8, 500, 648, dtype=torch.bfloat16))
    for step in (10, 11):
        graph.replay()
        state[1] = step
        assert all(torch.equal(a, b) for a, b in zip(out, both(x, res)))
        state[1] = step + 1


def test_rows_behind_32_bits(G):
    T, H = (1 << 32) // 8192 + 3, 8192
    x = torch.empty(T, H, device="cuda", dtype=torch.float16)
    x.fill_(1.0)
    x[-5:] = rand(1, 5, H, dtype=torch.float16)
    w = rand(2, H)
    y, _ = G.rms_norm(x, w)
    R = x[-5:].double()
    want = R * (R.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.double()
    near("y", y[-5:], want, want.abs() * ((H + 8) * E / 2 + 2.0 ** -20 + 2.0 ** -11))


def test_refusals(G):
    x, w = rand(1, 10, 64), rand(2, 64)
    f, g = G.rms_norm, G.rms_norm_grad
    state = G.dropout_state(1)
    for error, call in ((TypeError, lambda: f(x.double(), w)), (TypeError, lambda: f(x, w.half())), (ValueError, lambda: f(x, w[:63])),
                        (ValueError, lambda: f(x.cpu(), w)), (ValueError, lambda: f(x[0], w)), (ValueError, lambda: f(x, w, p=0.5)),
                        (ValueError, lambda: f(x, w, residual=x[:9])), (TypeError, lambda: f(x, w, residual=x.half())),
                        (ValueError, lambda: f(x, w, p=-0.1, state=state)), (G.PsgdError, lambda: f(x, w, eps=0.0)),
                        (G.PsgdError, lambda: f(x, w, eps=float("nan"))), (ValueError, lambda: f(rand(1, 1, 24001))),
                        (ValueError, lambda: f(x[:, :0])), (G.PsgdError, lambda: f(x, w, p=0.5, state=state, site=70000)),
                        (ValueError, lambda: g(x[:9], x, w)), (TypeError, lambda: g(x.half(), x, w)),
                        (ValueError, lambda: g(x, x, w, dr=x[:, :63])), (ValueError, lambda: g(x, x, None, weight_grad=w)),
                        (ValueError, lambda: g(x, x, w, accumulate=True)), (TypeError, lambda: g(x, x, w, weight_grad=w.half()))):
        with pytest.raises(error):
            call()
