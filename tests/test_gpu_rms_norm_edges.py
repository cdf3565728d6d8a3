"""The norm at the ends of its range: rows far from 1, a tiny eps, empty batches, results in the place of operands."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rms_norm import TYPES, check_forward, check_grad, rand  # noqa: E402


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


@pytest.mark.parametrize("width", [64, 650, 2048])
@pytest.mark.parametrize("scale", [1e-15, 1e13, 1e15, 1e16])
def test_rows_far_from_one(G, width, scale):
    # r s^3 is outside float32's range where s dy w and its projection are inside
    w, r = rand(1, width), rand(3, 5, width, scale=scale)
    for eps in (1e-6, 1e-30):
        check_forward(G, r, w, None, eps=eps)
        check_grad(G, rand(2, 5, width), r, w, None, eps=eps)
        check_grad(G, rand(2, 5, width), r, w, None, p=0.3, eps=eps)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("eps", [1e-6, 1e-26, 1e-30, 1e-36])
def test_zero_rows_with_a_tiny_eps(G, dtype, eps):
    zero, w = torch.zeros(3, 64, device="cuda", dtype=dtype), rand(1, 64)
    dy = rand(2, 3, 64, dtype=dtype, scale=1e-3 if dtype is not torch.float16 else 1.0)
    if dtype is torch.float16:  # 1 / sqrt(eps) is past float16: gradients of 2^-60 cannot be given, of 0 can
        dy.zero_()
    check_grad(G, dy, zero, w, None, eps=eps)
    y, _ = G.rms_norm(zero, w, eps=eps)
    assert not y.any()


# ------------------------------------------------------------------- empty batches --

@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weighted", [None, "frozen", "trained"])
def test_no_rows(G, p, residual, weighted):
    state = G.dropout_state(1)
    x = torch.empty(0, 64, device="cuda", requires_grad=True)
    res = torch.empty(0, 64, device="cuda", requires_grad=True) if residual else None
    w = None if weighted is None else torch.ones(64, device="cuda", requires_grad=weighted == "trained")
    with torch.no_grad():
        y, r = G.rms_norm(x, w, residual=res, p=p, state=state)
        assert y.shape == r.shape == (0, 64)
    y, r = G.rms_norm(x, w, residual=res, p=p, state=state)
    (y.sum() + r.sum()).backward()
    assert x.grad.shape == (0, 64) and (res is None or res.grad.shape == (0, 64))
    if weighted == "trained":
        assert not w.grad.any()
    dx, dr, dw = G.rms_norm_grad(y.detach(), r.detach(), None, p=p, state=state)
    assert dx.shape == dr.shape == (0, 64) and dw is None


# -------------------------------------------- results in the place of operands --
#
# By the library's own entries, which allow it: the functions allocate.

def _at(t):
    return None if t is None else t.data_ptr()


def _dtype(G, t):
    return {torch.float32: G.PSGD_F32, torch.bfloat16: G.PSGD_BF16, torch.float16: G.PSGD_F16}[t.dtype]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,width", [(37, 64), (601, 7), (2500, 651), (700, 2048), (300, 8449), (300, 16384)])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_results_in_the_place_of_operands(G, dtype, rows, width, p):
    lib, stream = G.lib(), torch.cuda.current_stream().cuda_stream
    x, res, dy, dr = (rand(i, rows, width, dtype=dtype) for i in range(4))
    w, state = rand(9, width), G.dropout_state(7, 3)
    y, r = G.rms_norm(x, w, residual=res, p=p, state=state, site=2)
    for over_x in ("y", "r"):
        a, b = x.clone(), res.clone()
        py, pr = (a, b) if over_x == "y" else (b, a)
        assert lib.psgd_rms_norm(rows, width, _dtype(G, x), _at(a), width, _at(b), width, _at(w), G.PSGD_F32, 1e-6, p, _at(state),
                                 2, None, _at(py), width, _at(pr), width, stream) == 0
        assert torch.equal(py, y) and torch.equal(pr, r)
    dx, dres, dw = G.rms_norm_grad(dy, r, w, dr=dr, p=p, state=state, site=2)
    for over in ("dr", "dy"):
        a, b, own = dy.clone(), dr.clone(), torch.empty_like(dw)
        out, ox = b if over == "dr" else a, torch.empty_like(dx) if p else None
        ws = torch.empty(min(rows, 2432) * width * 4, dtype=torch.uint8, device="cuda")
        assert lib.psgd_rms_norm_grad(rows, width, _dtype(G, x), _at(a), width, _at(r), width, _at(b), width, _at(w), G.PSGD_F32,
                                      1e-6, p, _at(state), 2, _at(ox), width, _at(out), width, _at(own), G.PSGD_F32, 0, _at(ws),
                                      ws.numel(), stream) == 0
        assert torch.equal(out, dres) and torch.equal(own, dw) and (ox is None or torch.equal(ox, dx))
