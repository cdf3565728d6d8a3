"""How far the gradients of the cross entropy are off in all: what the roundings to 16 bits make, and no more.

A rounding to nearest of a value v is off by half a step at most, u |v| with u = 2^-8
(bfloat16) or 2^-11 (float16), evenly spread: its square is u^2 v^2 / 3 at most in the
mean.  The roundings of different values are independent, so the squares add: a term
d x of dw that is rounded k times leaves k u^2 / 3 (d x)^2, and a 16-bit result u^2 / 3
of its own square.  k is 1 where d alone is rounded, and 2 where (bfloat16, over 3e9
multiplications) the exponential and the row with the target's probability are.
What sums and exponentials lose (1e-5) is far below that.  There are over 2e5 roundings,
the norm's own spread is under 5 %: 10 % are allowed.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_cross_entropy import inputs  # noqa: E402

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


@pytest.mark.parametrize("dtype,size", [(torch.bfloat16, (600, 2000, 256)), (torch.float16, (600, 2000, 256)),
                                        (torch.float16, (2240, 8001, 650)), (torch.bfloat16, (2240, 8001, 650))], ids=str)
@pytest.mark.parametrize("float32", [False, True])
def test_gradients_in_norm(G, dtype, size, float32):
    T, V, H = size
    x, w, target, b = inputs(*size, dtype, bias=torch.float32, seed=60)
    dw, db = torch.empty(V, H, device="cuda", dtype=torch.float32 if float32 else dtype), torch.empty(V, device="cuda")
    _, dx, _, _ = G.linear_cross_entropy_grad(x, w, target, bias=b, reduction="sum", weight_grad=dw, bias_grad=db)
    X, W = x.double(), w.double()
    logp = torch.log_softmax(X @ W.T + b.double(), 1)
    d, rows = logp.exp(), torch.arange(T, device="cuda")
    d[rows, target] = torch.expm1(logp[rows, target])
    u, k = U[dtype] ** 2 / 3, 2 if dtype is torch.bfloat16 and float(T) * V * H > 3e9 else 1
    square = d.square()
    for name, got, want, terms, half in (("dx", dx, d @ W, square @ W.square(), True),
                                         ("dw", dw, d.T @ X, k * square.T @ X.square(), not float32),
                                         ("db", db, d.sum(0), k * square.sum(0), False)):
        most = (u * float(terms.sum()) + (u * float(want.square().sum()) if half else 0.0)) ** 0.5
        off = float((got.double() - want).norm())
        print(name, off / float(want.norm()), off / most)
        assert off <= 1.1 * most, (name, off / most)
