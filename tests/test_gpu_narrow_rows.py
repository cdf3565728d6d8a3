"""The norm of rows of fewer values than a vector has: several share one, the tensor's last among them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rms_norm import TYPES, check_forward, check_grad, rand  # noqa: E402


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 6, 7, 9])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_few_rows(G, width, dtype):
    w = rand(9, width)
    for rows in (1, 2, 3, 4, 7, 8, 9, 10, 17, 601):
        x, res, dy, dr = (rand(i, rows, width, dtype=dtype) for i in range(4))
        for p in (0.0, 0.3):
            check_forward(G, x, w, res, p)
            check_grad(G, dy, x, w, dr, p)
        check_forward(G, x, None, None)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_what_lies_behind_does_not_matter(G, dtype):
    # operands in front of NaN: rows 0 .. 2 of 3 values end inside the second vector
    def behind(t):
        buf = torch.full((64,), float("nan"), device="cuda", dtype=dtype)
        buf[:9] = t.flatten()
        return buf[:9].view(3, 3)
    x, res, dy, dr = (rand(i, 3, 3, dtype=dtype) for i in range(4))
    w = rand(9, 3)
    check_forward(G, behind(x), w, behind(res))
    check_grad(G, behind(dy), behind(x), w, behind(dr))
