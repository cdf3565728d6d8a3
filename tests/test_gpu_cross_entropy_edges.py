"""The cross entropy at the ends of its range: impossible targets, infinite logits, many rows of one sign, empty batches,
sums added to 16-bit gradients, the bias's gradient alone."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_cross_entropy import ROUND, definition, inputs, near  # noqa: E402

LARGE = (2048, 8001, 400)  # over 3e9 multiplications: bfloat16 takes statistics and exponentials from one product


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


# ------------------------------------------------- targets that are masked out --
#
# A word whose bias is far below the others takes no probability: a row with that
# target has p - [v = y] of the other words' softmax and -1, however far below.  The
# definition is taken at a bias of -100, where the word's probability is under e^-60
# and the tolerance, which grows with the bias, still that of ordinary rows.

@pytest.mark.parametrize("value", [-1e3, -1e4, -1e6, -1e9, torch.finfo(torch.float32).min, -float("inf")])
@pytest.mark.parametrize("dtype,size", [(torch.bfloat16, (300, 700, 72)), (torch.float16, (300, 700, 72)),
                                        (torch.bfloat16, LARGE)], ids=str)
def test_gradients_of_rows_whose_target_is_masked(G, dtype, size, value):
    x, w, target, b = inputs(*size, dtype, bias=torch.float32, ignored=0.1, seed=50)
    gone = [3, 250, size[1] - 1]  # masked words
    target[torch.isin(target, torch.tensor(gone, device="cuda"))] = 7
    rows = [0, 17, 255, 256, size[0] - 1]
    for i, t in enumerate(rows):
        target[t] = gone[i % 3]
    b[gone] = -100.0
    want = definition(x, w, target, b, torch.full((size[0],), 1.0 / int((target != -100).sum()), device="cuda"))
    b[gone] = value
    loss, dx, dw, db = G.linear_cross_entropy_grad(x, w, target, bias=b)
    near("dx", dx, want["dx"]), near("dw", dw, want["dw"]), near("db", db, want["db"])
    losses = G.linear_cross_entropy(x, w, target, bias=b, reduction="none")
    if value >= -1e9:
        right = definition(x, w, target, b, torch.ones(size[0], device="cuda"))["losses"]
        near("losses", losses, right)
    else:
        assert bool(torch.isinf(losses[rows]).all()) and math.isinf(float(loss))
        assert int(torch.isinf(losses).sum()) == len(rows) and not bool(torch.isnan(losses).any())


def test_the_only_word_left_is_the_target(G):
    # every other word masked: a loss of 0 and no gradient
    x, w, target, b = inputs(40, 300, 64, bias=torch.float32, seed=51)
    target[:] = 5
    b[:5], b[6:] = -float("inf"), -float("inf")
    loss, dx, dw, db = G.linear_cross_entropy_grad(x, w, target, bias=b, reduction="sum")
    assert float(loss) == 0.0 and not dx.any() and not dw.any() and not db.any()


# ------------------------------------------------------------- infinite logits --

@pytest.mark.parametrize("dtype,size", [(torch.bfloat16, (300, 700, 72)), (torch.float16, (300, 700, 72)),
                                        (torch.bfloat16, LARGE), (torch.bfloat16, (1, 700, 72))], ids=str)
def test_a_target_of_infinite_logit_is_not_a_loss_of_zero(G, dtype, size):
    # the logarithm of the sum and the target's logit are both infinite: their difference is no number
    x, w, target, b = inputs(*size, dtype, bias=torch.float32, seed=52)
    target[0] = 9
    b[9] = float("inf")
    losses = G.linear_cross_entropy(x, w, target, bias=b, reduction="none")
    assert bool(torch.isnan(losses[target == 9]).all()) and not bool(torch.isfinite(losses).any())
    loss, dx, dw, db = G.linear_cross_entropy_grad(x, w, target, bias=b)
    assert math.isnan(float(loss)) and bool(torch.isnan(dx[0]).all()) and bool(torch.isnan(dw).all())
