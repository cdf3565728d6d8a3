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


# ------------------------------------------------------------ many rows of one sign --
#
# Words without weights have the same logits, whose exponentials and probabilities
# are known to the bit: 16-bit roundings are taken into the expected value, and what
# is left is how the products over the rows are summed.  That loses, of the sum,
#   n / 2 x 17 x 2^-23  a run's n instructions in the tensor core, 64 of float16 and 128 of
#                       bfloat16: each adds 16 products to the sum and cuts these 17 terms at
#                       a unit of the last place, of a sum that is half the run's on average
#   65 x 2^-25          64 runs, each addition rounded to nearest, of sums half the last on average
#   8 x 2^-24           the chunks, the scale and the end
# 6.7e-5 and 1.3e-4.  (Without runs 13000 instructions and more, which lost 1.3e-3 to 1.7e-3.)

@pytest.mark.parametrize("dtype,rows", [(torch.float16, 200001), (torch.bfloat16, 200001), (torch.bfloat16, 300001)], ids=str)
def test_many_rows_of_one_sign(G, dtype, rows):
    V, H = 200, 64
    g = torch.Generator("cuda").manual_seed(53)
    x = (0.5 + 0.5 * torch.rand(rows, H, generator=g, device="cuda")).to(dtype)
    w, b = torch.zeros(V, H, device="cuda", dtype=dtype), torch.zeros(V, device="cuda")
    target = torch.zeros(rows, device="cuda", dtype=torch.int64)
    dw, db = torch.empty(V, H, device="cuda"), torch.empty(V, device="cuda")
    G.linear_cross_entropy_grad(x, w, target, bias=b, reduction="sum", weight_grad=dw, bias_grad=db)
    tol = (32 if dtype is torch.float16 else 64) * 17 * 2.0 ** -23 + 65 * 2.0 ** -25 + 8 * 2.0 ** -24
    one = torch.ones(rows, 1, device="cuda", dtype=dtype)
    if float(rows) * V * H > 3e9:  # exponentials of 1 and -199, the factor 1 / 200 with the row
        factor = torch.tensor(1.0 / 200, device="cuda")
        d = torch.tensor([-199.0, 1.0], device="cuda", dtype=torch.float64)
        xs, one = (x.float() * factor).to(dtype), (one.float() * factor).to(dtype)
    else:
        up = 16384.0 if dtype is torch.float16 else 1.0
        d = (torch.tensor([1 / 200 - 1, 1 / 200], device="cuda", dtype=torch.float64) * up).to(dtype).double() / up
        xs = x
    for got, col in ((dw, xs.double().sum(0)), (db[:, None], one.double().sum(0))):
        want = torch.cat([d[:1, None] * col, (d[1:, None] * col).expand(V - 1, -1)])
        assert float(((got.double() - want).abs() / want.abs()).max()) <= tol


# ------------------------------------------------------------------- empty batches --

def test_no_rows_and_only_the_rows_gradient(G):
    w = torch.randn(300, 64, device="cuda").bfloat16()
    x, t = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True), torch.empty(0, dtype=torch.int64, device="cuda")
    for reduction in ("mean", "sum", "none"):
        x.grad = None
        G.linear_cross_entropy(x, w, t, reduction=reduction).sum().backward()
        assert x.grad.shape == (0, 64)


# ----------------------------------------------------- sums added to what is there --
#
# A call into float32 buffers gives the sums that are added; the float32 sum of one
# and the start value is rounded once to the buffer's type, and the sums are large
# beside its steps.

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("width", [128, 130, 133])
def test_accumulate_into_16_bits(G, dtype, width):
    x, w, target, b = inputs(300, 500, width, dtype, bias=dtype, seed=54)
    g = torch.Generator("cuda").manual_seed(54)
    start, first = (torch.randn(*s, generator=g, device="cuda").to(dtype) for s in ((500, width), (500,)))
    dw, db = torch.zeros(500, width, device="cuda"), torch.zeros(500, device="cuda")
    G.linear_cross_entropy_grad(x, w, target, bias=b, scale=4.0, reduction="sum", weight_grad=dw, bias_grad=db)
    assert float(dw.abs().max()) > 4 and float(db.abs().max()) > 2
    got, bias = start.clone(), first.clone()
    G.linear_cross_entropy_grad(x, w, target, bias=b, scale=4.0, reduction="sum", weight_grad=got, bias_grad=bias,
                                accumulate=True)
    for now, was, add in ((got, start, dw), (bias, first, db)):
        want = was.double() + add.double()
        # half a step of the result; the two calls' float32 sums of at most five pieces differ by 2^-21 of their terms' size
        tol = ROUND[dtype] * want.abs() + 2.0 ** -20 * (was.double().abs() + 16 * add.double().abs().max()) + 2.0 ** -25
        assert bool(((now.double() - want).abs() <= tol).all())
        assert float((now.double() - was.double()).abs().max()) > 2


# ---------------------------------------------------- the bias's gradient alone --

@pytest.mark.parametrize("dtype,size", [(torch.bfloat16, (300, 700, 72)), (torch.float16, (513, 1300, 651)),
                                        (torch.bfloat16, LARGE)], ids=str)
@pytest.mark.parametrize("rows_too", [False, True])
def test_the_biass_gradient_without_the_matrixs(G, dtype, size, rows_too):
    x, w, target, b = inputs(*size, dtype, bias=torch.float32, ignored=0.2, seed=55)
    weight = torch.full((size[0],), 1.0 / int((target != -100).sum()), device="cuda")
    want = definition(x, w, target, b, weight)
    b.requires_grad_(), x.requires_grad_(rows_too)
    G.linear_cross_entropy(x, w, target, bias=b).backward()
    near("db", b.grad, want["db"])
    if rows_too:
        near("dx", x.grad, want["dx"])
