"""How far the products' sums are off over long contractions.

The bounds are those of the arithmetic, relative to the sum of the terms'
magnitudes (for operands of one sign: to the result).  The tensor cores add 16
terms an instruction and truncate.  bfloat16 products have 16 bits, which a sum
of up to 256 of them still holds, so an instruction loses less than one unit
(2^-23) of a sum that grows evenly, and s of them at most (s + 1) / 2 x 2^-23.
float16 products have 22 bits and are cut one by one: 17 units.  m additions
rounded to nearest lose at most (m + 1) / 2 x 2^-24.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def truncated(instructions, dtype=torch.bfloat16):
    return (instructions + 1) / 2 * 2.0 ** -23 * (17 if dtype is torch.float16 else 1)


def rounded(additions):
    return (additions + 1) / 2 * 2.0 ** -24


def positive(seed, *shape, dtype=torch.bfloat16):
    return torch.rand(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").add_(0.5).to(dtype)


def offsets(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("rows", [512, 4096, 32768])
def test_weight_gradient_of_one_sign(G, rows, dtype):
    # pieces of 512 rows: without them 4096 rows of bfloat16 would lose 5e-6, twice the bound
    n, k = 520, 392
    dy, x = positive(1, rows, n, dtype=dtype), positive(2, rows, k, dtype=dtype)
    dw = G.experts_grad_weight(dy, x, offsets(0, rows))[0].double()
    want = dy.double().T @ x.double()
    off = float(((dw - want).abs() / want).max())
    assert off <= truncated(32, dtype) + rounded(rows // 512), off


def test_weight_gradient_of_equal_rows_and_many_of_them(G):
    # equal pieces round the same way each time: 2048 of them in one running sum were off by 3e-5
    rows, side = 1 << 20, 2048
    a, b = positive(3, side), positive(4, side)
    dy, x = a.expand(rows, side).contiguous(), b.expand(rows, side).contiguous()
    dw = G.experts_grad_weight(dy, x, offsets(0, 1, rows))
    want = torch.outer(a.double(), b.double())
    off = float(((dw[1].double() / (rows - 1) - want).abs() / want).max())
    assert off <= truncated(32) + rounded(128) + rounded(32), off
    assert torch.equal(dw[0].double(), want)


def test_weight_gradient_past_32_bit_offsets(G):
    rows, n, k = (1 << 21) + 37, 1048, 1032
    g = torch.Generator("cuda").manual_seed(5)
    dy, x = (torch.empty(rows, c, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for c in (n, k))
    dw = G.experts_grad_weight(dy, x, offsets(0, rows - 100, rows))
    want, size = (torch.zeros(n, k, dtype=torch.float64, device="cuda") for _ in range(2))
    for r in range(0, rows - 100, 1 << 18):
        a, b = (t[r:min(r + (1 << 18), rows - 100)].double() for t in (dy, x))
        want.addmm_(a.T, b)
        size.addmm_(a.abs().T, b.abs())
    off = float(((dw[0].double() - want).abs() / size).max())
    assert off <= truncated(32) + rounded(128) + rounded(33), off


@pytest.mark.parametrize("op", ["forward", "grad_input"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_longest_contraction_of_many_tiles(G, op, dtype):
    # 41 tiles, so that nothing but its length cuts the contraction: of 2^20 values in one piece float16 lost 5e-3
    side, depth, rows = 10304, 1 << 20, 3
    shape = (1, side, depth) if op == "forward" else (1, depth, side)
    g = torch.Generator("cuda").manual_seed(6)
    w = torch.empty(shape, dtype=dtype, device="cuda").uniform_(0.5, 1.5, generator=g).mul_(2.0 ** -10)
    x = torch.empty(rows, depth, dtype=dtype, device="cuda").uniform_(0.5, 1.5, generator=g).mul_(2.0 ** -10)
    off = offsets(0, rows)
    y = (G.experts_forward if op == "forward" else G.experts_grad_input)(x, w, off)
    want = torch.zeros(rows, side, dtype=torch.float64, device="cuda")
    for d in range(0, depth, 1 << 15):
        part = w[0, :, d:d + (1 << 15)].T if op == "forward" else w[0, d:d + (1 << 15)]
        want.addmm_(x[:, d:d + (1 << 15)].double(), part.double())
    off = float(((y.double() - want).abs() / want).max())
    u, parts = (2.0 ** -11, 32) if dtype is torch.float16 else (2.0 ** -8, 4)
    sums = truncated(depth // parts // 16, torch.float16) + rounded(parts)  # long sums cut bfloat16 products too
    if dtype is torch.float16:
        assert sums < 5e-3 - u  # what the bound has to tell apart
    assert off <= u + (1 + u) * sums, off
