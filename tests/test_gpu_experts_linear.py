"""``experts_linear`` and the operators under torch's autograd, on the GPU.

Operands are small whole numbers, so every product and every sum of them is
exact in float32 and each result is known to the bit.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def whole(seed, *shape, dtype=torch.bfloat16):
    return torch.randint(-2, 3, shape, generator=torch.Generator().manual_seed(seed)).to("cuda", dtype)


SIZES = [40, 0, 77, 3]
N, K, T = 72, 56, sum(SIZES)


def offsets():
    return torch.tensor([0, 40, 40, 117, 120], dtype=torch.int32, device="cuda")


def weight_gradient(dy, x):
    ends = offsets().tolist()
    return torch.stack([dy[a:b].float().T @ x[a:b].float() for a, b in zip(ends, ends[1:])])


def test_buffer_is_written_when_no_operand_needs_a_gradient(G):
    x, w, g = whole(1, T, K), whole(2, 4, N, K), whole(3, T, N)
    layout = G.GradientLayout([(N, K)] * 4)
    packed = torch.full((layout.total,), 7.0, device="cuda")
    buf = layout.experts_view(packed, 0, 4)
    G.experts_linear(x, w, offsets(), weight_grad=buf).backward(g)
    assert torch.equal(buf, weight_gradient(g, x))
