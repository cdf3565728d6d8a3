"""What the operators write in place or into ``out`` counts as written for torch's autograd."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def test_backward_over_a_clipped_tensor_stops(G):
    x, t = torch.randn(50, device="cuda", requires_grad=True), torch.randn(50, device="cuda")
    y = x * t  # needs t for x's gradient
    G.clip_grad_norm([t], 0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_versions(G):
    layout = G.GradientLayout([(8, 16)] * 2)
    off = torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda")
    x, w = torch.randn(7, 16, device="cuda").bfloat16(), torch.randn(2, 8, 16, device="cuda").bfloat16()
    y, dx = torch.empty(7, 8, device="cuda").bfloat16(), torch.empty(7, 16, device="cuda").bfloat16()
    buf, other = torch.zeros(layout.total, device="cuda"), torch.zeros(layout.total, device="cuda")
    for write, touched in ((lambda: G.experts_forward(x, w, off, out=y), [y]),
                           (lambda: G.experts_grad_input(y, w, off, out=dx), [dx]),
                           (lambda: G.experts_grad_weight(y, x, off, out=layout.experts_view(buf, 0, 2)), [buf]),
                           (lambda: layout.clip_grad_norm([buf, other], 1.0), [buf, other]),
                           (lambda: layout.clip_grad_norm([buf], 1.0, out=[other]), [other]),
                           (lambda: G.clip_grad_norm([buf], 1.0, out=[other]), [other])):
        every = [x, w, y, dx, buf, other]
        before = [t._version for t in every]
        write()
        for t, v in zip(every, before):
            assert (t._version > v) == any(t is u for u in touched)
    before = buf._version
    G.grad_norm([buf]), layout.grad_norm([buf])
    assert buf._version == before


def test_inference_tensors_are_written_too(G):
    with torch.inference_mode():
        t = torch.ones(64, device="cuda")
    u = torch.ones(64, device="cuda")
    v = u._version
    G.clip_grad_norm([t, u], 1.0)
    assert u._version > v
    assert abs(float(t[0]) - 128 ** -0.5) < 1e-6 and torch.equal(t, u)
