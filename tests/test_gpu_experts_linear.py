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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_a_weight_used_twice_and_micro_batches(G, dtype):
    w, buf = whole(2, 4, N, K), torch.full((4, N, K), 7.0, dtype=dtype, device="cuda")
    xs, gs = [whole(10 + i, T, K) for i in range(3)], [whole(20 + i, T, N) for i in range(3)]
    parts = [weight_gradient(g, x) for g, x in zip(gs, xs)]
    torch.autograd.backward([G.experts_linear(x, w, offsets(), weight_grad=buf) for x in xs], gs)
    assert torch.equal(buf.float(), sum(parts).to(dtype).float())
    buf.zero_()
    for x, g in zip(xs[:2], gs):
        G.experts_linear(x, w, offsets(), weight_grad=buf, accumulate=True).backward(g)
    assert torch.equal(buf.float(), (parts[0] + parts[1]).to(dtype).float())


def test_uses_on_two_streams(G):
    # each use's backward pass runs on its forward's stream; the buffer is whole on the caller's
    w, buf = whole(2, 4, N, K), torch.full((4, N, K), 7.0, device="cuda")
    xs, gs = [whole(10 + i, T, K) for i in range(2)], [whole(20 + i, T, N) for i in range(2)]
    want = sum(weight_gradient(g, x) for g, x in zip(gs, xs))
    streams, ys = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s, x in zip(streams, xs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ys.append(G.experts_linear(x, w, offsets(), weight_grad=buf))
    torch.cuda.synchronize()
    for s in streams:  # both streams are busy when the backward pass comes
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
    torch.autograd.backward(ys, gs)
    got = buf.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_products_are_differentiable(G):
    off, ends = offsets(), offsets().tolist()
    x, w, g = whole(1, T, K).requires_grad_(), whole(2, 4, N, K).requires_grad_(), whole(3, T, N)
    y = G.experts_forward(x, w, off)
    with torch.no_grad():
        assert not G.experts_forward(x, w, off).requires_grad
        assert torch.equal(y, G.experts_forward(x, w, off, out=torch.empty_like(y)))
        dx = G.experts_grad_input(g, w, off)
    y.backward(g)
    assert torch.equal(x.grad, dx)
    assert torch.equal(w.grad.float(), weight_gradient(g, x.detach()))
    # the input gradient is a product too: linear in dy and in w
    dy, w2, h = whole(4, T, N).requires_grad_(), whole(5, 4, N, K).requires_grad_(), whole(6, T, K)
    G.experts_grad_input(dy, w2, off).backward(h)
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        assert torch.equal(dy.grad[a:b].float(), h[a:b].float() @ w2[e].detach().float().T)
        assert torch.equal(w2.grad[e].float(), dy[a:b].detach().float().T @ h[a:b].float())
    assert not G.experts_grad_weight(dy, x, off).requires_grad


def test_out_refuses_operands_that_require_a_gradient(G):
    x, w, off = whole(1, T, K), whole(2, 4, N, K).requires_grad_(), offsets()
    for f, rows, cols in ((G.experts_forward, x, N), (G.experts_grad_input, whole(3, T, N), K)):
        out = torch.empty(T, cols, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(RuntimeError):
            f(rows, w, off, out=out)
        f(rows, w.detach(), off, out=out)
