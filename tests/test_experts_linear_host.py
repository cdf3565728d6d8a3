"""How ``experts_linear`` is tied to torch's autograd, with the products computed by torch on the CPU in their place."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def ops(monkeypatch):
    from rank_gradient_compression_layer_gb300 import operators as m

    def each(offsets):
        ends = offsets.tolist()
        return enumerate(zip(ends, ends[1:]))

    def forward(x, w, offsets, out=None):
        y = x.new_zeros(x.shape[0], w.shape[1])
        for e, (a, b) in each(offsets):
            y[a:b] = x[a:b] @ w[e].T
        return y

    def grad_input(dy, w, offsets, out=None):
        dx = dy.new_zeros(dy.shape[0], w.shape[2])
        for e, (a, b) in each(offsets):
            dx[a:b] = dy[a:b] @ w[e]
        return dx

    def grad_weight(dy, x, offsets, out=None):
        shape = (offsets.numel() - 1, dy.shape[1], x.shape[1])
        dw = torch.empty(shape) if out is None else out
        for e, (a, b) in each(offsets):
            dw[e] = dy[a:b].float().T @ x[a:b].float()
        return dw

    monkeypatch.setattr(m, "_torch_stream", lambda device: torch.Stream("cpu"), raising=False)
    monkeypatch.setattr(m, "experts_forward", forward)
    monkeypatch.setattr(m, "experts_grad_input", grad_input)
    monkeypatch.setattr(m, "experts_grad_weight", grad_weight)
    return m


# small whole numbers: every product and sum is exact in 16 bits
def whole(seed, *shape):
    return torch.randint(-2, 3, shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


OFFSETS = torch.tensor([0, 2, 2, 5], dtype=torch.int32)


def weight_gradient(g, x):
    return torch.stack([g[a:b].float().T @ x[a:b].float() for a, b in ((0, 2), (2, 2), (2, 5))])


def test_buffer_is_written_when_no_operand_needs_a_gradient(ops):
    # a first layer on data, whose weights are copies of parameters that live elsewhere
    x, w, g = whole(1, 5, 4), whole(2, 3, 6, 4), whole(3, 5, 6)
    buf = torch.full((3, 6, 4), 7.0)
    y = ops.experts_linear(x, w, OFFSETS, weight_grad=buf)
    assert y.requires_grad
    y.backward(g)
    assert torch.equal(buf, weight_gradient(g, x))
    assert x.grad is None and w.grad is None


def test_buffer_stays_without_a_backward_pass(ops):
    buf = torch.full((3, 6, 4), 7.0)
    with torch.no_grad():
        assert not ops.experts_linear(whole(1, 5, 4), whole(2, 3, 6, 4), OFFSETS, weight_grad=buf).requires_grad
    assert not ops.experts_linear(whole(1, 5, 4), whole(2, 3, 6, 4), OFFSETS).requires_grad
    assert bool((buf == 7).all())


def test_unfit_buffers_are_refused_at_the_call(ops):
    x, w = whole(1, 5, 4), whole(2, 3, 6, 4)
    with pytest.raises(ValueError):
        ops.experts_linear(x, w, OFFSETS, weight_grad=torch.empty(3, 4, 6))
    with pytest.raises(TypeError):
        ops.experts_linear(x, w, OFFSETS, weight_grad=torch.empty(3, 6, 4, dtype=torch.float64))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_a_weight_used_twice_gets_both_gradients(ops, dtype):
    x1, x2, w, g1, g2 = whole(1, 5, 4), whole(4, 5, 4), whole(2, 3, 6, 4), whole(3, 5, 6), whole(5, 5, 6)
    want = weight_gradient(g1, x1) + weight_gradient(g2, x2)
    buf = torch.full((3, 6, 4), 7.0, dtype=dtype)
    for _ in range(2):  # the next backward pass starts over
        y1, y2 = (ops.experts_linear(x, w, OFFSETS, weight_grad=buf) for x in (x1, x2))
        torch.autograd.backward([y1, y2], [g1, g2])
        assert torch.equal(buf, want.to(dtype))
    assert not ops._passes


def test_micro_batches_accumulate(ops):
    w, want = whole(2, 3, 6, 4), torch.zeros(3, 6, 4)
    buf = torch.zeros(3, 6, 4)
    for i in range(3):
        x, g = whole(10 + i, 5, 4), whole(20 + i, 5, 6)
        ops.experts_linear(x, w, OFFSETS, weight_grad=buf, accumulate=True).backward(g)
        want += weight_gradient(g, x)
    assert torch.equal(buf, want)


def test_unlike_layouts_at_one_address(ops):
    x, g, flat = whole(1, 5, 4), whole(3, 5, 6), torch.zeros(72)
    wide, other = flat.view(3, 6, 4), flat.view(4, 6, 3).permute(2, 1, 0)
    ys = [ops.experts_linear(x, whole(2, 3, 6, 4), OFFSETS, weight_grad=b) for b in (wide, other)]
    with pytest.raises(ValueError):
        torch.autograd.backward(ys, [g, g])
