"""The gradient norm and clipping of a context whose stream is not the caller's."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
SHAPES = [(70, 45), (33, 0), (16, 64)]


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def gradients(ctx, scale):
    return [torch.full((ctx.total,), float(w + 1) * scale, device="cuda") for w in range(ctx.workers)]


@pytest.mark.parametrize("clip", [False, True])
def test_norms_are_there_for_the_caller(G, clip):
    side = torch.cuda.Stream()
    ctx = G.PowerSGD(SHAPES, 1, 2, seed=5, stream=side)
    values = sum(n * max(m, 1) for n, m in SHAPES)
    grads = gradients(ctx, 0.5)
    torch.cuda.synchronize()
    for _ in range(3):
        kept = [g.clone() for g in grads]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):  # the context's stream is busy for some ten milliseconds
            torch.cuda._sleep(50_000_000)
        norms = ctx.clip_grad_norm(kept, 1e9) if clip else ctx.grad_norm(kept)
        got = norms.tolist()  # on the caller's stream
        for w, v in enumerate(got):
            want = 0.5 * (w + 1) * values ** 0.5
            assert abs(v - want) <= 1e-6 * want, (got, want)
        del norms
        torch.full((2,), -1.0, device="cuda")
    ctx.close()


def test_context_on_the_default_stream_called_from_another(G):
    ctx = G.PowerSGD(SHAPES, 1, 2, seed=5)
    grads = gradients(ctx, 2.0)
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = ctx.grad_norm(grads).tolist()
    values = sum(n * max(m, 1) for n, m in SHAPES)
    for w, v in enumerate(got):
        assert abs(v - 2.0 * (w + 1) * values ** 0.5) <= 1e-5 * v
    ctx.close()


def test_gradients_elsewhere_are_refused(G):
    ctx = G.PowerSGD(SHAPES, 1, 2, seed=5)
    with pytest.raises(ValueError):
        ctx.grad_norm([torch.zeros(ctx.total)] * 2)
    ctx.close()
