"""The gradient norm and clipping at the limits of their tables: 16 runs of
memory in the short one, 432 in one launch.

The gradients are whole numbers whose squares add up exactly, so the norm is
known to its one rounding; clipping scales by a power of two.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def whole(seed, n, dtype):
    return torch.randint(-4, 5, (n,), generator=torch.Generator().manual_seed(seed)).to("cuda", dtype)


def check(G, grads):
    squares = sum(int(g.double().pow(2).sum()) for g in grads)
    want = math.sqrt(squares)
    near = lambda v: abs(float(v) - want) <= 2.0 ** -24 * want
    assert near(G.grad_norm(grads))
    keep = [g.clone() for g in grads]
    out = [torch.full_like(g, 9.0) for g in grads]
    assert near(G.clip_grad_norm(grads, 1e9, out=out))  # a factor of 1
    assert all(torch.equal(o, k) and torch.equal(g, k) for o, g, k in zip(out, grads, keep))
    # the factor that the kernel takes is max_norm / (norm + 1e-6), rounded to float32
    quarter = (want + 1e-6) * 0.25
    assert near(G.clip_grad_norm(grads, quarter))
    for g, k in zip(grads, keep):
        off = (g.double() - k.double() * 0.25).abs()
        assert bool((off <= 2.0 ** (-7.9 if g.dtype is torch.bfloat16 else -10.9 if g.dtype is torch.float16 else -22)
                     * k.double().abs()).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("count", [15, 16, 17, 431, 432, 433, 863, 864, 865])
def test_runs_at_the_tables_limits(G, dtype, count):
    check(G, [whole(i, 1 + 7 * i % 53, dtype) for i in range(count)])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("before", [14, 15, 16, 430, 431, 432, 862, 863])
def test_a_tensor_whose_two_runs_part(G, dtype, before):
    # a long run that starts between 16-byte boundaries makes two; its second may start the next table
    flat, n = whole(1, 30001, dtype), 9000
    odd = [flat[1 + i * (n + 1):1 + i * (n + 1) + n] for i in range(3)]
    check(G, [whole(i, 8, dtype) for i in range(before)] + odd)


def test_memory_to_be_scaled_twice_is_refused(G):
    g, h = whole(1, 100, torch.float32), whole(2, 100, torch.float32)
    keep = g.clone()
    for grads, out in (([g, h, g], None), ([g, h], [keep, keep]), ([g, g[:7]], None)):
        with pytest.raises(ValueError):
            G.clip_grad_norm(grads, 1.0, out=out)
    layout = G.GradientLayout([(10, 10)])
    with pytest.raises(ValueError):
        layout.clip_grad_norm([g, g], 1.0)
    with pytest.raises(ValueError):
        layout.clip_grad_norm([g, h], 1.0, out=[keep, keep])
    # read alone, a tensor may count twice; empty ones have no memory
    assert abs(float(G.grad_norm([g, g])) - 2 ** 0.5 * float(keep.double().norm())) < 1e-5
    empty = [torch.empty(0, device="cuda"), g[:0], g, torch.empty(0, device="cuda")]
    assert abs(float(G.clip_grad_norm(empty, 1e9)) - float(keep.double().norm())) < 1e-5
