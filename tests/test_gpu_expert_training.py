"""The example that runs the operators together, and the operators in a captured graph and past 32-bit offsets."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def test_the_example_learns(G):
    spec = importlib.util.spec_from_file_location("expert_training", os.path.join(ROOT, "examples", "expert_training.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(steps=30, verbose=False)
    assert all(x == x for x in losses)
    assert losses[-1] < 0.5 * losses[0], losses


def test_operators_in_a_captured_graph(G):
    layout = G.GradientLayout([(72, 131)] * 3 + [(5, 0)])
    offsets = torch.tensor([0, 40, 40, 100], dtype=torch.int32, device="cuda")
    x, w = torch.zeros(100, 131, device="cuda").bfloat16(), torch.randn(3, 72, 131, device="cuda").bfloat16()
    buf, out = torch.zeros(layout.total, device="cuda"), torch.zeros(layout.total, device="cuda")

    def work():
        y = G.experts_forward(x, w, offsets)  # rows of 131 values: copied first
        dx = G.experts_grad_input(y, w, offsets)
        G.experts_grad_weight(y, x, offsets, out=layout.experts_view(buf, 0, 3))
        return y, dx, layout.clip_grad_norm([buf], 1.0, out=[out])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for seed in (1, 2):
        x.copy_(torch.randn(100, 131, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        offsets.copy_(torch.tensor([0, 30 * seed, 70, 90], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured] + [out.clone()]
        want = list(work()) + [out]
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    G.experts_sync()


def test_a_graph_keeps_its_workspace(G):
    # eager calls on the capture's stream that need more room do not take the graph's away
    s = torch.cuda.Stream()
    offsets = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    x, w = torch.randn(50, 131, device="cuda").bfloat16(), torch.randn(1, 64, 131, device="cuda").bfloat16()
    grads = [torch.randn(50000, device="cuda")]
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        want = G.experts_forward(x, w, offsets)
        G.grad_norm(grads)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y, norm = G.experts_forward(x, w, offsets), G.grad_norm(grads)
    with torch.cuda.stream(s):
        big = torch.randn(20000, 131, device="cuda").bfloat16()
        G.experts_forward(big, w, torch.tensor([0, 20000], dtype=torch.int32, device="cuda"))
        marks = [torch.full((1 << 18,), 7.0, device="cuda") for _ in range(40)]
    s.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert abs(float(norm) - float(grads[0].double().norm())) <= 1e-6 * float(norm)
    assert all(bool((m == 7).all()) for m in marks)


def near(got, a, b):
    """got against a @ b in float64, within the float32 sum's and one rounding's error."""
    a, b = a.double(), b.double()
    out, mag = a @ b, a.abs() @ b.abs()
    u = 2.0 ** -24 if got.dtype == torch.float32 else 2.0 ** -8
    tol = u * out.abs() + (1 + u) * (a.shape[1] + 8) * 2.0 ** -23 * mag
    assert bool(((got.double() - out).abs() <= tol).all())


def test_products_past_32_bit_offsets(G):
    # 2.2e9 values of x, dy and y each, and of the weight gradient
    T, k, n = (1 << 21) + 37, 1032, 1048
    x = torch.empty(T, k, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    w = torch.randn(2, n, k, device="cuda").bfloat16()
    offsets = torch.tensor([0, T - 100, T], dtype=torch.int32, device="cuda")
    y = G.experts_forward(x, w, offsets)
    near(y[-150:-100], x[-150:-100], w[0].t())
    near(y[-100:], x[-100:], w[1].t())
    dx = G.experts_grad_input(y, w, offsets)
    near(dx[-100:], y[-100:], w[1])
    dw = G.experts_grad_weight(y, x, offsets)
    near(dw[1], y[-100:].t(), x[-100:])
    del x, y, dx, dw
    E = 2048
    dy, x = torch.randn(64, n, device="cuda").bfloat16(), torch.randn(64, k, device="cuda").bfloat16()
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[E] = 64
    offsets[E - 1] = 24
    dw = G.experts_grad_weight(dy, x, offsets)
    near(dw[E - 1], dy[24:].t(), x[24:])
    near(dw[E - 2], dy[:24].t(), x[:24])
    assert bool((dw[E - 3] == 0).all()) and bool((dw[0] == 0).all())


@pytest.mark.parametrize("padded", [False, True])
def test_norm_past_32_bit_offsets(G, padded):
    n = (1 << 32) + 12345
    if padded:
        t = torch.zeros(n // 1030, 1030, dtype=torch.float16, device="cuda")[:, :1027]
    else:
        t = torch.zeros(n, dtype=torch.float16, device="cuda")
    flat = t if not padded else t[-1]
    flat[-3:] = torch.tensor([3.0, 0.0, 4.0])
    (t[0] if padded else t)[0] = 12.0
    assert float(G.clip_grad_norm([t], 1.0)) == 13.0
    assert [round(float(v), 3) for v in flat[-3:]] == [round(3 / 13, 3), 0.0, round(4 / 13, 3)]
