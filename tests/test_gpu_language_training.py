"""The example that runs the language model's operators together: that it runs, its gradients, and the same in a graph."""
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


@pytest.fixture(scope="module")
def M(G):
    spec = importlib.util.spec_from_file_location("language_training", os.path.join(ROOT, "examples", "language_training.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_example_runs(M):
    losses = M.train(steps=3, verbose=False)
    assert len(losses) == 3 and all(x == x and 0 < x < 20 for x in losses)


def case(G, M, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    layout = G.GradientLayout(M.SHAPES)
    p = M.in_half(M.parts(layout, M.first_parameters(layout, g)))
    p["bias"] = torch.randn(M.WORDS, generator=g, device="cuda") * 0.3
    tokens = torch.randint(0, M.WORDS, (M.TOKENS,), generator=g, device="cuda")
    target = torch.randint(0, M.WORDS, (M.TOKENS,), generator=g, device="cuda")
    target[:50] = -100
    return layout, p, tokens, target


def reference(G, M, p, tokens, target, state):
    """The same model in float64 under torch's autograd, its masks from dropped ones."""
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    order, offsets = M.sort_by_expert(tokens)
    tokens, target, ends = tokens[order], target[order], offsets.tolist()
    ones = torch.ones(M.TOKENS, M.WIDTH, device="cuda")
    branch_mask, head_mask = (G.dropout(ones, M.DROP, state, site=s).double() for s in (M.BRANCH, M.HEAD))

    def norm(r, w):
        return r * (r.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w

    def experts(x, w):
        return torch.cat([x[a:b] @ w[e].T for e, (a, b) in enumerate(zip(ends, ends[1:]))])
    x = q["embedding"][tokens]
    branch = experts(torch.relu(experts(norm(x, q["norm1"]), q["up"])), q["down"])
    z = norm(x + branch * branch_mask, q["norm2"]) * head_mask
    logp = torch.log_softmax(z @ q["head"].T + q["bias"], 1)
    keep = target >= 0
    loss = -logp[keep, target[keep]].mean()
    loss.backward()
    return float(loss.detach()), {k: v.grad for k, v in q.items()}


def test_gradients_of_the_whole_step(G, M):
    layout, p, tokens, target = case(G, M, 1)
    state = G.dropout_state(3, 5)
    buf = torch.zeros(layout.total, device="cuda")
    loss = M.gradients(p, tokens, target, state, M.parts(layout, buf))
    want, grads = reference(G, M, p, tokens, target, state)
    # every value that passes between two operators is rounded to bfloat16, 2^-8 of itself, the probabilities among
    # them; ten such roundings lie between a parameter and its gradient.  A relu may fall on either side of 0 where its
    # argument is within such a rounding of it, which moves whole entries: hence the norms
    assert abs(float(loss.detach()) - want) <= 10 * 2.0 ** -8 * want
    for name, got in M.parts(layout, buf).items():
        off = float((got.double() - grads[name]).norm() / grads[name].norm())
        assert off <= 10 * 2.0 ** -8, (name, off)


def test_the_whole_step_in_a_graph(G, M):
    layout, p, tokens, target = case(G, M, 2)
    state = G.dropout_state(4, 0)
    order, offsets = M.sort_by_expert(tokens)
    tokens, target = tokens[order].contiguous(), target[order].contiguous()
    buf = torch.zeros(layout.total, device="cuda")
    out = M.parts(layout, buf)

    def work():
        n1, r1 = G.rms_norm(p["embedding"][tokens], p["norm1"])
        a = G.experts_forward(n1, p["up"], offsets)
        n2, r2 = G.rms_norm(G.experts_forward(torch.relu(a), p["down"], offsets), p["norm2"], residual=r1, p=0.1, state=state)
        z = G.dropout(n2, 0.1, state, site=1)
        loss, dz, _, _ = G.linear_cross_entropy_grad(z, p["head"], target, bias=p["bias"], weight_grad=out["head"],
                                                     bias_grad=out["bias"])
        dx, dr, _ = G.rms_norm_grad(G.dropout(dz, 0.1, state, site=1), r2, p["norm2"], p=0.1, state=state,
                                    weight_grad=out["norm2"])
        norm = layout.clip_grad_norm([buf], 0.1)
        return loss, dx, dr, norm
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for step in (0, 7):
        state[1] = step
        graph.replay()
        got = [t.clone() for t in captured] + [buf.clone()]
        want = list(work()) + [buf]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    G.experts_sync()


def test_under_autograd_with_experts_linear(G, M):
    layout, p, tokens, target = case(G, M, 3)
    state = G.dropout_state(3, 5)
    order, offsets = M.sort_by_expert(tokens)
    q = {k: v.clone().requires_grad_() for k, v in p.items()}
    t, y = tokens[order], target[order]
    n1, r1 = G.rms_norm(q["embedding"][t], q["norm1"])
    a = torch.relu(G.experts_linear(n1, q["up"], offsets))
    n2, _ = G.rms_norm(G.experts_linear(a, q["down"], offsets), q["norm2"], residual=r1, p=M.DROP, state=state, site=M.BRANCH)
    loss = G.linear_cross_entropy(G.dropout(n2, M.DROP, state, site=M.HEAD), q["head"], y, bias=q["bias"])
    state[1] += 1
    loss.backward()
    state[1] -= 1
    want, grads = reference(G, M, p, tokens, target, state)
    assert abs(float(loss.detach()) - want) <= 10 * 2.0 ** -8 * want
    for name, v in q.items():
        off = float((v.grad.double() - grads[name]).norm() / grads[name].norm())
        assert off <= 11 * 2.0 ** -8, (name, off)  # gradients in bfloat16: one rounding more


def test_a_captured_backward_pass(G):
    # with no eager graph of the same leaves alive
    g = torch.Generator("cuda").manual_seed(6)
    x, w, v = (torch.randn(*s, generator=g, device="cuda").bfloat16().requires_grad_() for s in ((200, 136), (136,), (500, 136)))
    target, state = torch.randint(0, 500, (200,), generator=g, device="cuda"), G.dropout_state(1)

    def work():
        y, r = G.rms_norm(x, w, residual=x, p=0.2, state=state)
        loss = G.linear_cross_entropy(G.dropout(y, 0.2, state, site=1) + r, v, target)
        return (loss.detach(),) + torch.autograd.grad(loss, (x, w, v))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for step in (3, 4):
        state[1] = step
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip([t.clone() for t in got], work()))
