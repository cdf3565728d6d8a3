"""Products that give up a wait: what they leave, and who hears of it.

The waits are made to run out by loading nothing, with a limit of 50 ms; the
kernels then return by themselves and the device stays usable.
"""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def whole(seed, *shape):
    return torch.randint(-2, 3, shape, generator=torch.Generator().manual_seed(seed)).to("cuda", torch.bfloat16)


def told(G):
    try:
        G.experts_sync()
    except G.PsgdError as e:
        assert e.code == G.PSGD_ERR_TIMEOUT
        return True
    return False


@pytest.fixture
def product(G):
    off = torch.tensor([0, 300, 300, 341], dtype=torch.int32, device="cuda")
    x, w = whole(1, 341, 200), whole(2, 3, 264, 200)
    want = torch.cat([x[:300].float() @ w[0].float().T, x[300:].float() @ w[2].float().T]).bfloat16()
    torch.cuda.synchronize()
    told(G)
    yield lambda: G.experts_forward(x, w, off), want
    told(G)  # the next test starts from nothing untold on this stream


def in_thread(f):
    got = []

    def run():
        try:
            got.append(f())
        except Exception as e:  # handed to the caller
            got.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    return got[0]


def test_another_threads_stall_is_its_own(G, product):
    forward, want = product
    G.experts_sync()
    assert in_thread(lambda: G.lib().psgd_experts_set_wait(0, 1)) == 0
    assert torch.equal(forward(), want)
    G.experts_sync()


def abandon(G, forward):
    """A product that gives up, and has ended."""
    assert G.lib().psgd_experts_set_wait(50, 1) == 0
    try:
        forward()
        torch.cuda.current_stream().synchronize()
    finally:
        assert G.lib().psgd_experts_set_wait(0, 0) == 0


def test_another_streams_sync_does_not_take_the_report(G, product):
    forward, want = product
    mine, other = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (mine, other):
        with torch.cuda.stream(s):
            forward()
            G.experts_sync()
    with torch.cuda.stream(mine):
        abandon(G, forward)
    with torch.cuda.stream(other):
        told(G)
        told(G)
    with torch.cuda.stream(mine):
        assert told(G)
        assert not told(G)
        assert torch.equal(forward(), want)
        assert not told(G)


def test_another_threads_sync_does_not_take_the_report(G, product):
    forward, want = product
    assert torch.equal(forward(), want)
    assert not told(G)
    assert in_thread(lambda: abandon(G, forward)) is None
    assert in_thread(lambda: told(G)) is True
    assert told(G)
    assert not told(G)


def test_the_next_product_tells_of_an_abandoned_one(G, product):
    forward, want = product
    assert torch.equal(forward(), want)
    abandon(G, forward)
    with pytest.raises(G.PsgdError) as e:
        forward()
    assert e.value.code == G.PSGD_ERR_TIMEOUT
    assert torch.equal(forward(), want)
    assert not told(G)


def test_a_backward_pass_tells_of_an_abandoned_one(G, product):
    off = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    x, w = whole(3, 70, 64).requires_grad_(), whole(4, 1, 72, 64)
    y = G.experts_forward(x, w, off)
    abandon(G, product[0])
    with pytest.raises(G.PsgdError):
        y.sum().backward()
    assert torch.equal(product[0](), product[1])
    told(G)


def test_a_replayed_graph_is_told_of(G, product):
    forward, want = product
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        forward()
        side.synchronize()
    assert G.lib().psgd_experts_set_wait(50, 1) == 0
    with torch.cuda.graph(graph, stream=side):
        forward()
    assert G.lib().psgd_experts_set_wait(0, 0) == 0
    assert not told(G)
    for _ in range(2):
        graph.replay()
        assert told(G)
    assert torch.equal(forward(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_what_was_abandoned_is_nan(G, product, dtype):
    # no value of an earlier use of the memory passes for a result; rows of no expert and empty experts stay zero
    off = torch.tensor([2, 300, 300, 341], dtype=torch.int32, device="cuda")
    x, dy, w = whole(1, 343, 200).to(dtype), whole(2, 343, 264).to(dtype), whole(3, 3, 264, 200).to(dtype)
    y, dx = torch.ones_like(dy), torch.ones_like(x)
    dws = [torch.ones(3, 264, 200, dtype=t, device="cuda") for t in (torch.float32, dtype)]
    odd = torch.ones(3, 264, 201, device="cuda")[:, :, :200]
    for call in (lambda: G.experts_forward(x, w, off, out=y), lambda: G.experts_grad_input(dy, w, off, out=dx),
                 *(lambda b=b: G.experts_grad_weight(dy, x, off, out=b) for b in (*dws, odd))):
        abandon(G, call)
        assert told(G)
    for r in (y, dx):
        assert bool(torch.isnan(r[2:341]).all()) and bool((r[:2] == 0).all()) and bool((r[341:] == 0).all())
    for r in (*dws, odd):
        assert bool(torch.isnan(r[[0, 2]]).all()) and bool((r[1] == 0).all())


def test_what_was_abandoned_in_parts_is_nan(G, product):
    off = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    x, w = whole(1, 6, 8192), whole(2, 1, 128, 8192)  # summed in parts
    y = torch.ones(6, 128, dtype=torch.bfloat16, device="cuda")
    abandon(G, lambda: G.experts_forward(x, w, off, out=y))
    assert told(G) and bool(torch.isnan(y).all())
    off = torch.tensor([0, 6000], dtype=torch.int32, device="cuda")
    dy, x, dw = whole(3, 6000, 64), whole(4, 6000, 72), torch.ones(1, 64, 72, device="cuda")  # and in segments
    abandon(G, lambda: G.experts_grad_weight(dy, x, off, out=dw))
    assert told(G) and bool(torch.isnan(dw).all())


def test_a_long_product_does_not_outlast_its_own_waits(G, product):
    # some 20 ms of tiles before the one expert that ends inside 16 rows, with a limit of 4 ms
    experts, each, side = 16, 16384, 8192
    ends = [e * each for e in range(experts)] + [experts * each + 1]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(7)
    dy, x = (torch.randint(-2, 3, (ends[-1], side), generator=g, device="cuda", dtype=torch.int8).bfloat16()
             for _ in range(2))
    assert G.lib().psgd_experts_set_wait(4, 0) == 0
    try:
        dw = G.experts_grad_weight(dy, x, off)
        assert not told(G)
    finally:
        assert G.lib().psgd_experts_set_wait(0, 0) == 0
    for e in (0, experts - 1):
        a, b = ends[e], ends[e + 1]
        assert torch.equal(dw[e, :64].double(), dy[a:b, :64].double().T @ x[a:b].double())
