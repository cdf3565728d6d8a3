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


@pytest.fixture
def product(G):
    off = torch.tensor([0, 300, 300, 341], dtype=torch.int32, device="cuda")
    x, w = whole(1, 341, 200), whole(2, 3, 264, 200)
    want = torch.cat([x[:300].float() @ w[0].float().T, x[300:].float() @ w[2].float().T]).bfloat16()
    torch.cuda.synchronize()
    return lambda: G.experts_forward(x, w, off), want


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
