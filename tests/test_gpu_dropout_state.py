"""Dropout without a state is refused in the same way whether torch records the call or not."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


@pytest.mark.parametrize("grad", [False, True])
def test_refusals(G, grad):
    x, state = torch.randn(10, 8, device="cuda", requires_grad=grad), G.dropout_state(1)
    for error, call in ((ValueError, lambda: G.dropout(x, 0.5, None)), (ValueError, lambda: G.dropout(x, 0.0, None)),
                        (ValueError, lambda: G.rms_norm(x, p=0.5)), (ValueError, lambda: G.rms_norm(x, p=1.5, state=state)),
                        (ValueError, lambda: G.dropout(x, 0.5, state.cpu())), (TypeError, lambda: G.dropout(x, 0.5, state.int())),
                        (ValueError, lambda: G.rms_norm(x, p=0.5, state=state[:1])),
                        (G.PsgdError, lambda: G.dropout(x, 0.5, state, site=-1)),
                        (G.PsgdError, lambda: G.rms_norm(x, p=0.5, state=state, site=70000))):
        with pytest.raises(error):
            call()
    y, r = G.rms_norm(x, p=0.0)  # without dropout no state is needed
    assert r is x and y.requires_grad == grad
