"""Dropout against its definition: the generator on the host, bit for bit.

A kept value is x times one float32 number, rounded once to float32 and once to
its type: half a step of each.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def G():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


def words(counter, key):
    """Philox 4x32 with 10 rounds of (n, 4) counters, in 64-bit integers."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1)


def kept(n, p, seed, step, site=0, first=0):
    """Which of values first .. first + n - 1 are kept, and by what they are scaled."""
    i = np.arange(first, first + n, dtype=np.uint64)
    g = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    seed, step = seed % 2 ** 64, step % 2 ** 64
    low = np.uint64(0xFFFFFFFF)
    counter = np.stack([g & low, (g >> np.uint64(32)) | np.uint64(site << 16), np.full_like(g, step & 0xFFFFFFFF),
                        np.full_like(g, step >> 32)], -1)
    w = words(counter, (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(-1)
    cut = round(p * 65536)
    mine = bits[(i - np.uint64(first // 8 * 8)).astype(np.int64)] >= cut
    return torch.from_numpy(mine), 65536 / (65536 - cut) if cut < 65536 else 0.0


def check(y, x, p, seed, step, site=0):
    mask, scale = kept(x.numel(), p, seed, step, site)
    mask = mask.view(x.shape)
    y, want = y.cpu(), torch.where(mask, x.cpu().double() * scale, 0.0)
    assert bool((y[~mask] == 0).all())
    tol = want.abs() * (ROUND[x.dtype] + 2.0 ** -23) + (2.0 ** -25 if x.dtype is torch.float16 else 0.0)
    assert bool(((y.double() - want).abs() <= tol).all())


def test_published_vectors():
    # the generator's authors' known answers
    assert [int(v) for v in words(np.zeros((1, 4), dtype=np.uint64), (0, 0))[0]] == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    ones = np.full((1, 4), 0xFFFFFFFF, dtype=np.uint64)
    assert [int(v) for v in words(ones, (0xFFFFFFFF, 0xFFFFFFFF))[0]] == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 5), (33, 65), (700, 650), (5, 3, 17), (2, 1000003)], ids=str)
def test_values(G, dtype, shape):
    x = torch.randn(shape, device="cuda").to(dtype)
    for p, seed, step, site in ((0.1, 5, 0, 0), (0.65, -3, 2 ** 40 + 1, 65535), (0.5, 2 ** 62 + 7, -1, 9)):
        check(G.dropout(x, p, G.dropout_state(seed, step), site), x, p, seed, step, site)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 2.0 ** -16, 0.3, 1.0 - 2.0 ** -16, 1.0])
def test_probabilities(G, p):
    x = torch.randn(100000, device="cuda")
    y = G.dropout(x, p, G.dropout_state(1, 2))
    check(y, x, p, 1, 2)
    if p < 2.0 ** -17:
        assert torch.equal(x, y)
    if p == 1.0:
        assert not y.any()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_strides_and_alignment(G, dtype):
    state = G.dropout_state(3, 4)
    wide = torch.randn(67, 145, device="cuda").to(dtype)
    for x in (wide[:, 2:131], wide[:, 8:136], wide[1:, :], wide.t(), wide[:1].expand(40, 145), wide.reshape(-1)[3:],
              wide[::2, ::3], wide[:, 4], wide[:, :1], wide.view(67, 5, 29).transpose(0, 1)):
        check(G.dropout(x, 0.4, state), x.contiguous(), 0.4, 3, 4)
    out = torch.full((67, 150), 5.0, device="cuda").to(dtype)
    G.dropout(wide, 0.4, state, out=out[:, 3:148])
    check(out[:, 3:148], wide, 0.4, 3, 4)
    assert bool((out[:, :3] == 5).all()) and bool((out[:, 148:] == 5).all())
    same = wide.clone()
    G.dropout(same, 0.4, state, out=same)
    check(same, wide, 0.4, 3, 4)


def test_nothing_and_anything(G):
    state = G.dropout_state(1)
    assert G.dropout(torch.empty(0, 5, device="cuda"), 0.5, state).shape == (0, 5)
    x = torch.full((4096,), float("nan"), device="cuda")
    x[::3] = float("inf")
    y = G.dropout(x, 0.5, state).cpu()
    mask, _ = kept(4096, 0.5, 1, 0)
    assert bool((y[~mask] == 0).all()) and not bool(torch.isfinite(y[mask]).any())


def test_share_and_independence(G):
    # 2^24 draws: the share of kept values is within 6 standard deviations, and two sites' masks agree as often as chance has it
    x, n = torch.ones(1 << 24, device="cuda"), 1 << 24
    a, b = (G.dropout(x, 0.25, G.dropout_state(11, 5), site) != 0 for site in (1, 2))
    c = G.dropout(x, 0.25, G.dropout_state(11, 6), 1) != 0
    for m in (a, b, c):
        assert abs(float(m.double().mean()) - 0.75) < 6 * (0.75 * 0.25 / n) ** 0.5
    for m in (b, c):
        assert abs(float((a & m).double().mean()) - 0.5625) < 6 * (0.5625 * 0.4375 / n) ** 0.5


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_gradient(G, dtype):
    x = torch.randn(50, 77, device="cuda").to(dtype).requires_grad_()
    dy = torch.randn(77, 50, device="cuda").to(dtype).t()
    state = G.dropout_state(21, 3)
    y = G.dropout(x, 0.35, state, site=4)
    state[1] += 1  # the backward pass keeps to what the forward pass saw
    y.backward(dy)
    check(x.grad, dy.contiguous(), 0.35, 21, 3, 4)
    with torch.no_grad():
        check(G.dropout(x, 0.35, state, site=4), x.detach(), 0.35, 21, 4, 4)
    x.grad = None
    G.dropout(x, 0.35, state).sum().backward()  # a gradient of stride 0
    check(x.grad, torch.ones_like(x), 0.35, 21, 4)


def test_a_captured_call_goes_on_with_the_state(G):
    x, state = torch.randn(1000, device="cuda"), G.dropout_state(8, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.dropout(x, 0.5, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = G.dropout(x, 0.5, state)
        state[1] += 1
    for step in range(3):
        graph.replay()
        check(y, x, 0.5, 8, step)


def test_values_behind_32_bits(G):
    n = (1 << 32) + 12345
    x = torch.ones(n, device="cuda", dtype=torch.float16)
    y = G.dropout(x, 0.5, G.dropout_state(4, 4))
    mask, scale = kept(12345, 0.5, 4, 4, first=1 << 32)
    assert torch.equal(y[1 << 32:].cpu().double(), mask * scale)
    far = (1 << 35) + 8  # the counter's second word
    assert kept(8, 0.5, 4, 4, first=far)[0].shape == (8,)


def test_refusals(G):
    x, state = torch.randn(10, 8, device="cuda"), G.dropout_state(1)
    for error, call in ((TypeError, lambda: G.dropout(x.double(), 0.5, state)), (ValueError, lambda: G.dropout(x.cpu(), 0.5, state)),
                        (ValueError, lambda: G.dropout(x, 1.5, state)), (ValueError, lambda: G.dropout(x, float("nan"), state)),
                        (ValueError, lambda: G.dropout(x, 0.5, None)), (ValueError, lambda: G.dropout(x, 0.5, state.cpu())),
                        (TypeError, lambda: G.dropout(x, 0.5, state.int())), (ValueError, lambda: G.dropout(x, 0.5, state[:1])),
                        (G.PsgdError, lambda: G.dropout(x, 0.5, state, site=-1)),
                        (G.PsgdError, lambda: G.dropout(x, 0.5, state, site=65536)),
                        (TypeError, lambda: G.dropout(x, 0.5, state, out=x.half())),
                        (ValueError, lambda: G.dropout(x, 0.5, state, out=torch.empty(8, 10, device="cuda"))),
                        (ValueError, lambda: G.dropout(x, 0.5, state, out=torch.empty(8, 10, device="cuda").t())),
                        (RuntimeError, lambda: G.dropout(x.clone().requires_grad_(), 0.5, state, out=x))):
        with pytest.raises(error):
            call()
