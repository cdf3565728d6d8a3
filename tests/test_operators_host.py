"""Refusals of the operators' C entries, which touch no GPU, and the strides the binding reads."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def pkg():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


A = 1 << 20  # an aligned address that no call gets to use


def forward(lib, **kw):
    a = dict(rows=4, experts=2, n=8, k=8, dtype=1, x=A, ldx=8, w=A, ldw=8, ws=64, off=A, y=A, ldy=8, scratch=None, bytes=0)
    a.update(kw)
    return lib.psgd_experts_forward(a["rows"], a["experts"], a["n"], a["k"], a["dtype"], a["x"], a["ldx"], a["w"],
                                    a["ldw"], a["ws"], a["off"], a["y"], a["ldy"], a["scratch"], a["bytes"], None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=(1 << 30) + 1), dict(experts=0), dict(experts=2049), dict(n=0),
                                 dict(k=0), dict(n=(1 << 20) + 1), dict(dtype=0), dict(dtype=3), dict(x=None),
                                 dict(x=A + 1), dict(w=None), dict(off=None), dict(off=A + 2), dict(y=None),
                                 dict(y=A + 1), dict(ldx=-8), dict(ldy=7), dict(ws=-64), dict(x=A + 2), dict(ldx=9),
                                 dict(x=A + 2, scratch=A, bytes=32), dict(x=A + 2, scratch=A + 16, bytes=1 << 20)], ids=str)
def test_forward_refuses(pkg, bad):
    assert forward(pkg.lib(), **bad) == pkg.PSGD_ERR_INVALID
    assert pkg.lib().psgd_last_error()


def test_too_many_tiles_are_refused_before_the_copy(pkg):
    # unaligned rows, which a kernel would copy to the workspace first: a refusal comes before that launch
    big = dict(rows=1 << 30, n=1 << 20, x=A + 2, ldy=1 << 20, scratch=A, bytes=1 << 60)
    assert forward(pkg.lib(), **big) == pkg.PSGD_ERR_INVALID
    side = 1 << 20
    rc = pkg.lib().psgd_experts_grad_weight(4, 2048, side, side, 1, A + 2, side, A, side, A, 0, A, side, side * side,
                                            A, 1 << 60, None)
    assert rc == pkg.PSGD_ERR_INVALID and b"tiles" in pkg.lib().psgd_last_error()


@pytest.mark.parametrize("bad", [dict(out=2), dict(dw=None), dict(dw=A + 2), dict(lddw=7), dict(stride=63)], ids=str)
def test_grad_weight_refuses(pkg, bad):
    a = dict(out=0, dw=A, lddw=8, stride=64)
    a.update(bad)
    rc = pkg.lib().psgd_experts_grad_weight(4, 2, 8, 8, 1, A, 8, A, 8, A, a["out"], a["dw"], a["lddw"], a["stride"],
                                            None, 0, None)
    assert rc == pkg.PSGD_ERR_INVALID and pkg.lib().psgd_last_error()


@pytest.mark.parametrize("bad", [dict(count=-1), dict(src=None), dict(ptr=0), dict(ptr=A + 2), dict(rows=-1),
                                 dict(cols=1 << 43), dict(ld=3, rows=2), dict(dtype=7), dict(norm=None),
                                 dict(norm=A + 1), dict(ws=None), dict(ws=A + 8), dict(bytes=64), dict(max_norm=-1.0),
                                 dict(max_norm=float("nan")), dict(out=0)], ids=str)
def test_clip_refuses(pkg, bad):
    a = dict(count=1, ptr=A, rows=1, cols=4, ld=4, dtype=0, norm=A, ws=A, bytes=1 << 20, max_norm=1.0, out=A)
    a.update(bad)
    one = lambda v: (ctypes.c_int64 * 1)(v)
    src = None if "src" in bad else (ctypes.c_void_p * 1)(a["ptr"])
    rc = pkg.lib().psgd_clip_grad_norm(a["count"], src, (ctypes.c_void_p * 1)(a["out"]), one(a["rows"]), one(a["cols"]),
                                       one(a["ld"]), one(a["ld"]), a["dtype"], a["max_norm"], a["norm"], a["ws"],
                                       a["bytes"], None)
    assert rc == pkg.PSGD_ERR_INVALID and pkg.lib().psgd_last_error()


@pytest.mark.parametrize("bad", [dict(layers=0), dict(n=0), dict(m=-1), dict(buffers=0), dict(buffers=65), dict(ptr=0),
                                 dict(ptr=A + 4), dict(norm=None), dict(bytes=0)], ids=str)
def test_packed_norm_refuses(pkg, bad):
    a = dict(layers=1, n=4, m=4, buffers=1, ptr=A, norm=A, bytes=1 << 20)
    a.update(bad)
    one = lambda v: (ctypes.c_int64 * 1)(v)
    rc = pkg.lib().psgd_packed_grad_norm(a["layers"], one(a["n"]), one(a["m"]), a["buffers"],
                                         (ctypes.c_void_p * 65)(*[a["ptr"]] * 65), a["norm"], A, a["bytes"], None)
    assert rc == pkg.PSGD_ERR_INVALID and pkg.lib().psgd_last_error()


def test_workspace_of_a_product(pkg):
    size = ctypes.c_size_t()

    def need(op, a, lda, b, ldb, stride, n=24, k=20):
        assert pkg.lib().psgd_experts_workspace(op, 5, 3, n, k, a, lda, b, ldb, stride, ctypes.byref(size)) == 0
        return size.value
    up = lambda v: (v + 255) // 256 * 256
    from rank_gradient_compression_layer_gb300.operators import _plain
    for at, ld, stride in ((A, 24, 576), (A, 20, 480), (A + 2, 24, 576), (A, 0, 576), (A, 24, 0), (A, 24, 584)):
        # the binding's own look at the weights and at the rows
        assert _plain(at, ld, stride, 3, 20) == (need(0, A, 24, at, ld, stride) == 0)
        assert _plain(at, ld, 0, 1, 20) == (need(0, at, ld, A, 24, 576) == 0)
    x, w = up(5 * 24 * 2), up(3 * 24 * 24 * 2)  # rows of 20 values take 24
    assert need(0, A, 24, A, 24, 24 * 24) == 0
    assert need(0, A, 20, A, 24, 24 * 24) == x
    assert need(0, A + 2, 24, A, 24, 24 * 24) == x
    assert need(0, A, 0, A, 24, 24 * 24) == x
    assert need(0, A, 24, A, 20, 480) == w
    assert need(0, A, 24, A, 24, 0) == w            # one matrix for all experts
    assert need(0, A, 24, A, 24, 24 * 24 + 8) == w  # not a whole number of rows apart
    assert need(0, A, 20, A, 20, 480) == x + w
    assert need(1, A, 24, A, 24, 24 * 24) == 0
    assert need(1, A, 25, A, 24, 24 * 24) == up(5 * 24 * 2)
    assert need(2, A, 24, A, 20, 0) == x
    assert pkg.lib().psgd_experts_workspace(3, 5, 3, 24, 20, A, 24, A, 24, 576, ctypes.byref(size)) == pkg.PSGD_ERR_INVALID


def test_workspace_of_sums_in_parts(pkg):
    size = ctypes.c_size_t()

    def need(op, rows, experts, n, k):
        assert pkg.lib().psgd_experts_workspace(op, rows, experts, n, k, A, max(n, k), A, max(n, k), n * max(n, k),
                                                ctypes.byref(size)) == 0
        return size.value
    # 1 row, 1 tile of 128 blocks: 8 parts; 39 tiles or 95 blocks: none
    assert need(0, 1, 1, 256, 8192) == 8 * 1 * 256 * 4
    assert need(1, 1, 1, 8192, 256) == 8 * 1 * 256 * 4
    assert need(0, 1, 1, 38 * 256, 8192) == 2 * 1 * 38 * 256 * 4
    assert need(0, 1, 1, 39 * 256, 8192) == 0
    assert need(0, 1, 1, 256, 95 * 64) == 0
    assert need(0, 1, 1, 256, 96 * 64) == 6 * 1 * 256 * 4
    # one 256 x 256 tile, 30000 rows (469 blocks): segments of 16 blocks
    assert need(2, 30000, 1, 256, 256) == ((469 + 29) // 16 + 29 + 1) * 256 * 256 * 4
    assert need(2, 1024, 1, 256, 256) == 0
    assert need(2, 30000, 1, 2560, 2048) == 0
    assert need(2, 6000, 76, 256, 256) == 0 and need(2, 6000, 75, 256, 256) and need(2, 6100, 76, 256, 256)


def test_the_binding_knows_when_sums_need_room(pkg):
    # the binding leaves the library's answer unasked where it says none: the two have to agree at every limit
    import random
    from rank_gradient_compression_layer_gb300.operators import _rows_in_one_piece, _weights_in_one_piece
    size = ctypes.c_size_t()

    def room(op, rows, experts, n, k):
        ld = (max(n, k) + 7) // 8 * 8
        assert pkg.lib().psgd_experts_workspace(op, rows, experts, n, k, A, ld, A, ld, n * ld, ctypes.byref(size)) == 0
        return size.value > 0

    rng = random.Random(1)
    near = lambda *at: max(1, rng.choice(at) + rng.choice((-65, -64, -1, 0, 1, 64, 65)))
    for _ in range(20000):
        side, depth = near(1, 256, 256 * 37, 256 * 38, 256 * 39), near(64, 1024, 64 * 95, 64 * 96, 32768, 262144, 1 << 19)
        rows, experts = near(1, 256, 256 * 37, 256 * 75, 30000), rng.choice((1, 2, 3, 37, 38, 39, 75, 76, 77, 500))
        assert _rows_in_one_piece(pkg.PSGD_F16, rows, experts, side, depth) != room(0, rows, experts, side, depth)
        assert _rows_in_one_piece(pkg.PSGD_F16, rows, experts, side, depth) != room(1, rows, experts, depth, side)
        if depth <= 32768 or depth > 262144:  # the size is float16's, which bfloat16 needs less often in between
            assert (_rows_in_one_piece(pkg.PSGD_BF16, rows, experts, side, depth)
                    == _rows_in_one_piece(pkg.PSGD_F16, rows, experts, side, depth))
        rows = near(1, 64 * 16, 64 * 95, 64 * 96, 30000, 65536, 1 << 20)
        n, k = near(1, 256, 512, 256 * 7, 256 * 50, 256 * 51), near(1, 256, 256 * 7, 256 * 8)
        assert _weights_in_one_piece(rows, experts, n, k) != room(2, rows, experts, n, k)


def test_room_for_exact_sums_is_a_quarter_at_most(pkg):
    from rank_gradient_compression_layer_gb300.operators import _weights_in_one_piece
    size = ctypes.c_size_t()
    for rows, experts, n, k in ((70000, 1, 16384, 16384), (1 << 20, 1, 16384, 16384), (1 << 18, 64, 8192, 2048),
                                (1 << 20, 2, 2048, 2048), (65600, 8, 4096, 14336), (1 << 22, 1, 30000, 30001)):
        ld = (max(n, k) + 7) // 8 * 8
        assert pkg.lib().psgd_experts_workspace(2, rows, experts, n, k, A, ld, A, ld, 0, ctypes.byref(size)) == 0
        assert size.value <= (rows * (n + k) * 2 + experts * n * k * 4) // 4 + 256
        assert _weights_in_one_piece(rows, experts, n, k) == (size.value == 0)


def test_wait_limit_refuses(pkg):
    for ms in (-1, 60001):
        assert pkg.lib().psgd_experts_set_wait(ms, 0) == pkg.PSGD_ERR_INVALID
    assert pkg.lib().psgd_experts_set_wait(0, 0) == 0


def test_header_constants(pkg):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "psgd.h")).read()
    assert f"#define PSGD_MAX_EXPERTS {pkg.PSGD_MAX_EXPERTS}" in src
    assert re.search(r"#define PSGD_GRAD_NORM_WORKSPACE \(\(size_t\)1 << 20\)", src)
    assert pkg.PSGD_GRAD_NORM_WORKSPACE == 1 << 20
    assert "PSGD_F32 = 0, PSGD_BF16 = 1, PSGD_F16 = 2" in src
    assert (pkg.PSGD_F32, pkg.PSGD_BF16, pkg.PSGD_F16) == (0, 1, 2)


def test_rows_of_strided_tensors(pkg):
    from rank_gradient_compression_layer_gb300.operators import _two_dims
    t = torch.zeros(6, 10)
    assert _two_dims(t) == (1, 60, 60)
    assert _two_dims(t.t()) == (1, 60, 60)
    assert _two_dims(t[:, :7]) == (6, 7, 10)
    assert _two_dims(t[1:3, :7].t()) == (2, 7, 10)
    assert _two_dims(t[:, 3]) == (6, 1, 10)
    assert _two_dims(t[2:3, 1:2]) == (1, 1, 1)
    assert _two_dims(torch.zeros(4, 6, 5, 7).to(memory_format=torch.channels_last)) == (1, 840, 840)
    assert _two_dims(torch.zeros(4, 6, 10)[:, :, :7]) == (24, 7, 10)
    assert _two_dims(torch.zeros(4, 6, 10)[:, :5, :7]) is None
    assert _two_dims(t[:1].expand(6, 10)) is None


def test_layout_matches_the_context_layout(pkg):
    shapes = [(64, 27), (10, 0), (5, 6), (5, 6), (7, 0)]
    layout = pkg.GradientLayout(shapes)
    assert (layout.offsets, layout.lds, layout.total) == pkg.psgd_plan_layout(shapes)
    buf = torch.arange(layout.total, dtype=torch.float32)
    v = layout.experts_view(buf, 2, 2)
    assert v.shape == (2, 5, 6)
    assert torch.equal(v[1], layout.layer_view(buf, 3))
    for first, experts in ((0, 2), (1, 1), (2, 3), (4, 2)):
        with pytest.raises(ValueError):
            layout.experts_view(buf, first, experts)
