"""Refusals of the C entries of the language model's operators, which touch no GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def pkg():
    import rank_gradient_compression_layer_gb300 as p
    p.build()
    return p


A = 1 << 20  # an aligned address that no call gets to use


def loss_args(**kw):
    from rank_gradient_compression_layer_gb300.binding import CrossEntropyArgs
    a = dict(rows=4, vocab=9, width=8, x=A, ldx=8, w=A, ldw=8, target=A, target_bytes=8, ignore_index=-100, scale=1.0, dtype=1,
             loss=A)
    a.update(kw)
    args = CrossEntropyArgs()
    for name, value in a.items():
        setattr(args, name, value)
    return args


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=(1 << 30) + 1), dict(vocab=0), dict(vocab=(1 << 20) + 1), dict(width=0),
                                 dict(width=(1 << 20) + 1), dict(dtype=0), dict(dtype=3), dict(target_bytes=2), dict(x=None),
                                 dict(x=A + 1), dict(w=None), dict(target=None), dict(target=A + 4), dict(ldx=-8), dict(ldw=-1),
                                 dict(bias=A, bias_dtype=2), dict(bias=A + 1, bias_dtype=1), dict(bias=A + 2, bias_dtype=0),
                                 dict(row_scale=A + 2), dict(scale_dev=A + 1), dict(losses=A + 2), dict(loss=A + 2),
                                 dict(loss=None), dict(dx=A + 1, lddx=8), dict(dx=A, lddx=7), dict(dw=A, lddw=7, dw_dtype=1),
                                 dict(dw=A + 2, lddw=8, dw_dtype=0), dict(dw=A, lddw=8, dw_dtype=2), dict(db=A, db_dtype=2),
                                 dict(db=A + 1, db_dtype=1), dict(scale=float("nan"))], ids=str)
def test_cross_entropy_refuses(pkg, bad):
    lib, args = pkg.lib(), loss_args(**bad)
    assert lib.psgd_cross_entropy(ctypes.byref(args), A, 1 << 40, None) == pkg.PSGD_ERR_INVALID
    assert lib.psgd_last_error()


def test_cross_entropy_refuses_its_workspace(pkg):
    lib, size = pkg.lib(), ctypes.c_size_t()
    for kw in (dict(), dict(rows=300, dx=A, lddx=8, dw=A, lddw=8, dw_dtype=1)):
        args = loss_args(**kw)
        assert lib.psgd_cross_entropy_workspace(ctypes.byref(args), ctypes.byref(size)) == 0 and size.value
        for ws, bytes_ in ((None, 1 << 40), (A + 16, 1 << 40), (A, size.value - 1)):
            assert lib.psgd_cross_entropy(ctypes.byref(args), ws, bytes_, None) == pkg.PSGD_ERR_INVALID
    assert lib.psgd_cross_entropy_workspace(None, ctypes.byref(size)) == pkg.PSGD_ERR_INVALID
    assert lib.psgd_cross_entropy_workspace(ctypes.byref(args), None) == pkg.PSGD_ERR_INVALID
    assert lib.psgd_cross_entropy(None, A, 1 << 40, None) == pkg.PSGD_ERR_INVALID


def test_cross_entropy_keeps_to_chunks(pkg):
    # the buffers of the exponentials and of the rows do not grow with the rows
    lib, size = pkg.lib(), ctypes.c_size_t()
    for rows, vocab, width in ((1 << 20, 131072, 4096), (1 << 24, 256, 64), (300000, 33278, 650), (256, 1 << 20, 64)):
        args = loss_args(rows=rows, vocab=vocab, width=width, ldx=width, ldw=width, dx=A, lddx=width, dw=A, lddw=width, dw_dtype=0)
        assert lib.psgd_cross_entropy_workspace(ctypes.byref(args), ctypes.byref(size)) == 0
        copies = 2 * (rows + vocab) * (width + 8)
        assert size.value < (10 << 30) + 16 * rows + copies + 8 * vocab * width


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=-1), dict(rows=1 << 40, cols=1 << 10), dict(dtype=3), dict(x=None),
                                 dict(y=None), dict(x=A + 1), dict(y=A + 2, dtype=0), dict(p=-0.1), dict(p=1.1),
                                 dict(p=float("nan")), dict(state=None), dict(state=A + 4), dict(site=-1), dict(site=1 << 16),
                                 dict(seen=A + 4), dict(ldx=-1), dict(ldy=7)], ids=str)
def test_dropout_refuses(pkg, bad):
    a = dict(rows=4, cols=8, dtype=1, x=A, ldx=8, y=A, ldy=8, p=0.5, state=A, site=0, seen=None)
    a.update(bad)
    rc = pkg.lib().psgd_dropout(a["rows"], a["cols"], a["dtype"], a["x"], a["ldx"], a["y"], a["ldy"], a["p"], a["state"],
                                a["site"], a["seen"], None)
    assert rc == pkg.PSGD_ERR_INVALID and pkg.lib().psgd_last_error()


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(width=0), dict(width=24001), dict(dtype=3), dict(x=None), dict(x=A + 8),
                                 dict(res=A + 8), dict(y=None), dict(y=A + 2), dict(r=None, res=A), dict(r=None, p=0.5),
                                 dict(ldx=9), dict(ldx=7), dict(width=9, ldx=16, ldy=9), dict(w=A, wdt=2), dict(w=A + 1, wdt=1),
                                 dict(eps=0.0), dict(eps=float("inf")), dict(eps=float("nan")), dict(p=2.0),
                                 dict(p=0.5, state=None), dict(seen=A + 1)], ids=str)
def test_rms_norm_refuses(pkg, bad):
    a = dict(rows=4, width=8, dtype=1, x=A, ldx=8, res=None, ldres=8, w=None, wdt=1, eps=1e-6, p=0.0, state=A, site=0, seen=None,
             y=A, ldy=8, r=A, ldr=8)
    a.update(bad)
    rc = pkg.lib().psgd_rms_norm(*a.values(), None)
    assert rc == pkg.PSGD_ERR_INVALID and pkg.lib().psgd_last_error()


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(width=24001), dict(dtype=4), dict(dy=None), dict(r=None), dict(r=A + 8),
                                 dict(dr=A + 2), dict(dx=A, dro=A), dict(dx=A + 8, p=0.5), dict(dro=None), dict(lddy=12),
                                 dict(dw=A, dwdt=2), dict(dw=A + 2, dwdt=0), dict(dw=A, dwdt=0), dict(dw=A, dwdt=0, ws=A, n=64),
                                 dict(dw=A, dwdt=0, ws=A + 4, n=1 << 30), dict(eps=-1.0), dict(p=0.5, state=None)], ids=str)
def test_rms_norm_grad_refuses(pkg, bad):
    a = dict(rows=4, width=8, dtype=1, dy=A, lddy=8, r=A, ldr=8, dr=None, lddr=8, w=None, wdt=1, eps=1e-6, p=0.0, state=A, site=0,
             dx=None, lddx=8, dro=A, lddro=8, dw=None, dwdt=0, add=0, ws=None, n=0)
    a.update(bad)
    rc = pkg.lib().psgd_rms_norm_grad(*a.values(), None)
    assert rc == pkg.PSGD_ERR_INVALID and pkg.lib().psgd_last_error()


def test_structure_and_sizes_agree(pkg):
    # what the binding repeats of the header
    import os
    import re
    from rank_gradient_compression_layer_gb300 import binding
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "psgd.h")).read()
    body = re.search(r"typedef struct psgd_cross_entropy_args \{(.*?)\}", src, re.S).group(1)
    names = []
    for line in re.sub(r"/\*.*?\*/", "", body, flags=re.S).split(";"):
        m = re.match(r"\s*(?:const\s+)?\w+\s*\*?\s*(.*)", line.strip(), re.S)
        if m and line.strip():
            names += [n.strip(" *\n") for n in m.group(1).split(",")]
    assert names == [f[0] for f in binding.CrossEntropyArgs._fields_]
    assert int(re.search(r"PSGD_MAX_NORM_WIDTH (\d+)", src).group(1)) == binding.PSGD_MAX_NORM_WIDTH


@pytest.mark.parametrize("call", [lambda G, t: G.dropout(t, 0.5, t.long()), lambda G, t: G.rms_norm(t),
                                  lambda G, t: G.rms_norm_grad(t, t),
                                  lambda G, t: G.linear_cross_entropy(t.bfloat16(), t.bfloat16(), t[:, 0].long())])
def test_host_tensors_are_refused(pkg, call):
    with pytest.raises(ValueError):
        call(pkg, torch.zeros(4, 8))


def test_the_binding_knows_the_norms_workspace(pkg):
    from rank_gradient_compression_layer_gb300.language import _NORM_CTAS
    size = ctypes.c_size_t()
    for rows in (0, 1, _NORM_CTAS - 1, _NORM_CTAS, _NORM_CTAS + 1, 1 << 30):
        for width in (1, 651, 24000):
            assert pkg.lib().psgd_rms_norm_workspace(rows, width, ctypes.byref(size)) == 0
            assert size.value == min(rows, _NORM_CTAS) * width * 4
