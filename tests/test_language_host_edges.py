"""The language model's operators at the ends of what they accept, refuse and ask for; no GPU is touched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_language_host import A, loss_args, pkg  # noqa: E402,F401


def test_the_loss_of_no_rows_has_nothing_to_do(pkg):
    # an empty tensor's address is 0: no result is asked for, as with dx alone
    lib, size = pkg.lib(), ctypes.c_size_t()
    args = loss_args(rows=0, x=None, target=None, loss=None, lddx=8)
    assert lib.psgd_cross_entropy_workspace(ctypes.byref(args), ctypes.byref(size)) == 0
    assert lib.psgd_cross_entropy(ctypes.byref(args), A, size.value, None) == 0


@pytest.mark.parametrize("p", [0.0, 0.5])
def test_the_norm_of_no_rows_has_nothing_to_do(pkg, p):
    lib = pkg.lib()
    assert lib.psgd_rms_norm(0, 8, 1, None, 8, None, 8, None, 1, 1e-6, p, A, 0, None, None, 8, None, 8, None) == 0
    assert lib.psgd_rms_norm_grad(0, 8, 1, None, 8, None, 8, None, 8, None, 1, 1e-6, p, A, 0, None, 8, None, 8, None, 0, 0, None,
                                  0, None) == 0


@pytest.mark.parametrize("call", [lambda G, t: G.dropout(t, 0.5, None), lambda G, t: G.rms_norm(t, p=0.5)])
@pytest.mark.parametrize("grad", [False, True])
def test_dropout_without_a_state(pkg, call, grad):
    # the same error whether torch records the call or not
    with pytest.raises(ValueError):
        call(pkg, torch.zeros(4, 8, requires_grad=grad))


def test_the_biass_gradient_alone_needs_no_room_for_the_matrixs(pkg):
    lib, size = pkg.lib(), ctypes.c_size_t()
    kw = dict(rows=1024, vocab=131072, width=4096, ldx=4096, ldw=4096, bias=A, bias_dtype=0, db=A, db_dtype=0)
    args = loss_args(**kw)
    assert lib.psgd_cross_entropy_workspace(ctypes.byref(args), ctypes.byref(size)) == 0
    # the exponentials, and statistics of each 64 words: the matrix's sums would be 2 GiB
    assert size.value < 2 * 1024 * 131072 + 2 * 4 * 1024 * 131072 // 64 + (64 << 20)
