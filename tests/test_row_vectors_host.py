"""Where the norm's kernels read whole vectors of rows that do not start on them: nothing behind the tensor.

The kernels' own arithmetic (psgd_row_vectors.h), compiled for the host.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "psgd_row_vectors.h"
extern "C" int first_offset(long long row, int width) { return psgd::first_offset(row, width); }
extern "C" int vectors_of(int off, int width) { return psgd::vectors_of(off, width); }
extern "C" long long first_ragged(long long rows, int width) { return psgd::first_ragged(rows, width); }
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("rows")
    (at / "rule.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "rank_gradient_compression_layer_gb300", "csrc"), str(at / "rule.cpp"), "-o",
                    str(at / "rule.so")], check=True)
    lib = ctypes.CDLL(str(at / "rule.so"))
    lib.first_ragged.restype, lib.first_ragged.argtypes = ctypes.c_longlong, [ctypes.c_longlong, ctypes.c_int]
    lib.first_offset.argtypes = [ctypes.c_longlong, ctypes.c_int]
    return lib


@pytest.mark.parametrize("width", list(range(1, 26)) + [650, 651, 655, 8191])
def test_no_whole_vector_ends_behind_the_tensor(rule, width):
    for rows in range(1, 40):
        n, ragged = rows * width, rule.first_ragged(rows, width)
        for row in range(rows):
            off = rule.first_offset(row, width)
            vecs = rule.vectors_of(off, width)
            start = row * width - off
            assert start % 8 == 0 and 0 <= off < 8
            assert start + 8 * vecs >= (row + 1) * width > start + 8 * (vecs - 1)
            # all vectors but the last are read whole, and that one too up to `ragged`
            whole = vecs - 1 if row >= ragged else vecs
            assert start + 8 * whole <= n, (rows, row)
            if row >= ragged:  # and none is read value by value without need
                assert start + 8 * vecs > n, (rows, row)


def test_rows_past_32_bits(rule):
    for width in (1, 3, 7, 651):
        rows = (1 << 35) + 5
        assert rule.first_offset(rows - 1, width) == (rows - 1) * width % 8
        assert rule.first_ragged(rows, width) == rows * width // 8 * 8 // width
