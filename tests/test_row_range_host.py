"""The rows of a ragged batch's sequence (csrc/row_range.h) on the CPU: the first row of a
sequence without a query is read before its length is looked at, so it has to exist."""
import ctypes
import itertools
import os
import subprocess

import pytest

from vector_quantized_bit_gb300 import _build


@pytest.fixture(scope="module")
def rows_of(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src, so = d / "rows.cpp", d / "rows.so"
    src.write_text("""#include "row_range.h"
extern "C" void rows_of(int start, int end, int n_rows, int max_queries, int* out) {
  bool fine;
  const vqkv::RowRange r = vqkv::rows_of_starts(start, end, n_rows, max_queries, &fine);
  out[0] = r.first, out[1] = r.n, out[2] = fine;
}
""")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", os.path.join(_build.PKG, "csrc"),
                    str(src), "-o", str(so)], check=True)
    f = ctypes.CDLL(str(so)).rows_of

    def go(*a):
        out = (ctypes.c_int * 3)()
        f(*a, out)
        return tuple(out)
    return go


BITS = [-2**31, -2**31 + 1, -7, -1, 0, 1, 2, 3, 4, 5, 6, 100, 2**27, 2**30, 2**31 - 2, 2**31 - 1]


@pytest.mark.parametrize("n_rows", [1, 2, 5, 2**27])
@pytest.mark.parametrize("most", [1, 3, 2**27])
def test_every_row_named_exists(rows_of, n_rows, most):
    for start, end in itertools.product(BITS, BITS):
        first, n, fine = rows_of(start, end, n_rows, most)
        assert 0 <= first < n_rows and 0 <= n and first + n <= n_rows, (start, end)
        ascend = 0 <= start <= end <= n_rows
        assert n == (min(end - start, most) if ascend else 0), (start, end)
        assert fine == (ascend and end - start <= most), (start, end)
        assert n == 0 or first == start


def test_last_sequences_without_a_query(rows_of):
    """Starts 0, 1, 2, 2, 2 of two rows: sequences 2 and 3 would begin at row 2, which is not there."""
    assert [rows_of(a, b, 2, 1) for a, b in ((0, 1), (1, 2), (2, 2), (2, 2))] == [(0, 1, 1), (1, 1, 1), (0, 0, 1), (0, 0, 1)]
