"""The vectors that the norm's gradient reads, by the kernel's own index
arithmetic (csrc/mx_rowvec.h) on a host: every read lies in the matrix and
covers the row."""

import ctypes
import os
import subprocess

import pytest

SOURCE = r"""
#include "mx_rowvec.h"
using namespace mxk;
// Of the vectors of every row: those that reach outside the matrix, those that
// do not hold what the row has in them, and those unaligned; the rows' elements
// that none holds.
template <bool ODD>
void check(int64_t rows, int cols, int64_t* bad) {
  for (int64_t row = 0; row < rows; ++row) {
    const RowVectors<ODD> v(rows, cols, row);
    int64_t own = 0;
    for (int i = 0; i < v.count; ++i) {
      const int64_t at = v.at(row, i);
      const int read = v.cut(row, i) ? v.held(row, i) : 8;
      bad[0] += at < 0 || at + read > rows * cols;
      bad[1] += read < v.hi(i);
      bad[2] += at % 8 != 0;
      for (int e = v.lo(i); e < v.hi(i); ++e) own += at + e == row * cols + own;
    }
    bad[3] += own != cols;
  }
}
extern "C" void check_matrix(int64_t rows, int cols, int64_t* bad) {
  cols % 8 ? check<true>(rows, cols, bad) : check<false>(rows, cols, bad);
}
"""


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    d = tmp_path_factory.mktemp("rowvec")
    (d / "check.cpp").write_text(SOURCE)
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "fp8_quantization_mx_b200", "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{csrc}", str(d / "check.cpp"),
                    "-o", str(d / "check.so")], check=True)
    lib = ctypes.CDLL(str(d / "check.so"))
    lib.check_matrix.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]

    def run(rows, cols):
        bad = (ctypes.c_int64 * 4)()
        lib.check_matrix(rows, cols, bad)
        return list(bad)

    return run


@pytest.mark.parametrize("cols", [*range(1, 34), 131, 1001, 4096])
def test_vectors_stay_in_the_matrix_and_cover_the_row(check, cols):
    for rows in range(1, 41):
        assert check(rows, cols) == [0, 0, 0, 0], rows
