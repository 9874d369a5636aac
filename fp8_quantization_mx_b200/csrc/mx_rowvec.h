// The rows of a contiguous [rows, cols] matrix as vectors of 8 elements. Plain
// index arithmetic: it compiles without CUDA too, so that its bounds can be
// checked on a host.

#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MX_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MX_HOST_DEVICE inline
#endif

namespace mxk {

// ODD: cols is no multiple of 8, so that rows start at any element of a vector.
// The vectors are those of the memory then, shifted by the row's start among
// them; the first and the last of a row hold elements of its neighbours (of
// several rows where cols < 7). The rows that share one RowVectors are a
// multiple of 8 apart, or all start where `row` does.
template <bool ODD>
struct RowVectors {
  int64_t rows, cols, tail;   // rows before `tail` end 8 elements or more before the matrix does
  int shift, count;
  MX_HOST_DEVICE RowVectors(int64_t rows_, int64_t cols_, int64_t row)
      : rows(rows_),
        cols(cols_),
        tail(rows_ - 1 - (cols_ < 8 ? 7 / static_cast<int>(cols_) : 0)),
        shift(ODD ? static_cast<int>(row * cols_ & 7) : 0),
        count(ODD ? (shift + static_cast<int>(cols_) + 7) / 8 : static_cast<int>(cols_) / 8) {}
  // The first element of vector i of a row: a multiple of 8, at least 0.
  MX_HOST_DEVICE int64_t at(int64_t row, int i) const { return row * cols - shift + 8 * i; }
  // The row's own elements of vector i: lo..hi - 1.
  MX_HOST_DEVICE int lo(int i) const { return i == 0 ? shift : 0; }
  MX_HOST_DEVICE int hi(int i) const {
    const int n = shift + static_cast<int>(cols) - 8 * i;
    return n < 8 ? n : 8;
  }
  MX_HOST_DEVICE bool whole(int i) const { return !ODD || (lo(i) == 0 && hi(i) == 8); }
  // Whether the matrix's end may cut vector i of a row (with few columns, that of
  // several rows), and how many of its elements there are then.
  MX_HOST_DEVICE bool cut(int64_t row, int i) const { return ODD && i == count - 1 && row >= tail; }
  MX_HOST_DEVICE int held(int64_t row, int i) const {
    const int64_t left = rows * cols - at(row, i);
    return left < 8 ? static_cast<int>(left) : 8;
  }
};

}  // namespace mxk
