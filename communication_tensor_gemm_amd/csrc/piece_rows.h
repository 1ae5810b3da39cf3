// Pieces of eight elements numbered through all rows of a matrix, for kernels
// without a sum along the row: a workgroup takes kSegment of them, so every
// lane has work whatever the row's length.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {
namespace mx {

constexpr int kThreads = 256, kPieces = 4;
constexpr int kSegment = kThreads * kPieces;  // eight-element pieces of one workgroup

// d pieces to a row.  n / d for n below 2^31 is one product and a shift: with
// 2^(s-1) < d <= 2^s and m = floor(2^(31+s) / d) + 1, it is floor(n m / 2^(31+s)).
struct Rows {
  uint32_t d, m, shift;  // shift = s - 1
  uint32_t pieces;       // of a chunk of rows (one per blockIdx.y), below 2^31
  int64_t rows;          // of a chunk
};
__device__ __forceinline__ uint32_t row_of(const Rows& r, uint32_t n) { return __umulhi(n, r.m) >> r.shift; }

// cols: a multiple of 8, at least 32
static inline Rows split_rows(int64_t rows, int64_t cols, dim3* grid) {
  Rows r;
  r.d = static_cast<uint32_t>(cols / 8);
  uint32_t s = 0;
  while ((uint64_t{1} << s) < r.d) ++s;
  r.shift = s - 1;  // d is at least 4
  r.m = static_cast<uint32_t>((uint64_t{1} << (31 + s)) / r.d + 1);
  const int64_t most = ((int64_t{1} << 31) - kSegment) / r.d;  // rows whose pieces stay below 2^31
  r.rows = rows < most ? rows : most;
  r.pieces = static_cast<uint32_t>(r.rows * r.d);
  *grid = dim3((r.pieces + kSegment - 1) / kSegment, static_cast<unsigned>((rows + r.rows - 1) / r.rows));
  return r;
}

}  // namespace mx
}  // namespace dg
