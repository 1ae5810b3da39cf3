// How the MX products are cut into workgroups.  Plain C++: the CPU tests
// compile it and go over sizes.
#pragma once
#include <stdint.h>

#if defined(__HIPCC__)
#define DG_MX_HD __host__ __device__
#else
#define DG_MX_HD
#endif

namespace dg {
namespace mx {

// Tiles of `size` that n rows or columns take; n up to 2^31 - 1, whose sum with
// a size does not fit 32 bits with a sign.
DG_MX_HD inline int32_t tile_count(int32_t n, int32_t size) {
  return static_cast<int32_t>((static_cast<uint32_t>(n) + static_cast<uint32_t>(size) - 1u) / static_cast<uint32_t>(size));
}

// A launch holds fewer than 2^32 threads along x: workgroups beyond kGridX go
// on along y, as workgroup y * kGridX + x; those past the last do nothing.
constexpr uint32_t kGridX = 1u << 21;  // of at most 1024 threads
inline uint32_t grid_x(int64_t workgroups) { return workgroups < kGridX ? static_cast<uint32_t>(workgroups) : kGridX; }
inline uint32_t grid_y(int64_t workgroups) { return static_cast<uint32_t>((workgroups + kGridX - 1) / kGridX); }

// Columns of a workgroup of the kernel for few rows: the columns' share of what
// makes row tiles x column tiles a multiple of the CUs, and never more than
// `most`, the 16 per column block that the workgroup computes (several row
// tiles that do not divide the CUs leave a share larger than that).
inline int rows_step(int64_t N, int64_t tiles, int most, int cus) {
  const int64_t per = static_cast<int64_t>(most) * cus, all = (N * tiles + per - 1) / per * cus / tiles;
  const int64_t even = all > 0 ? (N + all - 1) / all : most;
  return static_cast<int>(even < 4 ? 4 : (even > most ? most : even));
}

}  // namespace mx
}  // namespace dg
