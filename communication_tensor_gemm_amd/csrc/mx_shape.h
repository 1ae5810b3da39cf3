// How the MX products are cut into workgroups.  Plain C++: the CPU tests
// compile it and go over sizes.
#pragma once
#include <stdint.h>

namespace dg {
namespace mx {

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
