// Which kernel an F8 product takes, and how its K is cut.  Plain C++: the CPU
// tests compile it and go over sizes.
#pragma once
#include <stdint.h>

namespace dg {

// K in at most `want` parts of equal multiples of 512 elements, the last of what is left.
inline int64_t f8_part(int64_t K, int64_t parts) { return (K + 512 * parts - 1) / (512 * parts) * 512; }
inline int f8_parts(int64_t K, int64_t want) {
  const int64_t each = f8_part(K, want);
  return static_cast<int>((K + each - 1) / each);
}

// Values of a row of the parts' sums.
inline int64_t f8_split_pitch(int64_t N) { return (N + 3) / 4 * 4; }

// Which kernel a product takes: for few rows (`rows` of 16, 32, 64 at a time), or tiles (rows = 0) of `size`, K in `parts`.
struct F8Choice {
  int rows, size, parts;
};

// (Times in us, bf16 out, operands in the last-level cache.)
//
// Up to 32 rows stream the weights.  From 33 to 64 rows, tiles of 64 x 128 take
// over where they occupy 3/8 of the CUs (rows / tiles: 64 x 8192 x 3584 13.8 /
// 14.1, 48 x 13312 x 16384 77 / 70, 64 x 13312 x 16384 82 / 71; 32 x 13312 x 16384
// 61 / 68).  Past one round they always do: all their rounds together are more than
// half full.
//
// Up to one 64 x 128 tile per CU, the least of three estimates: those tiles (5
// + 0.35 per slab of 128 elements; tiles of 128 x 128, of which half as many run,
// 22.1 against 15.6 at 256 x 8192 x 3584), the same with K in parts, as
// many as there are CUs for but of eight slabs at least (128 x 512 x 16384: 16
// parts 14.9, 32 17.9), and a second kernel that adds them (12 + 0.35 per slab of
// a part), and the kernel for few rows, 32 at a time (4.5 + 1.7 per 2048 elements and round of
// workgroups; 64 at a time 2.9).  Measured, rows / tiles / parts: 100 x 1024 x
// 4096 7.8 / 15 / 11, 128 x 512 x 16384 18 / 49 / 15, 256 x 2048 x 8192 22 / 27 /
// 17, 512 x 1024 x 16384 39 / 49 / 23, 1024 x 1024 x 4096 23 / 16 / 19 and x 16384
// 70 / 50 / 36.
//
// More tiles: of 256 x 256, which read the operands half as often, or of 128 x
// 128, which leave fewer CUs idle in the last round: a round of the larger ones
// takes as long as three of the smaller ones with one per CU.
inline F8Choice f8_choice(int64_t M, int64_t N, int64_t K, int cus) {
  auto tiles = [&](int64_t high, int64_t wide) { return (M + high - 1) / high * ((N + wide - 1) / wide); };
  auto rounds = [&](int64_t n) { return (n + cus - 1) / cus; };
  if (M <= 16) return {16, 0, 1};
  if (M <= 32) return {32, 0, 1};
  const int64_t low = tiles(64, 128);
  if (low <= cus) {
    const double slabs = static_cast<double>(K) / 128, wgs = static_cast<double>(tiles(32, 32)) / cus;
    const int64_t most = K / 1024 > 1 ? K / 1024 : 1;
    const int parts = f8_parts(K, cus / low < most ? cus / low : most);
    const double rows = M <= 64 ? 4.5 + 2.9 * slabs / 16 : 4.5 + 1.7 * slabs / 16 * (wgs > 0.8 ? 1.25 * wgs : 1.0);
    const double whole = 5 + 0.35 * slabs, split = 12 + 0.35 * static_cast<double>(f8_part(K, parts)) / 128;
    if (parts > 1 && split < whole && split < rows) return {0, 64, parts};
    if (M <= 64) return 8 * low >= 3 * cus ? F8Choice{0, 64, 1} : F8Choice{64, 0, 1};
    return rows < whole ? F8Choice{32, 0, 1} : F8Choice{0, 64, 1};
  }
  if (M <= 64) return {0, 64, 1};
  return {0, 3 * rounds(tiles(256, 256)) <= rounds(tiles(128, 128)) ? 256 : 128, 1};
}

inline int64_t f8_gemm_workspace(int64_t M, int64_t N, int64_t K, int cus) {
  const F8Choice c = f8_choice(M, N, K, cus);
  return c.parts > 1 ? c.parts * M * f8_split_pitch(N) * 4 : 0;
}

}  // namespace dg
