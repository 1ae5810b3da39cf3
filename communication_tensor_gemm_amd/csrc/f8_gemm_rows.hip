// F8 product for few rows of A (a decoding step).
//
// It has to read the weights once: N * K * 129/128 bytes, which bounds it.  So
// nothing of B goes through LDS: a wave streams rows of B from memory straight
// into the registers of the MFMA that multiplies them, 16 x 16 x 128 with
// per-block scales (v_mfma_scale_f32_16x16x128_f8f6f4).  The first MFMA
// operand is B and the second A, so a lane ends with four neighbouring columns
// of one row of D.  The workgroup's waves split K among them in chunks of 256
// and add their sums through LDS in a fixed order.
//
// Loads.  A vector load runs at 64 bytes a cycle where four neighbouring lanes
// read 64 consecutive bytes, and at one lane a cycle where each reads another
// row, as the MFMA's layout wants it.  So four neighbouring lanes read 64
// bytes of a row, each lane of four rows in turn, and the 4 x 4 pieces of 16
// bytes are transposed among the four lanes by DPP moves.  A lane then holds 64
// consecutive bytes of its row, which two MFMAs multiply.  Which elements of a
// block a lane has does not matter as long as A and B agree and the elements
// that the hardware scales together are of one block of 128: the two lower
// quarters of the wave hold the chunk's first block, the two upper ones its
// second, and quarter q passes the scale of block q % 2.
//
// A comes through LDS where its rows fit and K is long (kLds), copied once and densely;
// else from L2 where it is used, in the same way as B.
//
// 1 x 13312 x 16384 (220 MB): 38.5 us, 5.7 TB/s, launch and the latency of the
// first loads included (a copy: 6.2).  More rows of that width, whose A is read
// again by every workgroup: 4 43 us, 8 49, 16 52, 32 62; 1 x 8192 x 1024 4.2, 16 4.2.
#include "f8_common.h"
#include "mx_tiles.h"

namespace dg {
namespace f8 {

constexpr int kChunk = 256;  // elements of K per step of a wave
constexpr int kWaves = 8;
// bytes of A, its scales and their padding in LDS: three workgroups to a CU, or two
constexpr int kLdsA = 48 * 1024, kMoreLdsA = 78 * 1024;
constexpr int kPadA = 64, kPadS = 16;  // between rows: the 16 rows of a read on distinct banks

// LDS bytes of `rows` rows of A and their scales
__host__ __device__ inline int64_t lds_a_bytes(int64_t rows, int64_t K) {
  return rows * (K + kPadA + f8_scale_pitch(K) + kPadS);
}

// Transposes 4 x 4 pieces of 16 bytes within each four lanes: lane p's piece s
// becomes lane s's piece p.
__device__ __forceinline__ void transpose_quads(i32x4 (&v)[4], bool odd, bool high) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    int x[4] = {v[0][d], v[1][d], v[2][d], v[3][d]}, y[4];
#pragma unroll
    for (int t = 0; t < 4; t += 2) {
      const int from0 = __builtin_amdgcn_mov_dpp(x[t], 0xB1, 0xf, 0xf, true);  // of lane ^ 1
      const int from1 = __builtin_amdgcn_mov_dpp(x[t + 1], 0xB1, 0xf, 0xf, true);
      y[t] = odd ? from1 : x[t];
      y[t + 1] = odd ? x[t + 1] : from0;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int from0 = __builtin_amdgcn_mov_dpp(y[t], 0x4E, 0xf, 0xf, true);  // of lane ^ 2
      const int from2 = __builtin_amdgcn_mov_dpp(y[t + 2], 0x4E, 0xf, 0xf, true);
      v[t][d] = high ? from2 : y[t];
      v[t + 2][d] = high ? y[t + 2] : from0;
    }
  }
}

// kLdsBytes: of A in LDS; 0: A from memory
template <int MB, int NB, bool kBf16, int kLdsBytes>
__global__ __launch_bounds__(64 * kWaves) void f8_gemm_rows_kernel(MxGemmArgs a, int step) {  // step: columns of a workgroup
  constexpr bool kLds = kLdsBytes > 0;
  constexpr int kAhead = NB == 1 ? 2 : 1;  // chunks asked for before they are multiplied
  constexpr int kSums = kWaves / 2 * MB * NB * 64 * 16;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLdsBytes > kSums ? kLdsBytes : kSums];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int32_t n_tiles = tile_count(a.N, step);
  const uint32_t block = blockIdx.y * kGridX + blockIdx.x;
  const int32_t row_tile = static_cast<int32_t>(block / static_cast<uint32_t>(n_tiles));
  const int32_t row0 = row_tile * 16 * MB;
  if (row0 >= a.M) return;
  const int32_t rows = min(a.M - row0, 16 * MB);
  const int32_t n0 = static_cast<int32_t>(block - static_cast<uint32_t>(row_tile) * static_cast<uint32_t>(n_tiles)) * step;
  const int32_t cols = min(a.N - n0, step);
  const uint32_t k_bytes = static_cast<uint32_t>(a.K), s_bytes = static_cast<uint32_t>(f8_scale_pitch(a.K));
  const auto rB = make_rsrc(a.B + static_cast<int64_t>(n0) * k_bytes, cols * k_bytes);
  const auto rBs = make_rsrc(a.Bs + static_cast<int64_t>(n0) * s_bytes, cols * s_bytes);
  const auto rA = make_rsrc(a.A + static_cast<int64_t>(row0) * k_bytes, rows * k_bytes);
  const auto rAs = make_rsrc(a.As + static_cast<int64_t>(row0) * s_bytes, rows * s_bytes);
  // Loads: four neighbouring lanes have 64 consecutive bytes of a row, lane l in
  // load t those of row 4 (r / 4) + t from 64 q + 16 (l % 4) on
  const int p = lane & 3, row4 = r & 12;
  const bool odd = lane & 1, high = lane & 2;
  struct Chunk {
    i32x4 b[NB][4];
    int s[NB];
  };
  const int chunks = (a.K + kChunk - 1) / kChunk;
  // chunk c of B: past K (a second block, or all of a chunk) zeros; every load
  // is issued, whatever lies past K, for the wait below counts them
  auto load_b = [&](int c, Chunk& f) {
    const int k0 = c * kChunk;
    const uint32_t past = k0 + 64 * q < a.K ? 0u : kOutOfRange, s_past = k0 + 128 * (q & 1) < a.K ? 0u : kOutOfRange;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        f.b[j][t] = load16(rB, ((16 * j + row4 + t) * k_bytes + 64 * q + 16 * p) | past, k0);
      f.s[j] = __builtin_amdgcn_raw_buffer_load_b8(rBs, ((16 * j + r) * s_bytes + (q & 1)) | s_past, k0 / kF8Block, 0);
    }
  };

  // A: into LDS by rows, or (kLds false) from memory where it is used
  const uint32_t pa = k_bytes + kPadA, ps = s_bytes + kPadS;
  uint8_t* const lds_s = lds + rows * pa;
  if constexpr (kLds) {
    typedef __attribute__((address_space(3))) void* lds_ptr_t;
    const int pieces = (k_bytes + 1023) / 1024, all = rows * pieces;
    for (int i = wave; i < all; i += kWaves) {
      const int row = i / pieces, at = (i - row * pieces) * 1024;
      if (at + 16 * lane < static_cast<int>(k_bytes))  // the lanes past the row's end are off
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_ptr_t)(lds + row * pa + at), 16, row * k_bytes + at + 16 * lane, 0, 0, 0);
    }
    const int s_pieces = (s_bytes + 1023) / 1024, s_all = rows * s_pieces;
    for (int i = wave; i < s_all; i += kWaves) {
      const int row = i / s_pieces, at = (i - row * s_pieces) * 1024;
      if (at + 16 * lane < static_cast<int>(s_bytes))
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rAs, (lds_ptr_t)(lds_s + row * ps + at), 16, row * s_bytes + at + 16 * lane, 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);  // A's loads before B's, which are not waited for below
  }
  Chunk f[kAhead];
#pragma unroll
  for (int v = 0; v < kAhead; ++v) load_b(wave + v * kWaves, f[v]);
  if constexpr (kLds) {
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<kAhead * NB * 5>();
    barrier_only();
  }

  f32x4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  auto multiply = [&](int c, Chunk& f) {
    const int k0 = c * kChunk;
    if (k0 >= a.K) return;
    const bool in = k0 + 64 * q < a.K, s_in = k0 + 128 * (q & 1) < a.K;
    i32x4 fa[MB][4];
    int sa[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      if constexpr (kLds) {
        const uint32_t row = min(16 * i + r, rows - 1);  // without a row: the last one, not stored
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          // past K lies the padding or another row: not to be multiplied, not even by zero
          const i32x4 v = *reinterpret_cast<const i32x4*>(lds + row * pa + (in ? k0 + 64 * q + 16 * s : 0));
          fa[i][s] = in ? v : i32x4{0, 0, 0, 0};
        }
        const int v = lds_s[row * ps + (s_in ? k0 / kF8Block + (q & 1) : 0)];
        sa[i] = s_in ? v : 0;
      } else {
        const uint32_t past = in ? 0u : kOutOfRange, s_past = s_in ? 0u : kOutOfRange;
#pragma unroll
        for (int t = 0; t < 4; ++t) fa[i][t] = load16(rA, ((16 * i + row4 + t) * k_bytes + 64 * q + 16 * p) | past, k0);
        sa[i] = __builtin_amdgcn_raw_buffer_load_b8(rAs, ((16 * i + r) * s_bytes + (q & 1)) | s_past, k0 / kF8Block, 0);
      }
    }
    if constexpr (!kLds) {
#pragma unroll
      for (int i = 0; i < MB; ++i) transpose_quads(fa[i], odd, high);
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) transpose_quads(f.b[j], odd, high);
#pragma unroll
    for (int s = 0; s < 4; s += 2)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const i32x4 b0 = f.b[j][s], b1 = f.b[j][s + 1];
        const i32x8 vb = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const i32x4 a0 = fa[i][s], a1 = fa[i][s + 1];
          const i32x8 va = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, acc[i][j], 0, 0, 0, f.s[j], 0, sa[i]);
        }
      }
  };
  for (int c = wave; c < chunks; c += kAhead * kWaves) {
#pragma unroll
    for (int v = 0; v < kAhead; ++v) {
      multiply(c + v * kWaves, f[v]);
      __builtin_amdgcn_sched_barrier(0);  // the next loads' registers are not live above
      load_b(c + (kAhead + v) * kWaves, f[v]);
    }
  }

  // sum over the waves, halving their number: fixed order
  f32x4(*const sums)[MB * NB][64] = reinterpret_cast<f32x4(*)[MB * NB][64]>(lds);
  if constexpr (kLds) __syncthreads();  // every wave is done with A
#pragma unroll
  for (int n = kWaves / 2; n > 0; n >>= 1) {
    if (wave >= n && wave < 2 * n) {
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) sums[wave - n][i * NB + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave < n) {
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] += sums[wave][i * NB + j][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
  const bool wide = wide_rows<kBf16>(a) && n0 % 4 == 0;
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    if (16 * i + r >= rows) continue;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int32_t c = 16 * j + 4 * q;
      if (c < cols) store_four<kBf16>(a, 0, row0 + 16 * i + r, n0 + c, cols - c, wide, acc[i][j]);
    }
  }
}

template <int MB, int NB, int kLdsBytes>
static hipError_t rows_lds_t(const MxGemmArgs& a, hipStream_t st) {
  const int64_t tiles = tile_count(a.M, 16 * MB);
  const int step = rows_step(a.N, tiles, 16 * NB, a.cus);
  const int64_t blocks = tiles * tile_count(a.N, step);
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  const dim3 grid(grid_x(blocks), grid_y(blocks)), block(64 * kWaves);
  if (a.out_bf16)
    hipLaunchKernelGGL((f8_gemm_rows_kernel<MB, NB, true, kLdsBytes>), grid, block, 0, st, a, step);
  else
    hipLaunchKernelGGL((f8_gemm_rows_kernel<MB, NB, false, kLdsBytes>), grid, block, 0, st, a, step);
  return hipGetLastError();
}

// 32 columns to a workgroup, for half the reads of A; but up to 16 rows with more
// than a chunk of K to each wave have A in LDS where it fits, and then 16 columns,
// in two chunks ahead (with / without: 1 x 8192 x 4096 9.1 us / 11.4, 8 x 8192 x
// 3584 9.1 / 9.4; 1 x 8192 x 2048 6.6 / 6.4, 16 x 8192 x 1024 5.6 / 4.2, 32 x 8192 x
// 1024 7.2 / 5.2).  A long K is worth more LDS at two workgroups per CU instead of
// three: 4 x 13312 x 16384 48 -> 42 us, 8 x 8192 x 8192 19 -> 14; a shorter one not
// (16 x 13312 x 4608 15 and 17).
template <int MB>
static hipError_t rows_t(const MxGemmArgs& a, hipStream_t st) {
  if constexpr (MB == 1) {
    const int64_t bytes = lds_a_bytes(a.M < 16 ? a.M : 16, a.K);
    if (bytes <= kLdsA && a.K > kChunk * kWaves) return rows_lds_t<1, 1, kLdsA>(a, st);
    if (bytes <= kMoreLdsA && a.K >= 8192) return rows_lds_t<1, 1, kMoreLdsA>(a, st);
  }
  return rows_lds_t<MB, 2, 0>(a, st);
}

}  // namespace f8

hipError_t launch_f8_gemm(const MxGemmArgs& a, float* work, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  const F8Choice c = f8_choice(a.M, a.N, a.K, a.cus);
  if (c.rows == 16) return f8::rows_t<1>(a, st);
  if (c.rows == 32) return f8::rows_t<2>(a, st);
  if (c.rows == 64) return f8::rows_t<4>(a, st);
  if (c.parts > 1) return launch_f8_gemm_split(a, c.parts, work, f8_split_pitch(a.N), st);
  return launch_f8_gemm_tile(c.size, a, st);
}

}  // namespace dg
