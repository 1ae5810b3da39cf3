// MX product for few rows of A (a decoding step, an expert with a few tokens).
//
// It has to read the weights once: N * K * 17/32 bytes, which bounds it.  So
// nothing of B goes through LDS: a wave streams rows of B from memory straight
// into the registers of the MFMA that multiplies them, 16 x 16 x 128 with
// per-block scales (v_mfma_scale_f32_16x16x128_f8f6f4).  The first MFMA
// operand is B and the second A, so a lane ends with four neighbouring columns
// of one row of D.  The workgroup's waves split K among them in chunks of
// 512 and add their sums through LDS in a fixed order.
//
// Loads.  A vector load runs at 64 bytes a cycle where four neighbouring lanes
// read 64 consecutive bytes, and at one lane (16 bytes) a cycle where each
// reads another row, as the MFMA's layout wants it.  With loads in that layout
// the product was bound by them: 34 us for one row of E4M3 by 13312 x 16384, 60
// for 16 rows, 95 for 64.  So four neighbouring lanes read 64 bytes of a row,
// each lane of four rows in turn, and the 4 x 4 pieces are transposed among
// the four lanes by DPP moves (32 to 64 VALU instructions per chunk); the four
// MFMAs of a chunk then multiply blocks 4 q + s of a row (q = l / 16, s = 0 ..
// 3) where they would have multiplied blocks 4 s + q, and a lane's four scales
// are one dword.  34 -> 23 us, 60 -> 29, 95 -> 54.
//
// A comes through LDS where its rows fit there (kLds), copied once and densely;
// else from L2 where it is used, in the same way as B.
//
// Columns.  A workgroup takes at most 16 NB columns, and as many fewer as make
// the workgroups a multiple of the CUs: 13312 columns are 1024 times 13 rather
// than 832 times 16, of which some CUs would have four and some three (27.2 ->
// 24.0 us).
//
// At 1 x 13312 x 16384 (116 MB) it reads 5.2 TB/s, launch and the latency of
// the first loads included (5.6 with E2M1 rows); a plain read of such a tensor
// reaches 6.2.  More rows of that width, whose A is read again by every
// workgroup (E4M3 / E2M1, us): 2 23, 4 and 8 26, 16 29 / 26, 32 38 / 30, 64
// 54 / 42.
//
// Operand layout of the MFMA (k within its 128): lane l has row l % 16 of its
// operand; an E2M1 operand's lane holds the 32 elements of block l / 16; an
// E4M3 operand's lane holds elements 16 (l / 16) .. + 15 in its first four
// registers and 64 + 16 (l / 16) .. + 15 in the last four.  The scale byte
// that a lane passes is that of block l / 16 of its row, in both cases.
#include "mx_tiles.h"

namespace dg {
namespace mx {

constexpr int kChunk = 512;  // elements of K per step of a wave
constexpr int kLdsA = 48 * 1024;      // bytes of A, its scales and their padding in LDS
constexpr int kPadA = 64, kPadS = 16;  // between rows: the 16 rows of a read on distinct banks

// LDS bytes of `rows` rows of A and their scales
__host__ __device__ inline int64_t lds_a_bytes(int64_t rows, int64_t K, int a_format) {
  return rows * (mx_row_bytes(K, a_format) + kPadA + scale_pitch(K) + kPadS);
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

template <int MB, int NB, bool A8, bool kBf16, bool kLds, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void mx_gemm_rows_kernel(MxGemmArgs a, int step) {  // step: columns of a workgroup
  constexpr int kAL = A8 ? 8 : 4;  // 16-byte pieces of a lane per chunk of a row of A
  constexpr int kAhead = NB == 1 ? 2 : 1;  // chunks asked for before they are multiplied (twice as many: no faster)
  constexpr int kSums = kWaves / 2 * MB * NB * 64 * 16;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds && kLdsA > kSums ? kLdsA : kSums];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int32_t n_tiles = tile_count(a.N, step);
  const uint32_t block = blockIdx.y * kGridX + blockIdx.x;
  const int32_t row_tile = static_cast<int32_t>(block / static_cast<uint32_t>(n_tiles));
  GroupTile t;
  int64_t b_row = 0, bias0 = 0;
  if (a.offsets) {
    t = find_group_tile(a.offsets, a.groups, a.M, 16 * MB, row_tile);
    if (t.group < 0) return;
    b_row = bias0 = static_cast<int64_t>(t.group) * a.N;
  } else {
    t.row0 = row_tile * 16 * MB;
    t.rows = a.M - t.row0;
    if (t.rows <= 0) return;
  }
  const int32_t rows = min(t.rows, 16 * MB);
  const int32_t n_tile = static_cast<int32_t>(block - static_cast<uint32_t>(row_tile) * static_cast<uint32_t>(n_tiles));
  const int32_t n0 = n_tile * step, cols = min(a.N - n0, step);
  b_row += n0;
  const uint32_t b_bytes = static_cast<uint32_t>(a.K / 2), a_bytes = static_cast<uint32_t>(A8 ? a.K : a.K / 2);
  const uint32_t s_bytes = static_cast<uint32_t>(scale_pitch(a.K));
  const auto rB = make_rsrc(a.B + b_row * b_bytes, cols * b_bytes);
  const auto rBs = make_rsrc(a.Bs + b_row * s_bytes, cols * s_bytes);
  const auto rA = make_rsrc(a.A + static_cast<int64_t>(t.row0) * a_bytes, rows * a_bytes);
  const auto rAs = make_rsrc(a.As + static_cast<int64_t>(t.row0) * s_bytes, rows * s_bytes);
  // Loads: four neighbouring lanes have 64 consecutive bytes of a row, lane l in
  // load t those of row 4 (r / 4) + t and block 4 q + l % 4
  const int p = lane & 3, row4 = r & 12;
  const bool odd = lane & 1, high = lane & 2;
  const int from = 4 * (4 * r + q);  // scales: lane 4 r + q loads what lane 16 q + r needs
  struct Chunk {
    i32x4 b[NB][4];
    int s[NB];
  };
  const int chunks = (a.K + kChunk - 1) / kChunk;
  // kLds: every load is issued, whatever lies past K, for the wait below counts
  // them; else the compiler may skip a wave's loads that are all past K
  auto masked = [&](bool in, uint32_t at) { return kLds ? at | (in ? 0u : kOutOfRange) : in ? at : kOutOfRange; };
  // chunk c of B: blocks past K (and all of a chunk past it) as zeros
  auto load_b = [&](int c, Chunk& f) {
    const int k0 = c * kChunk;
    const bool in = k0 + 32 * (4 * q + p) < a.K;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        f.b[j][t] = load16(rB, masked(in, (16 * j + row4 + t) * b_bytes + 64 * q + 16 * p), k0 / 2);
      f.s[j] = __builtin_amdgcn_raw_buffer_load_b32(rBs, masked(k0 < a.K, (16 * j + lane / 4) * s_bytes + 4 * p), k0 / kMxBlock, 0);
    }
  };

  // A: into LDS by rows, or (kLds false) from memory where it is used
  const uint32_t pa = a_bytes + kPadA, ps = s_bytes + kPadS;
  uint8_t* const lds_s = lds + rows * pa;
  if constexpr (kLds) {
    typedef __attribute__((address_space(3))) void* lds_ptr_t;
    const int pieces = (a_bytes + 1023) / 1024, all = rows * pieces;
    for (int i = wave; i < all; i += kWaves) {
      const int row = i / pieces, at = (i - row * pieces) * 1024;
      if (at + 16 * lane < static_cast<int>(a_bytes))  // the lanes past the row's end are off
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_ptr_t)(lds + row * pa + at), 16, row * a_bytes + at + 16 * lane, 0, 0, 0);
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
    // the blocks of the four MFMAs: 4 q + s in E2M1; in E4M3, whose lanes hold
    // halves of two blocks, halves q % 2 of 4 (q / 2) + s and 8 + 4 (q / 2) + s
    i32x4 fa[MB][kAL / 4][4];
    int sa[MB];
    auto block_of = [&](int h, int s) { return A8 ? 8 * h + 4 * (q >> 1) + s : 4 * q + s; };
    auto byte_of = [&](int h, int s) { return A8 ? 32 * block_of(h, s) + 16 * (q & 1) : 16 * block_of(h, s); };
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      if constexpr (kLds) {
        const uint32_t row = min(16 * i + r, rows - 1);  // without a row: the last one, not stored
#pragma unroll
        for (int h = 0; h < kAL / 4; ++h)
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            // past K lies the padding or another row: not to be multiplied, not even by zero
            const bool in = k0 + 32 * block_of(h, s) < a.K;
            const i32x4 v = *reinterpret_cast<const i32x4*>(lds + row * pa + (in ? (A8 ? k0 : k0 / 2) + byte_of(h, s) : 0));
            fa[i][h][s] = in ? v : i32x4{0, 0, 0, 0};
          }
        sa[i] = *reinterpret_cast<const int*>(lds_s + row * ps + k0 / kMxBlock + 4 * q);
      } else {
#pragma unroll
        for (int h = 0; h < kAL / 4; ++h) {
          const bool in = k0 + 32 * block_of(h, p) < a.K;
#pragma unroll
          for (int t = 0; t < 4; ++t)
            fa[i][h][t] = load16(rA, in ? (16 * i + row4 + t) * a_bytes + byte_of(h, p) : kOutOfRange, A8 ? k0 : k0 / 2);
        }
        sa[i] = __builtin_amdgcn_raw_buffer_load_b32(rAs, (16 * i + lane / 4) * s_bytes + 4 * p, k0 / kMxBlock, 0);
      }
    }
    if constexpr (!kLds) {
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        sa[i] = __builtin_amdgcn_ds_bpermute(from, sa[i]);
#pragma unroll
        for (int h = 0; h < kAL / 4; ++h) transpose_quads(fa[i][h], odd, high);
      }
    }
    // a scale byte past K may hold anything, also the NaN scale
    const int left = min(max((static_cast<int>(a.K) - k0) / kMxBlock - 4 * q, 0), 4);
    const int keep = left == 4 ? -1 : (1 << (8 * left)) - 1;
    int sb[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      sb[j] = __builtin_amdgcn_ds_bpermute(from, f.s[j]) & keep;
      transpose_quads(f.b[j], odd, high);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) sa[i] &= keep;
#define DG_STEP(S)                                                                                                              \
  _Pragma("unroll") for (int j = 0; j < NB; ++j) {                                                                              \
    const i32x8 vb = {f.b[j][S][0], f.b[j][S][1], f.b[j][S][2], f.b[j][S][3], 0, 0, 0, 0};                                      \
    _Pragma("unroll") for (int i = 0; i < MB; ++i) {                                                                            \
      const i32x4 lo = fa[i][0][S];                                                                                             \
      if constexpr (A8) {                                                                                                       \
        const i32x4 hi = fa[i][kAL / 4 - 1][S];                                                                                 \
        const i32x8 va = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};                                              \
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, acc[i][j], 4, 0, S, sb[j], S, sa[i]);              \
      } else {                                                                                                                  \
        const i32x8 va = {lo[0], lo[1], lo[2], lo[3], 0, 0, 0, 0};                                                              \
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, acc[i][j], 4, 4, S, sb[j], S, sa[i]);              \
      }                                                                                                                         \
    }                                                                                                                           \
  }
    DG_STEP(0)
    DG_STEP(1)
    DG_STEP(2)
    DG_STEP(3)
#undef DG_STEP
  };
  for (int c = wave; c < chunks; c += kAhead * kWaves) {
#pragma unroll
    for (int v = 0; v < kAhead; ++v) {
      multiply(c + v * kWaves, f[v]);
      __builtin_amdgcn_sched_barrier(0);  // the next loads' registers are not live above (spills: 54 -> 93 us at 64 rows)
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
      if (c < cols)
        store_four<kBf16>(a, bias0, t.row0 + 16 * i + r, n0 + c, cols - c, wide, acc[i][j]);
    }
  }
}

template <int MB, int NB, bool kLds, int kWaves>
static hipError_t rows_waves_t(const MxGemmArgs& a, hipStream_t st) {
  const int64_t tiles = a.offsets ? most_group_tiles(a.M, a.groups, 16 * MB) : tile_count(a.M, 16 * MB);
  const int step = a.offsets ? 16 * NB : rows_step(a.N, tiles, 16 * NB, a.cus);
  const int64_t blocks = tiles * tile_count(a.N, step);
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  const dim3 grid(grid_x(blocks), grid_y(blocks)), block(64 * kWaves);
  if (a.a_format == MX_E4M3) {
    if (a.out_bf16)
      hipLaunchKernelGGL((mx_gemm_rows_kernel<MB, NB, true, true, kLds, kWaves>), grid, block, 0, st, a, step);
    else
      hipLaunchKernelGGL((mx_gemm_rows_kernel<MB, NB, true, false, kLds, kWaves>), grid, block, 0, st, a, step);
  } else {
    if (a.out_bf16)
      hipLaunchKernelGGL((mx_gemm_rows_kernel<MB, NB, false, true, kLds, kWaves>), grid, block, 0, st, a, step);
    else
      hipLaunchKernelGGL((mx_gemm_rows_kernel<MB, NB, false, false, kLds, kWaves>), grid, block, 0, st, a, step);
  }
  return hipGetLastError();
}

// Eight waves to a workgroup; four where there are many workgroups of few
// chunks each, so that more of them are under way at once (by group, 64 rows, 32
// x 2048 x K, four / eight, us: K = 1024 E2M1 15.6 / 18.1, E4M3 16.4 / 24.2;
// 4096 24.0 / 26.4, 23.6 / 25.8; 8192 39.0 / 38.8, 42.5 / 42.0; dense at 8192 x
// 8192 and one row eight take 9.5 us, four 11.3).
template <int MB, int NB, bool kLds>
static hipError_t rows_lds_t(const MxGemmArgs& a, hipStream_t st) {
  return a.offsets && a.K <= 8 * kChunk ? rows_waves_t<MB, NB, kLds, 4>(a, st) : rows_waves_t<MB, NB, kLds, 8>(a, st);
}

// Rows that fit into LDS leave a wave little else to load than B: 16 columns,
// in two chunks ahead (1 x 13312 x 16384: E4M3 23.7 us, with 32 columns 26.8,
// E2M1 21.9 and 24.7; 1 x 8192 x 3584 6.7 and 7.1, 6.4 and 6.7).  More of them: 32
// columns, for half the reads of A (16 rows: 28.8 us, with 16 columns 35.5; 64
// rows: 54 and 82).  A short K is not told apart, and there the first form loses
// (4 x 8192 x 4096 7.3 against 7.2, 16 x 8192 x 1024 5.9 against 4.5).
template <int MB>
static hipError_t rows_t(const MxGemmArgs& a, hipStream_t st) {
  // of a group: as many rows as a tile can have
  const int64_t rows = a.M < 16 * MB ? a.M : 16 * MB;
  if (lds_a_bytes(rows, a.K, a.a_format) <= kLdsA) return rows_lds_t<MB, 1, true>(a, st);
  return rows_lds_t<MB, 2, false>(a, st);
}

}  // namespace mx

// (Times in us, E2M1 then E4M3, operands from memory.)
//
// Few rows stream the weights; from 65 rows on (of a group, on average), tiles,
// where two passes of 64 rows read all weights twice (tiles / two passes: 65 x
// 13312 x 16384 56 / 64, 64 / 90; 128 rows 60 / 71, 74 / 102; 65 x 8192 x 3584 13.2
// / 13.5, 17.1 / 19.5).  For groups that bound is too high: 16 x 4096 x 4096 takes
// 45 / 55 here with 512 rows (35 / 41 on tiles of 128) and 71 / 134 with 1024 (50 /
// 56), whether evenly spread or half of them in one group.
//
// Few tiles would leave most CUs idle: then 32 rows at a time here, K split over
// a workgroup's waves (this / tiles of 128: 126 x 113 x 15168 11 / 51, 14 / 62;
// 128 x 512 x 1024 4.8 / 6.6, 5.3 / 8.0; 512 x 1024 x 3584 8.4 / 12.6, 12.4 / 17.3;
// 512 x 2048, 64 tiles: K = 3584 14.5 / 13.8, 20.6 / 17.7, K = 15168 36 / 50, 53 / 63).
//
// Tiles of 256 x 256 read the operands half as often, tiles of 128 x 128 leave
// fewer CUs idle in the last round.  A round of the larger ones takes as long
// as three of the smaller ones with one per CU (M x 8192 x 4096, larger /
// smaller: M = 1024 34 / 27, 50 / 37; 1536 37 / 39, 52 / 52; 2048 41 / 47, 58 / 69;
// 2304 63 / 57, 95 / 79; 4096 75 / 93, 109 / 134; 1024 x 13312 x 16384 122 / 168,
// 177 / 234; 2048 x 4096 x 1024 15.6 / 13.1, 20 / 16).  A group's last tile is taken
// as half full.
hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  const int64_t rows = a.offsets ? a.M / a.groups : a.M;
  if (rows <= 16) return mx::rows_t<1>(a, st);
  if (rows <= 32) return mx::rows_t<2>(a, st);
  if (rows <= 64) return mx::rows_t<4>(a, st);
  auto tiles = [&](int64_t size) {
    const int64_t row_tiles = a.offsets ? a.M / size + (a.groups + 1) / 2 : (a.M + size - 1) / size;
    return row_tiles * ((a.N + size - 1) / size);
  };
  auto rounds = [&](int64_t size) { return (tiles(size) + a.cus - 1) / a.cus; };
  if (tiles(128) <= a.cus / 8 || (tiles(128) <= a.cus / 4 && a.K > 4096)) return mx::rows_lds_t<2, 2, false>(a, st);
  return launch_mx_gemm_tile(3 * rounds(256) <= rounds(128) ? 256 : 128, a, st);
}

}  // namespace dg
