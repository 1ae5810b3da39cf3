// MX product for few rows of A (a decoding step, an expert with a few tokens).
//
// It has to read the weights once: N * K * 17/32 bytes, which bounds it.  So
// nothing of B goes through LDS: a wave owns 16 NB columns and streams their
// rows of B from memory straight into the registers of the MFMA that
// multiplies them, 16 x 16 x 128 with per-block scales
// (v_mfma_scale_f32_16x16x128_f8f6f4).  The first MFMA operand is B and the
// second A, so a lane ends with four neighbouring columns of one row of D.
//
// The workgroup's waves split K among them in chunks of 512 (a row's chunk of
// scales is one 16-byte load, its chunk of E2M1 codes 256 contiguous bytes,
// four loads per lane), and add their sums through LDS in a fixed order.
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
constexpr int kWaves = 8;

template <int MB, int NB, bool A8, bool kBf16>
__global__ __launch_bounds__(64 * kWaves) void mx_gemm_rows_kernel(MxGemmArgs a) {
  constexpr int kAL = A8 ? 8 : 4;  // 16-byte loads of a lane per chunk of a row of A
  __shared__ f32x4 sums[kWaves / 2][MB * NB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int32_t n_tiles = (a.N + 16 * NB - 1) / (16 * NB);
  const int32_t row_tile = static_cast<int32_t>(blockIdx.x) / n_tiles;
  GroupTile t;
  int64_t b_row = 0, bias0 = 0;
  if (a.offsets) {
    t = find_group_tile(a.offsets, a.groups, a.M, 16 * MB, row_tile);
    if (t.group < 0) return;
    b_row = bias0 = static_cast<int64_t>(t.group) * a.N;
  } else {
    t.row0 = row_tile * 16 * MB;
    t.rows = a.M - t.row0;
  }
  const int32_t rows = min(t.rows, 16 * MB);
  const int32_t n0 = (static_cast<int32_t>(blockIdx.x) - row_tile * n_tiles) * 16 * NB, cols = min(a.N - n0, 16 * NB);
  b_row += n0;
  const uint32_t b_bytes = static_cast<uint32_t>(a.K / 2), a_bytes = static_cast<uint32_t>(A8 ? a.K : a.K / 2);
  const uint32_t s_bytes = static_cast<uint32_t>(scale_pitch(a.K));
  const auto rB = make_rsrc(a.B + b_row * b_bytes, cols * b_bytes);
  const auto rBs = make_rsrc(a.Bs + b_row * s_bytes, cols * s_bytes);
  const auto rA = make_rsrc(a.A + static_cast<int64_t>(t.row0) * a_bytes, rows * a_bytes);
  const auto rAs = make_rsrc(a.As + static_cast<int64_t>(t.row0) * s_bytes, rows * s_bytes);
  uint32_t ob[NB], obs[NB], oa[MB], oas[MB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    ob[j] = static_cast<uint32_t>(16 * j + r) * b_bytes + 16 * q;
    obs[j] = static_cast<uint32_t>(16 * j + r) * s_bytes;
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    oa[i] = static_cast<uint32_t>(16 * i + r) * a_bytes + 16 * q;
    oas[i] = static_cast<uint32_t>(16 * i + r) * s_bytes;
  }

  f32x4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  const int chunks = (a.K + kChunk - 1) / kChunk;
  auto step = [&](int c, auto last) {
    constexpr bool kLast = decltype(last)::value;
    const int k0 = c * kChunk;
    i32x4 fb[NB][4], sb[NB], fa[MB][kAL], sa[MB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // past K: the piece of 32 elements would be the next row's
        const bool in = !kLast || k0 + 128 * u + 32 * q < a.K;
        fb[j][u] = load16(rB, in ? ob[j] + 64 * u : kOutOfRange, k0 / 2);
      }
      sb[j] = load16(rBs, obs[j], k0 / kMxBlock);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
#pragma unroll
      for (int u = 0; u < kAL; ++u) {
        const bool in = !kLast || (A8 ? k0 + 64 * u + 16 * q < a.K : k0 + 128 * u + 32 * q < a.K);
        fa[i][u] = load16(rA, in ? oa[i] + 64 * u : kOutOfRange, A8 ? k0 : k0 / 2);
      }
      sa[i] = load16(rAs, oas[i], k0 / kMxBlock);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      // a scale byte past K may hold anything, also the NaN scale
      const bool in = !kLast || k0 + 128 * u + 32 * q < a.K;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const i32x8 vb = {fb[j][u][0], fb[j][u][1], fb[j][u][2], fb[j][u][3], 0, 0, 0, 0};
        const int vsb = in ? static_cast<int>(static_cast<uint32_t>(sb[j][u]) >> (8 * q)) : 0;
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const int vsa = in ? static_cast<int>(static_cast<uint32_t>(sa[i][u]) >> (8 * q)) : 0;
          if constexpr (A8) {
            const i32x4 lo = fa[i][2 * u], hi = fa[i][2 * u + 1];
            const i32x8 va = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, acc[i][j], 4, 0, 0, vsb, 0, vsa);
          } else {
            const i32x8 va = {fa[i][u][0], fa[i][u][1], fa[i][u][2], fa[i][u][3], 0, 0, 0, 0};
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, acc[i][j], 4, 4, 0, vsb, 0, vsa);
          }
        }
      }
    }
  };
  const int whole = a.K / kChunk;
  for (int c = wave; c < whole; c += kWaves) step(c, std::false_type{});
  if (whole < chunks && whole % kWaves == wave) step(whole, std::true_type{});

  // sum over the waves, halving their number: fixed order
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
  const bool wide = wide_rows<kBf16>(a);
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

template <int MB, int NB>
static hipError_t rows_t(const MxGemmArgs& a, hipStream_t st) {
  const int64_t tiles = a.offsets ? most_group_tiles(a.M, a.groups, 16 * MB) : (a.M + 16 * MB - 1) / (16 * MB);
  const int64_t blocks = tiles * ((a.N + 16 * NB - 1) / (16 * NB));
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * kWaves);
  if (a.a_format == MX_E4M3) {
    if (a.out_bf16)
      hipLaunchKernelGGL((mx_gemm_rows_kernel<MB, NB, true, true>), grid, block, 0, st, a);
    else
      hipLaunchKernelGGL((mx_gemm_rows_kernel<MB, NB, true, false>), grid, block, 0, st, a);
  } else {
    if (a.out_bf16)
      hipLaunchKernelGGL((mx_gemm_rows_kernel<MB, NB, false, true>), grid, block, 0, st, a);
    else
      hipLaunchKernelGGL((mx_gemm_rows_kernel<MB, NB, false, false>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace mx

// Few rows stream the weights; from 65 rows on (of a group, on average), tiles.
hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t st) {
  if (a.M == 0) return hipSuccess;
  const int64_t rows = a.offsets ? a.M / a.groups : a.M;
  if (rows <= 16) return mx::rows_t<1, 1>(a, st);
  if (rows <= 32) return mx::rows_t<2, 2>(a, st);
  if (rows <= 64) return mx::rows_t<4, 2>(a, st);
  const int64_t tiles = ((rows + 255) / 256) * ((a.N + 255) / 256) * (a.offsets ? a.groups : 1);
  return launch_mx_gemm_tile(tiles >= 192 ? 256 : 128, a, st);
}

}  // namespace dg
