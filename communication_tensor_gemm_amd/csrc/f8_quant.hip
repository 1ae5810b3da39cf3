// Quantisation of a matrix to an F8 tensor, by rows and transposed, the
// transposition of an F8 tensor, and back to plain values.
//
// Per block of 128: X = the least integer with max |x| <= 448 * 2^X, code =
// round(x * 2^-X) to nearest even (f8_common.h, block_byte).  All forms are
// bound by memory: 1, 2 or 4 bytes in and 1.01 out per element and output.
//
// By rows only: a thread takes eight elements, a block is 16 adjacent lanes (a
// DPP row), which exchange their maximum; four such pieces per thread are
// loaded before the first is used.
//
// Transposed too: a workgroup has a square of 128 x 128, thread t columns 8 (t
// % 16) .. + 7 of rows 8 (t / 16) .. + 7: 16 lanes read one row's 128 columns,
// a row's maximum is a DPP row's, a column's one over the thread's eight rows,
// the wave's four groups of lanes and, through LDS, the four waves.  The
// eight codes of a column's eight rows are packed in the thread's registers
// (no transposition of bytes), go through LDS, swizzled, and leave as whole
// lines of 128 bytes.
//
// 8192 x 13312 bf16 by rows 55 us, 6.0 TB/s (a copy: 6.2), transposed 60, both
// 87, 5.0 TB/s; fp32 by rows 98, both 138; back to bf16 56, to fp32 116.  Transposing 8192 x 16384 52 us,
// 5.2 TB/s (8192 x 13312 45 us, 4.9): 128-byte pieces of rows on both sides, and
// single bytes of the scales' lines (without those bytes 4 less).  777 x 3584 by rows 4.1 us, transposed 5.1: a launch's latency.
#include "f8_common.h"
#include "piece_rows.h"

namespace dg {
namespace f8 {

constexpr int PT_F8 = 2;  // source of the square kernel: an F8 tensor

template <int T, int A>
__global__ __launch_bounds__(kThreads) void f8_rows_kernel(F8QuantizeArgs a, Rows rows) {
  const int64_t pitch = f8_pitch(a.cols), spitch = f8_scale_pitch(a.cols);
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * rows.rows;
  const int64_t left = (a.rows - row0) * rows.d;
  const uint32_t pieces = left < rows.pieces ? static_cast<uint32_t>(left) : rows.pieces;
  const uint32_t first = blockIdx.x * kSegment + threadIdx.x;
  Raw8<T> raw[kPieces];
  int64_t row[kPieces];
  int32_t col[kPieces];
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const uint32_t i = first + c * kThreads;
    raw[c].zero();
    if (i < pieces) {
      const uint32_t r = row_of(rows, i);
      row[c] = row0 + r;
      col[c] = static_cast<int32_t>(i - r * rows.d);
      const int64_t at = 8 * static_cast<int64_t>(col[c]);
      if (at < a.cols) raw[c].template load<A>(a.x, row[c] * a.ldx + at, static_cast<int>(min(a.cols - at, int64_t{8})));
    }
  }
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    // the pieces of a block are 16 adjacent lanes: all of them are in or none is
    if (first + c * kThreads >= pieces) continue;
    if constexpr (T == PT_BF16) {
      uint32_t m2 = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) m2 = max_pair(m2, raw[c].w[j] & 0x7fff7fffu);
      const uint32_t byte = block_byte(row16_max(max(m2 << 16, m2 & 0xffff0000u)));
      u32x2 w = pack8_bf16(raw[c].w, block_factor(byte));
      if (byte == 255u) w = u32x2{0, 0};
      store_wide<A>(reinterpret_cast<u32x2*>(a.codes + row[c] * pitch + 8 * static_cast<int64_t>(col[c])), w);
      if ((col[c] & 15) == 0) a.scales[row[c] * spitch + (col[c] >> 4)] = static_cast<uint8_t>(byte);
    } else {
      float v[8];
      raw[c].get(v);
      store_block8<A>(v, a.codes, row[c] * pitch, col[c], a.scales, row[c] * spitch);
    }
  }
  // the scale bytes past the last block, by the first lane of the row's last block
  const int32_t blocks = static_cast<int32_t>(pitch / kF8Block), pad = static_cast<int32_t>(spitch) - blocks;
  if (pad > 0) {
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
      if (first + c * kThreads < pieces && col[c] == 16 * blocks - 16)
        for (int32_t k = 0; k < pad; ++k) a.scales[row[c] * spitch + blocks + k] = 0;
  }
}

// Eight consecutive elements of a row of the square, as loaded.
template <int SRC>
struct Piece {
  Raw8<SRC> raw;
  // elements 4 h .. + 3 of the eight
  __device__ __forceinline__ void four(int h, float (&v)[4]) const {
    float f[8];
    raw.get(f);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = f[4 * h + j];
  }
};
template <>
struct Piece<PT_F8> {
  u32x2 w;
  uint32_t byte;
  __device__ __forceinline__ void four(int h, float (&v)[4]) const {
    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], block_factor(byte), false);
    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], block_factor(byte), true);
    v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
  }
};

// Lane P of each 16 in all of them.
template <int P>
__device__ __forceinline__ uint32_t row16_lane(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x150 + P, 0xf, 0xf, true));
}

// The squares' order (8 bands: transpose 8192 x 16384 58.5 us, 1 band 68, 2 61, 4 59,
// 16 61, 32 65): workgroup b runs on XCD b mod 8 and takes place b / 8 of
// that XCD's contiguous share; the order goes down kBands bands of rows, then
// one square to the right, so that the bytes of a line of scales (one per square,
// of either tensor) meet in one L2.  Each group of bands starts at a column of
// its own: where rows are a power of two apart, XCDs at the same columns of
// different rows would share the memory's channels (transpose 8192 x 16384 59 us, so
// 54; 8192 x 16384 bf16 both ways 126 and 105; 8192 x 13312 85 and 87).
constexpr uint32_t kXcds = 8, kBands = 8;
struct Squares {
  uint32_t bands, across;
};
__device__ __forceinline__ bool square_of(const Squares& q, uint32_t block, uint32_t& band, uint32_t& kb) {
  const uint32_t n = q.bands * q.across, x = block % kXcds, i = block / kXcds, each = n / kXcds, more = n % kXcds;
  if (i >= each + (x < more ? 1u : 0u)) return false;
  const uint32_t w = x * each + min(x, more) + i, group = w / (kBands * q.across), in = w - group * kBands * q.across;
  const uint32_t high = min(kBands, q.bands - group * kBands);
  band = group * kBands + in % high;
  const uint32_t from = ((group * 0x9E3779B1u >> 16) * q.across) >> 16;  // (across < 2^16, or any start will do)
  kb = in / high + from % q.across;
  kb -= kb >= q.across ? q.across : 0;
  return true;
}

// One square.  rows, cols: what of it is inside the matrix; WHOLE: all of it
// (no comparison per row then; address arithmetic and comparisons, not memory,
// bounded the kernel: pointers are made once per thread and go on by scalars).
template <int SRC, int A, bool WHOLE>
__device__ __forceinline__ void square_body(const F8QuantizeArgs& a, uint32_t band, uint32_t kb, int rows, int cols,
                                            uint32_t (&most)[4][128], uint8_t (&turned)[128 * 128]) {
  const int t = threadIdx.x, c8 = t & 15, rg = t >> 4, wave = t >> 6;
  const int64_t row0 = static_cast<int64_t>(band) * 128, col0 = static_cast<int64_t>(kb) * 128;
  const int64_t spitch = f8_scale_pitch(a.cols);
  const int left = WHOLE ? 8 : cols - 8 * c8;  // columns from the thread's first on
  auto inside = [&](int p) { return WHOLE || (8 * rg + p < rows && left > 0); };
  Piece<SRC> in[8];
  if constexpr (SRC == PT_F8) {
    const uint8_t* const x = static_cast<const uint8_t*>(a.x) + (row0 + 8 * rg) * a.ldx + col0 + 8 * c8;
#pragma unroll
    for (int p = 0; p < 8; ++p)
      // (codes past the columns are no values: their column is not written)
      in[p].w = inside(p) ? load_wide<A>(reinterpret_cast<const u32x2*>(x + p * a.ldx)) : u32x2{0, 0};
    // the scales of the thread's rows: one per lane, handed on
    uint32_t bytes = 0;
    if (c8 < 8 && (WHOLE || 8 * rg + c8 < rows)) bytes = a.x_scales[(row0 + 8 * rg + c8) * spitch + kb];
    in[0].byte = row16_lane<0>(bytes);
    in[1].byte = row16_lane<1>(bytes);
    in[2].byte = row16_lane<2>(bytes);
    in[3].byte = row16_lane<3>(bytes);
    in[4].byte = row16_lane<4>(bytes);
    in[5].byte = row16_lane<5>(bytes);
    in[6].byte = row16_lane<6>(bytes);
    in[7].byte = row16_lane<7>(bytes);
  } else {
    constexpr int es = SRC == PT_F32 ? 4 : 2;
    // (fp32: a lane's 32 bytes are two loads of half of each line's bytes, and past
    // the caches the line came twice: 8192 x 13312 both ways 184 us, with plain loads 139)
    constexpr int kLoad = A == STREAM && SRC == PT_F32 ? ALIGNED : A;
    const uint8_t* const x = static_cast<const uint8_t*>(a.x) + ((row0 + 8 * rg) * a.ldx + col0 + 8 * c8) * es;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      in[p].raw.zero();
      if (inside(p)) in[p].raw.template load<kLoad>(x + p * a.ldx * es, 0, left);
    }
  }
  // magnitudes: of the thread's rows (rm) and columns (cm)
  uint32_t rm[8], cm[8];
  if constexpr (SRC == PT_BF16) {
    uint32_t pair[4] = {0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t m2 = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t m = in[p].raw.w[j] & 0x7fff7fffu;
        m2 = max_pair(m2, m);
        pair[j] = max_pair(pair[j], m);
      }
      rm[p] = max(m2 << 16, m2 & 0xffff0000u);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cm[2 * j] = pair[j] << 16;
      cm[2 * j + 1] = pair[j] & 0xffff0000u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) cm[j] = 0;
    bool none = false;  // a row's block is NaN
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      rm[p] = 0;
      if constexpr (SRC == PT_F8) none |= in[p].byte == 255u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[4];
        in[p].four(h, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          rm[p] = max(rm[p], magnitude(v[j]));
          cm[4 * h + j] = max(cm[4 * h + j], magnitude(v[j]));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) cm[j] = none ? 0x7f800000u : cm[j];
  }
  // columns: over the wave's four groups of rows, then over the waves
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const auto x = __builtin_amdgcn_permlane16_swap(cm[j], cm[j], false, false);
    const uint32_t m = max(x[0], x[1]);
    const auto y = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    cm[j] = max(y[0], y[1]);
  }
  if ((t & 63) < 16) {
    *reinterpret_cast<u32x4*>(&most[wave][8 * c8]) = u32x4{cm[0], cm[1], cm[2], cm[3]};
    *reinterpret_cast<u32x4*>(&most[wave][8 * c8 + 4]) = u32x4{cm[4], cm[5], cm[6], cm[7]};
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) cm[j] = max(max(most[0][8 * c8 + j], most[1][8 * c8 + j]), max(most[2][8 * c8 + j], most[3][8 * c8 + j]));
  uint32_t all = 0;
  if (a.square) {
#pragma unroll
    for (int j = 0; j < 8; ++j) all = max(all, cm[j]);
    all = row16_max(all);
  }
  if constexpr (SRC != PT_F8) {
    if (a.codes) {
      const int64_t pitch = f8_pitch(a.cols);
      uint8_t* const to = a.codes + (row0 + 8 * rg) * pitch + col0 + 8 * c8;
      uint32_t own = 0;  // the scale byte of row 8 rg + c8
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const uint32_t byte = block_byte(a.square ? all : row16_max(rm[p]));
        own = c8 == p ? byte : own;
        if (!WHOLE && 8 * rg + p >= rows) continue;  // (past the columns: zeros up to the pitch)
        u32x2 w;
        if constexpr (SRC == PT_BF16) {
          w = pack8_bf16(in[p].raw.w, block_factor(byte));
        } else {
          float v[8];
          in[p].raw.get(v);
          w = pack8(v, block_factor(byte));
        }
        if (byte == 255u) w = u32x2{0, 0};
        store_wide<A>(reinterpret_cast<u32x2*>(to + p * pitch), w);
      }
      uint8_t* const s = a.scales + (row0 + 8 * rg) * spitch;
      if (c8 < 8 && (WHOLE || 8 * rg + c8 < rows)) s[c8 * spitch + kb] = static_cast<uint8_t>(own);
      const int64_t blocks = pitch / kF8Block;
      if (kb == blocks - 1 && c8 < spitch - blocks)
        for (int p = 0; p < 8; ++p)
          if (8 * rg + p < rows) s[p * spitch + blocks + c8] = 0;
    }
  }
  if (!a.codes_t) return;
  const int64_t pitch_t = f8_pitch(a.rows), spitch_t = f8_scale_pitch(a.rows), blocks_t = pitch_t / kF8Block;
  uint32_t own = 0;  // the scale byte of column 8 c8 + rg
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8][4];
#pragma unroll
    for (int p = 0; p < 8; ++p) in[p].four(h, v[p]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 4 * h + i;
      const uint32_t byte = block_byte(a.square ? all : cm[j]);
      own = rg == j ? byte : own;
      const float r[8] = {v[0][i], v[1][i], v[2][i], v[3][i], v[4][i], v[5][i], v[6][i], v[7][i]};
      u32x2 w = pack8(r, block_factor(byte));
      if (byte == 255u) w = u32x2{0, 0};
      // column 8 c8 + j, its rows' pieces of 8 permuted by c8: the 16 columns of a write are on banks of their own
      *reinterpret_cast<u32x2*>(turned + (8 * c8 + j) * 128 + 8 * (rg ^ c8)) = w;
    }
  }
  uint8_t* const s = a.scales_t + (col0 + 8 * c8) * spitch_t;
  if (rg < 8 && (WHOLE || rg < left)) s[rg * spitch_t + band] = static_cast<uint8_t>(own);
  if (band == blocks_t - 1 && rg < spitch_t - blocks_t)
    for (int j = 0; j < 8; ++j)
      if (j < left) s[j * spitch_t + blocks_t + rg] = 0;
  __syncthreads();
  uint8_t* const to = a.codes_t + (col0 + (t >> 3)) * pitch_t + row0 + 16 * (t & 7);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = (t >> 3) + 32 * i, m = t & 7, perm = c >> 3;
    if (!WHOLE && c >= cols) continue;
    const u32x4 w = *reinterpret_cast<const u32x4*>(turned + c * 128 + 16 * (m ^ (perm >> 1)));
    store_wide<A>(reinterpret_cast<u32x4*>(to + 32 * i * pitch_t), perm & 1 ? u32x4{w[2], w[3], w[0], w[1]} : w);
  }
}

template <int SRC, int A>
__global__ __launch_bounds__(kThreads) void f8_square_kernel(F8QuantizeArgs a, Squares squares) {
  __shared__ __attribute__((aligned(16))) uint32_t most[4][128];
  __shared__ __attribute__((aligned(16))) uint8_t turned[128 * 128];
  uint32_t band, kb;
  if (!square_of(squares, blockIdx.y * kGridX + blockIdx.x, band, kb)) return;
  const int rows = static_cast<int>(min(a.rows - static_cast<int64_t>(band) * 128, int64_t{128}));
  const int cols = static_cast<int>(min(a.cols - static_cast<int64_t>(kb) * 128, int64_t{128}));
  if (rows == 128 && cols == 128)
    square_body<SRC, A, true>(a, band, kb, rows, cols, most, turned);
  else
    square_body<SRC, A, false>(a, band, kb, rows, cols, most, turned);
}

template <int T, int A>
__global__ __launch_bounds__(kThreads) void f8_dequantize_kernel(F8DequantizeArgs a, Rows rows) {
  const int64_t pitch = f8_pitch(a.cols), spitch = f8_scale_pitch(a.cols);
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * rows.rows;
  const int64_t left = (a.rows - row0) * rows.d;
  const uint32_t pieces = left < rows.pieces ? static_cast<uint32_t>(left) : rows.pieces;
  const uint32_t first = blockIdx.x * kSegment + threadIdx.x;
  u32x2 w[kPieces];
  uint32_t sb[kPieces];
  int64_t row[kPieces];
  int32_t col[kPieces];
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const uint32_t i = first + c * kThreads;
    if (i < pieces) {
      const uint32_t r = row_of(rows, i);
      row[c] = row0 + r;
      col[c] = static_cast<int32_t>(i - r * rows.d);
      w[c] = load_wide<A>(reinterpret_cast<const u32x2*>(a.codes + row[c] * pitch + 8 * static_cast<int64_t>(col[c])));
      sb[c] = a.scales[row[c] * spitch + (col[c] >> 4)];
    }
  }
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    if (first + c * kThreads >= pieces) continue;
    const int64_t at = 8 * static_cast<int64_t>(col[c]);
    if (at >= a.cols) continue;
    float v[8];
    unpack8(w[c], block_factor(sb[c]), v);
    if (sb[c] == 255u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __builtin_nanf("");
    }
    Raw8<T> out;
    out.set(v);
    out.template store<A>(a.y, row[c] * a.ldy + at, static_cast<int>(min(a.cols - at, int64_t{8})));
  }
}

// How the plain side is reached: whole aligned pieces where its rows allow them.
static int plain_access(const void* p, int64_t ld, int es, int64_t cols, int64_t bytes) {
  if (((reinterpret_cast<uint64_t>(p) | static_cast<uint64_t>(ld * es)) & 15) != 0 || cols % 8 != 0) return ANY;
  return bytes < kLastLevelCache ? ALIGNED : STREAM;
}

template <int T>
static void rows_t(const F8QuantizeArgs& a, int access, hipStream_t st) {
  dim3 grid;
  const Rows rows = split_rows(a.rows, f8_pitch(a.cols), &grid);
  if (access == STREAM)
    hipLaunchKernelGGL((f8_rows_kernel<T, STREAM>), grid, dim3(kThreads), 0, st, a, rows);
  else if (access == ALIGNED)
    hipLaunchKernelGGL((f8_rows_kernel<T, ALIGNED>), grid, dim3(kThreads), 0, st, a, rows);
  else
    hipLaunchKernelGGL((f8_rows_kernel<T, ANY>), grid, dim3(kThreads), 0, st, a, rows);
}

template <int SRC>
static void square_t(const F8QuantizeArgs& a, int access, hipStream_t st) {
  const Squares n{static_cast<uint32_t>(f8_blocks(a.rows)), static_cast<uint32_t>(f8_blocks(a.cols))};
  const int64_t squares = (static_cast<int64_t>(n.bands) * n.across + kXcds - 1) / kXcds * kXcds;
  const dim3 grid(grid_x(squares), grid_y(squares));
  if (access == STREAM)
    hipLaunchKernelGGL((f8_square_kernel<SRC, STREAM>), grid, dim3(kThreads), 0, st, a, n);
  else if (access == ALIGNED || SRC == PT_F8)
    hipLaunchKernelGGL((f8_square_kernel<SRC, ALIGNED>), grid, dim3(kThreads), 0, st, a, n);
  else
    hipLaunchKernelGGL((f8_square_kernel<SRC, (SRC == PT_F8 ? ALIGNED : ANY)>), grid, dim3(kThreads), 0, st, a, n);
}

template <int T>
static void quantize_t(const F8QuantizeArgs& a, hipStream_t st) {
  const int es = T == PT_F32 ? 4 : 2;
  const int access = plain_access(a.x, a.ldx, es, a.cols, a.rows * a.cols * (es + (a.codes ? 1 : 0) + (a.codes_t ? 1 : 0)));
  if (a.codes_t || a.square)
    square_t<T>(a, access, st);
  else
    rows_t<T>(a, access, st);
}

template <int T>
static void dequantize_t(const F8DequantizeArgs& a, hipStream_t st) {
  const int es = T == PT_F32 ? 4 : 2, access = plain_access(a.y, a.ldy, es, a.cols, a.rows * a.cols * (es + 1));
  dim3 grid;
  const Rows rows = split_rows(a.rows, f8_pitch(a.cols), &grid);
  if (access == STREAM)
    hipLaunchKernelGGL((f8_dequantize_kernel<T, STREAM>), grid, dim3(kThreads), 0, st, a, rows);
  else if (access == ALIGNED)
    hipLaunchKernelGGL((f8_dequantize_kernel<T, ALIGNED>), grid, dim3(kThreads), 0, st, a, rows);
  else
    hipLaunchKernelGGL((f8_dequantize_kernel<T, ANY>), grid, dim3(kThreads), 0, st, a, rows);
}

}  // namespace f8

hipError_t launch_f8_quantize(int x_type, const F8QuantizeArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (x_type == PT_F32)
    f8::quantize_t<PT_F32>(a, st);
  else
    f8::quantize_t<PT_BF16>(a, st);
  return hipGetLastError();
}

hipError_t launch_f8_transpose(const F8QuantizeArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  f8::square_t<f8::PT_F8>(a, 2 * a.rows * a.cols < kLastLevelCache ? f8::ALIGNED : f8::STREAM, st);
  return hipGetLastError();
}

hipError_t launch_f8_dequantize(int y_type, const F8DequantizeArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (y_type == PT_F32)
    f8::dequantize_t<PT_F32>(a, st);
  else
    f8::dequantize_t<PT_BF16>(a, st);
  return hipGetLastError();
}

}  // namespace dg
