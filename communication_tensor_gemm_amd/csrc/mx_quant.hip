// Quantisation of a matrix to an MX tensor, and back.
//
// Per block of 32: X = floor(log2(max |x|)) - emax, element = round(x * 2^-X)
// to nearest even, saturating (mx_common.h, block_scale).  Both directions
// are bound by memory: 2 or 4 bytes in and 0.53 (E2M1) or 1.03 (E4M3) out per
// element.  A thread takes eight elements, so a bf16 load is 16 bytes and a
// block is four adjacent lanes, which exchange their maximum inside the quad;
// four such pieces per thread are loaded before the first is used.  8192 x
// 13312 bf16 to E4M3: 54 us, 6.1 TB/s (a copy: 6.2); 777 x 3584 to E2M1 and back:
// 3.7 and 4.2 us, a launch's latency more than its bytes (2.3 us for both).
#include "mx_common.h"

namespace dg {
namespace mx {

constexpr int kThreads = 256, kPieces = 4;
constexpr int kSegment = kThreads * kPieces;  // eight-element pieces of one workgroup

// Pieces are numbered through all rows (d to a row), a workgroup takes
// kSegment of them, so every lane has work whatever the row's length.  n / d
// for n below 2^31 is one product and a shift: with 2^(s-1) < d <= 2^s and m =
// floor(2^(31+s) / d) + 1, it is floor(n m / 2^(31+s)).
struct Rows {
  uint32_t d, m, shift;  // shift = s - 1
  uint32_t pieces;       // of a chunk of rows (one per blockIdx.y), below 2^31
  int64_t rows;          // of a chunk
};
__device__ __forceinline__ uint32_t row_of(const Rows& r, uint32_t n) { return __umulhi(n, r.m) >> r.shift; }

template <int T, int FMT, int A>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantizeArgs a, Rows rows) {
  const int64_t pitch = scale_pitch(a.cols), row_bytes = mx_row_bytes(a.cols, FMT);
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
    if (i < pieces) {
      const uint32_t r = row_of(rows, i);
      row[c] = row0 + r;
      col[c] = static_cast<int32_t>(i - r * rows.d);
      raw[c].template load<A>(a.x, row[c] * a.ldx + 8 * static_cast<int64_t>(col[c]), 8);
    }
  }
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    // the pieces of a block are four adjacent lanes: all of them are in or none is
    if (first + c * kThreads < pieces) {
      if constexpr (T == PT_BF16) {
        store_block_bf16<FMT, A>(raw[c].w, a.codes, row[c] * row_bytes, col[c], a.scales, row[c] * pitch);
      } else {
        float v[8];
        raw[c].get(v);
        store_block<FMT, A>(v, a.codes, row[c] * row_bytes, col[c], a.scales, row[c] * pitch);
      }
    }
  }
  // the scale bytes past K / 32, by the lane of the row's last block
  const int32_t blocks = static_cast<int32_t>(a.cols / kMxBlock), pad = static_cast<int32_t>(pitch) - blocks;
  if (pad > 0) {
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
      if (first + c * kThreads < pieces && col[c] == 4 * blocks - 4)
        for (int32_t k = 0; k < pad; ++k) a.scales[row[c] * pitch + blocks + k] = 0;
  }
}

// bytes of one E8M0 scale as a float (255: NaN)
__device__ __forceinline__ float scale_value(uint32_t b) {
  if (b == 255u) return __builtin_nanf("");
  return __builtin_bit_cast(float, b == 0u ? 0x00400000u : b << 23);
}

template <int T, int FMT, int A>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(DequantizeArgs a, Rows rows) {
  const int64_t pitch = scale_pitch(a.cols), row_bytes = mx_row_bytes(a.cols, FMT);
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
      if constexpr (FMT == MX_E4M3)
        w[c] = load_wide<A>(reinterpret_cast<const u32x2*>(a.codes + row[c] * row_bytes + 8 * static_cast<int64_t>(col[c])));
      else
        w[c][0] = load_wide<A>(reinterpret_cast<const uint32_t*>(a.codes + row[c] * row_bytes + 4 * static_cast<int64_t>(col[c])));
      sb[c] = a.scales[row[c] * pitch + (col[c] >> 2)];
    }
  }
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    if (first + c * kThreads >= pieces) continue;
    float v[8];
    if constexpr (FMT == MX_E4M3) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[c][h]), false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[c][h]), true);
        v[4 * h] = lo[0]; v[4 * h + 1] = lo[1]; v[4 * h + 2] = hi[0]; v[4 * h + 3] = hi[1];
      }
    } else {
      const f32x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c][0], 1.0f, 0);
      const f32x2 e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c][0], 1.0f, 1);
      const f32x2 e2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c][0], 1.0f, 2);
      const f32x2 e3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[c][0], 1.0f, 3);
      v[0] = e0[0]; v[1] = e0[1]; v[2] = e1[0]; v[3] = e1[1];
      v[4] = e2[0]; v[5] = e2[1]; v[6] = e3[0]; v[7] = e3[1];
    }
    const float s = scale_value(sb[c]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= s;
    Raw8<T> out;
    out.set(v);
    out.template store<A>(a.y, row[c] * a.ldy + 8 * static_cast<int64_t>(col[c]), 8);
  }
}

static Rows split_rows(int64_t rows, int64_t cols, dim3* grid) {
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

template <int T, int FMT>
static hipError_t quantize_t(const QuantizeArgs& a, hipStream_t st) {
  dim3 grid;
  const Rows rows = split_rows(a.rows, a.cols, &grid);
  const int es = T == PT_F32 ? 4 : 2;
  if (((reinterpret_cast<uint64_t>(a.x) | static_cast<uint64_t>(a.ldx * es)) & 15) != 0)
    hipLaunchKernelGGL((quantize_kernel<T, FMT, ANY>), grid, dim3(kThreads), 0, st, a, rows);
  else if (a.rows * a.cols * (es + (FMT == MX_E4M3)) < kLastLevelCache)
    hipLaunchKernelGGL((quantize_kernel<T, FMT, ALIGNED>), grid, dim3(kThreads), 0, st, a, rows);
  else
    hipLaunchKernelGGL((quantize_kernel<T, FMT, STREAM>), grid, dim3(kThreads), 0, st, a, rows);
  return hipGetLastError();
}

template <int T, int FMT>
static hipError_t dequantize_t(const DequantizeArgs& a, hipStream_t st) {
  dim3 grid;
  const Rows rows = split_rows(a.rows, a.cols, &grid);
  const int es = T == PT_F32 ? 4 : 2;
  if (((reinterpret_cast<uint64_t>(a.y) | static_cast<uint64_t>(a.ldy * es)) & 15) != 0)
    hipLaunchKernelGGL((dequantize_kernel<T, FMT, ANY>), grid, dim3(kThreads), 0, st, a, rows);
  else if (a.rows * a.cols * (es + (FMT == MX_E4M3)) < kLastLevelCache)
    hipLaunchKernelGGL((dequantize_kernel<T, FMT, ALIGNED>), grid, dim3(kThreads), 0, st, a, rows);
  else
    hipLaunchKernelGGL((dequantize_kernel<T, FMT, STREAM>), grid, dim3(kThreads), 0, st, a, rows);
  return hipGetLastError();
}

}  // namespace mx

hipError_t launch_mx_quantize(int x_type, int format, const QuantizeArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (x_type == PT_F32)
    return format == MX_E2M1 ? mx::quantize_t<PT_F32, MX_E2M1>(a, st) : mx::quantize_t<PT_F32, MX_E4M3>(a, st);
  return format == MX_E2M1 ? mx::quantize_t<PT_BF16, MX_E2M1>(a, st) : mx::quantize_t<PT_BF16, MX_E4M3>(a, st);
}

hipError_t launch_mx_dequantize(int y_type, int format, const DequantizeArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (y_type == PT_F32)
    return format == MX_E2M1 ? mx::dequantize_t<PT_F32, MX_E2M1>(a, st) : mx::dequantize_t<PT_F32, MX_E4M3>(a, st);
  return format == MX_E2M1 ? mx::dequantize_t<PT_BF16, MX_E2M1>(a, st) : mx::dequantize_t<PT_BF16, MX_E4M3>(a, st);
}

}  // namespace dg
