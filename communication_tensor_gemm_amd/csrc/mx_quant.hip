// Quantisation of a matrix to an MX tensor, and back.
//
// Per block of 32: X = floor(log2(max |x|)) - emax, element = round(x * 2^-X)
// to nearest even, saturating (mx_common.h, block_scale).  Both directions
// are bound by memory: 2 or 4 bytes in and 0.53 (E2M1) or 1.03 (E4M3) out per
// element.  A thread takes eight elements, so a bf16 load is 16 bytes and a
// block is four adjacent lanes, which exchange their maximum inside the quad;
// four such pieces per thread are loaded before the first is used.
#include "mx_common.h"

namespace dg {
namespace mx {

constexpr int kThreads = 256, kPieces = 4;
constexpr int kSegment = kThreads * kPieces;  // eight-element pieces of one workgroup

// A workgroup's pieces: a segment of one row, or several short rows.
struct Pieces {
  int64_t row0;
  int32_t rows, d, first, n;  // rows, pieces per row, first piece of the row, pieces in all
};
__device__ __forceinline__ Pieces my_pieces(int64_t rows, int32_t d, int32_t per_group, int32_t segment) {
  Pieces p;
  p.d = d;
  p.row0 = static_cast<int64_t>(blockIdx.x) * per_group;
  const int64_t left = rows - p.row0;
  p.rows = static_cast<int32_t>(left < per_group ? left : per_group);
  p.first = static_cast<int32_t>(blockIdx.y) * segment;
  p.n = per_group == 1 ? min(segment, d - p.first) : p.rows * d;
  return p;
}

template <int T, int FMT, bool kAligned>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantizeArgs a, int32_t per_group, int32_t segment) {
  const int32_t d = static_cast<int32_t>(a.cols / 8);
  const int64_t pitch = scale_pitch(a.cols), row_bytes = mx_row_bytes(a.cols, FMT);
  const Pieces p = my_pieces(a.rows, d, per_group, segment);
  Raw8<T> raw[kPieces];
  int64_t row[kPieces];
  int32_t col[kPieces];
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int32_t i = c * kThreads + static_cast<int32_t>(threadIdx.x);
    if (i < p.n) {
      const int32_t r = per_group == 1 ? 0 : i / d;
      row[c] = p.row0 + r;
      col[c] = p.first + (i - r * d);
      raw[c].template load<kAligned>(a.x, row[c] * a.ldx + 8 * static_cast<int64_t>(col[c]), 8);
    }
  }
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    // the pieces of a block are four adjacent lanes: all of them are in or none is
    if (c * kThreads + static_cast<int32_t>(threadIdx.x) < p.n) {
      float v[8];
      raw[c].get(v);
      store_block<FMT>(v, a.codes, row[c] * row_bytes, col[c], a.scales, row[c] * pitch);
    }
  }
  // the row's scale bytes past K / 32
  const int32_t pad = static_cast<int32_t>(pitch - a.cols / kMxBlock);
  if (pad > 0 && p.first + segment >= d)
    for (int32_t i = threadIdx.x; i < p.rows * pad; i += kThreads) {
      const int32_t r = i / pad;
      a.scales[(p.row0 + r) * pitch + a.cols / kMxBlock + (i - r * pad)] = 0;
    }
}

// bytes of one E8M0 scale as a float (255: NaN)
__device__ __forceinline__ float scale_value(uint32_t b) {
  if (b == 255u) return __builtin_nanf("");
  return __builtin_bit_cast(float, b == 0u ? 0x00400000u : b << 23);
}

template <int T, int FMT, bool kAligned>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(DequantizeArgs a, int32_t per_group, int32_t segment) {
  const int32_t d = static_cast<int32_t>(a.cols / 8);
  const int64_t pitch = scale_pitch(a.cols), row_bytes = mx_row_bytes(a.cols, FMT);
  const Pieces p = my_pieces(a.rows, d, per_group, segment);
  u32x2 w[kPieces];
  uint32_t sb[kPieces];
  int64_t row[kPieces];
  int32_t col[kPieces];
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int32_t i = c * kThreads + static_cast<int32_t>(threadIdx.x);
    if (i < p.n) {
      const int32_t r = per_group == 1 ? 0 : i / d;
      row[c] = p.row0 + r;
      col[c] = p.first + (i - r * d);
      if constexpr (FMT == MX_E4M3)
        w[c] = *reinterpret_cast<const u32x2*>(a.codes + row[c] * row_bytes + 8 * static_cast<int64_t>(col[c]));
      else
        w[c][0] = *reinterpret_cast<const uint32_t*>(a.codes + row[c] * row_bytes + 4 * static_cast<int64_t>(col[c]));
      sb[c] = a.scales[row[c] * pitch + (col[c] >> 2)];
    }
  }
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    if (c * kThreads + static_cast<int32_t>(threadIdx.x) >= p.n) continue;
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
    out.template store<kAligned>(a.y, row[c] * a.ldy + 8 * static_cast<int64_t>(col[c]), 8);
  }
}

// rows per workgroup (short rows) and pieces per segment (long rows)
static void split_rows(int64_t rows, int64_t cols, int32_t* per_group, int32_t* segment, dim3* grid) {
  const int64_t d = cols / 8;
  int64_t segs = 1;
  if (d >= kSegment) {
    *per_group = 1;
    segs = (d + kSegment - 1) / kSegment;
    // equal segments of whole blocks
    *segment = static_cast<int32_t>(((d + segs - 1) / segs + 3) / 4 * 4);
    segs = (d + *segment - 1) / *segment;
  } else {
    *per_group = static_cast<int32_t>(kSegment / d);
    *segment = static_cast<int32_t>(d);
  }
  *grid = dim3(static_cast<unsigned>((rows + *per_group - 1) / *per_group), static_cast<unsigned>(segs));
}

template <int T, int FMT>
static hipError_t quantize_t(const QuantizeArgs& a, hipStream_t st) {
  int32_t per_group, segment;
  dim3 grid;
  split_rows(a.rows, a.cols, &per_group, &segment, &grid);
  const int es = T == PT_F32 ? 4 : 2;
  if (((reinterpret_cast<uint64_t>(a.x) | static_cast<uint64_t>(a.ldx * es)) & 15) == 0)
    hipLaunchKernelGGL((quantize_kernel<T, FMT, true>), grid, dim3(kThreads), 0, st, a, per_group, segment);
  else
    hipLaunchKernelGGL((quantize_kernel<T, FMT, false>), grid, dim3(kThreads), 0, st, a, per_group, segment);
  return hipGetLastError();
}

template <int T, int FMT>
static hipError_t dequantize_t(const DequantizeArgs& a, hipStream_t st) {
  int32_t per_group, segment;
  dim3 grid;
  split_rows(a.rows, a.cols, &per_group, &segment, &grid);
  const int es = T == PT_F32 ? 4 : 2;
  if (((reinterpret_cast<uint64_t>(a.y) | static_cast<uint64_t>(a.ldy * es)) & 15) == 0)
    hipLaunchKernelGGL((dequantize_kernel<T, FMT, true>), grid, dim3(kThreads), 0, st, a, per_group, segment);
  else
    hipLaunchKernelGGL((dequantize_kernel<T, FMT, false>), grid, dim3(kThreads), 0, st, a, per_group, segment);
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
