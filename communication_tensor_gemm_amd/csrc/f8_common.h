// Internal interface of the 8-bit training operators (F8 tensors, their
// products, the layer norm) and the device helpers that they share.
//
// An F8 tensor of rows x cols: per row f8_pitch(cols) E4M3 codes, zero past
// cols, and one E8M0 byte b per block of 128 codes, the block's values being
// code * 2^(b - 127) (b = 255: the block is NaN), a row of scales taking
// f8_scale_pitch(cols) bytes.
#pragma once
#include "f8_shape.h"
#include "mx_common.h"
#include "mx_shape.h"

namespace dg {

constexpr int kF8Block = 128;
__host__ __device__ inline int64_t f8_blocks(int64_t k) { return (k + kF8Block - 1) / kF8Block; }
__host__ __device__ inline int64_t f8_pitch(int64_t k) { return f8_blocks(k) * kF8Block; }
__host__ __device__ inline int64_t f8_scale_pitch(int64_t k) { return (f8_blocks(k) + 15) / 16 * 16; }

// what the layer norm writes: the input's type, e4m3 with one given scale, or F8 blocks
enum LayerNormOut { LO_SAME = 0, LO_E4M3 = 1, LO_F8 = 2 };

struct F8QuantizeArgs {
  const void* x;           // rows of ldx elements, or the codes of an F8 tensor
  const uint8_t* x_scales; // of that tensor
  int64_t ldx;
  int64_t rows, cols;
  uint8_t *codes, *scales;      // by rows, or NULL
  uint8_t *codes_t, *scales_t;  // of the transpose, or NULL
  int32_t square;               // blocks of 128 x 128 share a scale
};

struct F8DequantizeArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols;
  void* y;
  int64_t ldy;
};

struct LayerNormArgs {
  const void* x;
  const void* residual;  // or NULL
  const void* weight;    // cols
  const void* bias;      // cols, or NULL
  void* y;
  void* h;               // x + residual in x's type, or NULL (no residual)
  float* mean;           // or NULL
  float* rstd;           // or NULL
  uint8_t* scales;       // LO_F8
  uint8_t *kept, *kept_scales;  // the normalised rows as an F8 tensor, or NULL
  int64_t ldx, ldr, ldy, ldh;
  int64_t rows;
  int32_t cols;
  float eps;
  float inv_scale;       // LO_E4M3: 1 / scale
};

struct LayerNormBackwardArgs {
  const void* dy;
  const void* h;            // the stream, or its normalised rows as an F8 tensor
  const uint8_t* h_scales;  // then its scales
  const void* dh;           // or NULL
  const float* mean;
  const float* rstd;
  const void* weight;
  void* dx;
  float* dweight;
  float* dbias;    // or NULL
  float* partial;  // [blocks][2][cols]
  int64_t lddy, ldh, lddh, lddx;
  int64_t rows;
  int32_t cols;
};

hipError_t launch_f8_quantize(int x_type, const F8QuantizeArgs& a, hipStream_t st);
hipError_t launch_f8_transpose(const F8QuantizeArgs& a, hipStream_t st);
hipError_t launch_f8_dequantize(int y_type, const F8DequantizeArgs& a, hipStream_t st);
hipError_t launch_layer_norm(int type, int out, const LayerNormArgs& a, hipStream_t st);
int64_t layer_norm_backward_blocks(int64_t rows, int64_t cols);
hipError_t launch_layer_norm_backward(int type, const LayerNormBackwardArgs& a, hipStream_t st);
// Products: MxGemmArgs with F8 operands (no groups); work: of f8_gemm_workspace bytes.
hipError_t launch_f8_gemm(const MxGemmArgs& a, float* work, hipStream_t st);
// on tiles of 256 x 256, 128 x 128 or (size 64) 64 x 128
hipError_t launch_f8_gemm_tile(int size, const MxGemmArgs& a, hipStream_t st);
// on tiles of 64 x 128 with K in `parts` (f8_parts of it: every part has some of K), whose sums go through `sums`, parts
// x M rows of `pitch` values (a multiple of 4)
hipError_t launch_f8_gemm_split(const MxGemmArgs& a, int parts, float* sums, int64_t pitch, hipStream_t st);

#if defined(__HIPCC__)
namespace f8 {
using namespace mx;

// The block scale: the byte X + 127 of the least X with amax <= 448 * 2^X, at
// least -127; 255 for an infinity or a NaN.  amax is given by its bits (no
// sign); 448 = 1.75 * 2^8, and the exponent field of a subnormal is 0, where X
// is -127 in any case.
__device__ __forceinline__ uint32_t block_byte(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23);
  const int b = max(e - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
  return e == 255 ? 255u : static_cast<uint32_t>(b);
}

// 2^X as the scaling conversions take it: they read the exponent field, and 0 stands for 2^-127.
__device__ __forceinline__ float block_factor(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// The maximum over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t m) {
  m = quad_max(m);
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x141, 0xf, 0xf, true)));  // half mirror
  return max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x140, 0xf, 0xf, true)));  // mirror
}

// Four values over 2^X to E4M3 bytes, round to nearest even.  None is beyond 448 * 2^X.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float factor) {
  s16x2 r{0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, factor, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, factor, true);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ u32x2 pack8(const float (&v)[8], float factor) {
  return u32x2{pack4(v[0], v[1], v[2], v[3], factor), pack4(v[4], v[5], v[6], v[7], factor)};
}
// The same from eight bf16 values as they were loaded.
__device__ __forceinline__ u32x2 pack8_bf16(u32x4 v, float factor) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // (a bit cast of a vector's element would take the vector's first)
    const uint32_t e0 = v[2 * h], e1 = v[2 * h + 1];
    s16x2 r{0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, e0), factor, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, e1), factor, true);
    w[h] = __builtin_bit_cast(uint32_t, r);
  }
  return w;
}

// Eight codes over their scale's factor (not of a NaN block).
__device__ __forceinline__ void unpack8(u32x2 w, float factor, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], factor, false);
    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], factor, true);
    v[4 * h] = lo[0]; v[4 * h + 1] = lo[1]; v[4 * h + 2] = hi[0]; v[4 * h + 3] = hi[1];
  }
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

// The larger of two pairs of bf16 magnitudes.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// Quantise and store one lane's eight values of a row's block (all 16 lanes of
// the block call it), and, by the first of them, the block's scale byte.
template <int A>
__device__ __forceinline__ void store_block8(const float (&v)[8], uint8_t* codes, int64_t code_row, int col8,
                                             uint8_t* scales, int64_t scale_row) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, magnitude(v[j]));
  const uint32_t byte = block_byte(row16_max(m));
  u32x2 w = pack8(v, block_factor(byte));
  if (byte == 255u) w = u32x2{0, 0};
  store_wide<A>(reinterpret_cast<u32x2*>(codes + code_row + 8 * static_cast<int64_t>(col8)), w);
  if ((col8 & 15) == 0) scales[scale_row + (col8 >> 4)] = static_cast<uint8_t>(byte);
}

}  // namespace f8
#endif  // __HIPCC__
}  // namespace dg
