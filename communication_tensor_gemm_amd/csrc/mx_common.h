// Internal interface of the low-precision operators (MX tensors, their
// products, the RMS norm) and the device helpers that they share.
//
// An MX tensor of rows x K: per row K elements (E4M3: one byte each; E2M1:
// two per byte, the even element in the low nibble) and one E8M0 byte b per
// block of 32 consecutive elements, the block's values being element *
// 2^(b - 127) (b = 255: the block is NaN).  A row of scales takes
// scale_pitch(K) bytes: K / 32 rounded up to whole 16-byte chunks, so that a
// chunk (512 elements' scales) is one aligned 16-byte load anywhere; for K a
// multiple of 512 it is the plain rows x K/32 matrix.  Bytes past K / 32 are
// zero when a kernel here writes them and ignored when one reads them (the
// elements they would scale read as zero).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace dg {

enum MxFormat { MX_E2M1 = 0, MX_E4M3 = 1 };
enum PlainType { PT_F32 = 0, PT_BF16 = 1 };
// what the RMS norm writes: the input's type, e4m3 with one given scale, or MX blocks
enum NormOut { NO_SAME = 0, NO_E4M3 = 1, NO_MX_E2M1 = 2, NO_MX_E4M3 = 3 };

constexpr int kMxBlock = 32;

__host__ __device__ inline int64_t scale_pitch(int64_t k) { return (k / kMxBlock + 15) / 16 * 16; }
__host__ __device__ inline int64_t mx_row_bytes(int64_t k, int format) { return format == MX_E2M1 ? k / 2 : k; }

struct QuantizeArgs {
  const void* x;   // rows of ldx elements
  int64_t ldx;
  int64_t rows, cols;
  uint8_t* codes;  // rows x mx_row_bytes(cols)
  uint8_t* scales; // rows x scale_pitch(cols)
};

struct DequantizeArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols;
  void* y;
  int64_t ldy;
};

struct NormArgs {
  const void* x;
  const void* residual;  // or NULL
  const void* weight;    // cols
  void* y;
  void* h;               // x + residual in x's type, or NULL (no residual)
  float* rstd;           // or NULL
  uint8_t* scales;       // MX outputs
  int64_t ldx, ldr, ldy, ldh;
  int64_t rows;
  int32_t cols;
  float eps;
  float inv_scale;       // NO_E4M3: 1 / scale
};

struct NormBackwardArgs {
  const void* dy;
  const void* h;
  const void* dh;  // or NULL
  const float* rstd;
  const void* weight;
  void* dx;
  float* dweight;
  float* partial;  // [blocks][cols]
  int64_t lddy, ldh, lddh, lddx;
  int64_t rows;
  int32_t cols;
};

// One product D = alpha * A * B^T + beta * C (+ bias), or, with offsets, one
// per group of rows with the group's own B and bias.
struct MxGemmArgs {
  const uint8_t* A;
  const uint8_t* As;
  const uint8_t* B;
  const uint8_t* Bs;
  const void* C;      // read only when beta != 0
  const void* bias;   // N (per group) values of the output type, or NULL
  void* D;
  const int32_t* offsets;  // groups + 1 row offsets on the device, or NULL
  int64_t ldc, ldd;
  int32_t M, N, K;
  int32_t groups;     // 0: no groups
  int32_t a_format;
  int32_t out_bf16;
  int32_t cus;        // CUs of the device
  float alpha, beta;
};

hipError_t launch_mx_quantize(int x_type, int format, const QuantizeArgs& a, hipStream_t st);
hipError_t launch_mx_dequantize(int y_type, int format, const DequantizeArgs& a, hipStream_t st);
hipError_t launch_rms_norm(int type, int out, const NormArgs& a, hipStream_t st);
int64_t rms_norm_backward_blocks(int64_t rows, int64_t cols);
hipError_t launch_rms_norm_backward(int type, const NormBackwardArgs& a, hipStream_t st);
hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t st);
// on tiles of `size` (256 or 128) squared
hipError_t launch_mx_gemm_tile(int size, const MxGemmArgs& a, hipStream_t st);

// Bytes of the last-level cache, shared by the whole device.
constexpr int64_t kLastLevelCache = int64_t{256} << 20;
// Largest row that the RMS norm kernels keep in registers.
constexpr int kNormMaxCols = 32768;

#if defined(__HIPCC__)
namespace mx {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
typedef __attribute__((ext_vector_type(2))) short s16x2;
// the same at any alignment of their element: still one access of full width
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }

// Two values rounded to bf16 (to nearest even, a NaN stays one), the first
// low: one v_cvt_pk_bf16_f32, where integer rounding takes 14 instructions (the
// norm's gradient is bound by such instructions as much as by memory).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// How a kernel reaches its large matrices.  ANY: addresses are aligned to the
// element only, and a piece of eight may have fewer left in its row; whole
// pieces still move in accesses of full width (a 1021 x 5123 fp32 norm, whose
// rows start on every 4-byte offset: 31 us with element accesses, 10 with
// these).  ALIGNED: 16-byte aligned, whole pieces.  STREAM: the same, past
// the caches: where the operator's bytes exceed the last-level cache, what it
// writes could not stay there (quantise 8192 x 13312: 59 us without, 54 with;
// norm 8192 x 16384: 165 and 156; its gradient 8192 x 8192: 107 and 99), and
// below that size the next operator finds it there.
enum Access { ANY = 0, ALIGNED = 1, STREAM = 2 };

template <int A, typename V>
__device__ __forceinline__ V load_wide(const V* p) {
  if constexpr (A == STREAM)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}
template <int A, typename V>
__device__ __forceinline__ void store_wide(V* p, V v) {
  if constexpr (A == STREAM)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

// Eight consecutive elements of a row, as loaded.  n (ANY): elements left in
// the row from the first; those past its end read as zero.
template <int T>
struct Raw8;
template <>
struct Raw8<PT_BF16> {
  u32x4 w;
  template <int A>
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    const uint16_t* s = static_cast<const uint16_t*>(p) + i;
    if constexpr (A != ANY) {
      w = load_wide<A>(reinterpret_cast<const u32x4*>(s));
    } else if (n >= 8) {
      w = *reinterpret_cast<const u32x4_any*>(s);
    } else {
      uint32_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = j < n ? s[j] : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = e[2 * j] | (e[2 * j + 1] << 16);
    }
  }
  __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_lo(w[j]);
      f[2 * j + 1] = bf16_hi(w[j]);
    }
  }
  // round to the type; f keeps the rounded values
  __device__ __forceinline__ void set(float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
    get(f);
  }
  template <int A>
  __device__ __forceinline__ void store(void* p, int64_t i, int n) const {
    uint16_t* d = static_cast<uint16_t*>(p) + i;
    if constexpr (A != ANY) {
      store_wide<A>(reinterpret_cast<u32x4*>(d), w);
    } else if (n >= 8) {
      *reinterpret_cast<u32x4_any*>(d) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) d[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
    }
  }
};
template <>
struct Raw8<PT_F32> {
  f32x4 a, b;
  template <int A>
  __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
    const float* s = static_cast<const float*>(p) + i;
    if constexpr (A != ANY) {
      a = load_wide<A>(reinterpret_cast<const f32x4*>(s));
      b = load_wide<A>(reinterpret_cast<const f32x4*>(s + 4));
    } else if (n >= 8) {
      a = *reinterpret_cast<const f32x4_any*>(s);
      b = *reinterpret_cast<const f32x4_any*>(s + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = j < n ? s[j] : 0.0f;
        b[j] = j + 4 < n ? s[j + 4] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void zero() { a = b = f32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = a[j];
      f[j + 4] = b[j];
    }
  }
  __device__ __forceinline__ void set(float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = f[j];
      b[j] = f[j + 4];
    }
  }
  template <int A>
  __device__ __forceinline__ void store(void* p, int64_t i, int n) const {
    float* d = static_cast<float*>(p) + i;
    if constexpr (A != ANY) {
      store_wide<A>(reinterpret_cast<f32x4*>(d), a);
      store_wide<A>(reinterpret_cast<f32x4*>(d + 4), b);
    } else if (n >= 8) {
      *reinterpret_cast<f32x4_any*>(d) = a;
      *reinterpret_cast<f32x4_any*>(d + 4) = b;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < n) d[j] = a[j];
        if (j + 4 < n) d[j + 4] = b[j];
      }
    }
  }
};

// Eight values to e4m3 bytes, round to nearest even.  The conversion
// instruction gives NaN past 464, so the values are clamped to +-448 first;
// v_med3 makes a bound of a NaN, so where there can be one it is kept apart.
template <bool kNan>
__device__ __forceinline__ u32x2 pack_e4m3(const float (&v)[8]) {
  float c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] = __builtin_amdgcn_fmed3f(v[j], -448.0f, 448.0f);
    if constexpr (kNan) c[j] = v[j] != v[j] ? v[j] : c[j];
  }
  u32x2 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * h], c[4 * h + 1], w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * h + 2], c[4 * h + 3], w, true);
    r[h] = static_cast<uint32_t>(w);
  }
  return r;
}

// Eight values to e2m1 codes, round to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&v)[8]) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
  return w;
}

// The block scale of the microscaling formats: 2^X with X = floor(log2(amax))
// - emax, emax the exponent of the element format's largest value (E2M1: 2,
// E4M3: 8), X at least -127 (what E8M0 holds).  Returns the byte X + 127, and
// the exact factor 2^-X in `inv`.  A block with an infinity or a NaN has no
// scale: byte 255, and inv = 0.  amax is given by its bits (no sign): the
// exponent field of a subnormal is 0, where X is -127 in any case.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, float& inv) {
  constexpr int emax = FMT == MX_E2M1 ? 2 : 8;
  const int e = static_cast<int>(amax_bits >> 23);
  if (e == 255) {
    inv = 0.0f;
    return 255u;
  }
  const int b = max(e - emax, 0);
  inv = __builtin_bit_cast(float, static_cast<uint32_t>(254 - b) << 23);
  return static_cast<uint32_t>(b);
}

// The larger of a block's four lanes' values: the lanes 4b .. 4b + 3 of one
// block exchange within the quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0xB1, 0xf, 0xf, true)));
  return max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x4E, 0xf, 0xf, true)));
}

// Store one lane's eight codes of a block, and the block's scale byte.
template <int FMT, int A>
__device__ __forceinline__ void store_codes(u32x2 w, uint32_t byte, uint8_t* codes, int64_t code_row, int col8,
                                            uint8_t* scales, int64_t scale_row) {
  // a block without a scale has zero codes
  w[0] = byte == 255u ? 0u : w[0];
  if constexpr (FMT == MX_E4M3) {
    w[1] = byte == 255u ? 0u : w[1];
    store_wide<A>(reinterpret_cast<u32x2*>(codes + code_row + 8 * static_cast<int64_t>(col8)), w);
  } else {
    const uint32_t lo = w[0];
    store_wide<A>(reinterpret_cast<uint32_t*>(codes + code_row + 4 * static_cast<int64_t>(col8)), lo);
  }
  if ((col8 & 3) == 0) scales[scale_row + (col8 >> 2)] = static_cast<uint8_t>(byte);
}

// Quantise and store one lane's eight elements of a block (every lane of the
// quad calls it).
template <int FMT, int A>
__device__ __forceinline__ void store_block(const float (&v)[8], uint8_t* codes, int64_t code_row, int col8,
                                            uint8_t* scales, int64_t scale_row) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
  float inv;
  const uint32_t byte = block_scale<FMT>(quad_max(m), inv);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = v[j] * inv;
  u32x2 w{0, 0};
  if constexpr (FMT == MX_E4M3)
    w = pack_e4m3<false>(q);
  else
    w[0] = pack_e2m1(q);
  store_codes<FMT, A>(w, byte, codes, code_row, col8, scales, scale_row);
}

// The same from eight bf16 values as they were loaded, on pairs: the
// magnitudes' maximum and the clamp to 448 * 2^X are 16-bit integer
// operations, and the conversions take bf16 pairs and the scale (4 against 11
// instructions per element; they, not memory, bounded the quantiser).
template <int FMT, int A>
__device__ __forceinline__ void store_block_bf16(u32x4 v, uint8_t* codes, int64_t code_row, int col8, uint8_t* scales,
                                                 int64_t scale_row) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  uint32_t mag[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) mag[j] = v[j] & 0x7fff7fffu;
  auto max2 = [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
  };
  const uint32_t m2 = max2(max2(mag[0], mag[1]), max2(mag[2], mag[3]));
  float inv;
  const uint32_t byte = block_scale<FMT>(quad_max(max(m2 << 16, m2 & 0xffff0000u)), inv);
  // 2^X; the conversion takes its exponent field, so 0 stands for 2^-127
  const float scale = __builtin_bit_cast(float, byte << 23);
  u32x2 w{0, 0};
  if constexpr (FMT == MX_E4M3) {
    const uint32_t top = ((byte + 8u) << 7 | 0x60u) * 0x10001u;  // 448 * 2^X
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t t = __builtin_bit_cast(
          uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, mag[j]), __builtin_bit_cast(u16x2, top)));
      c[j] = t | (v[j] & 0x80008000u);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s16x2 r{0, 0};
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, c[2 * h]), scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, c[2 * h + 1]), scale, true);
      w[h] = __builtin_bit_cast(uint32_t, r);
    }
  } else {
    // (a bit cast of a vector's element would take the vector's first)
    const uint32_t e0 = v[0], e1 = v[1], e2 = v[2], e3 = v[3];
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, e0), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, e1), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, e2), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, e3), scale, 3);
    w[0] = r;
  }
  store_codes<FMT, A>(w, byte, codes, code_row, col8, scales, scale_row);
}

}  // namespace mx
#endif  // __HIPCC__
}  // namespace dg
