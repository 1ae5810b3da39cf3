// F8 product on square tiles, for many rows of A (mx_tile_loop.h has the main
// loop).
#include "f8_common.h"
#include "mx_tile_loop.h"

namespace dg {
namespace f8 {

template <bool kBf16, int NBM, int NBN, int KG, bool kSplit>
__global__ __launch_bounds__(256 * KG) __attribute__((amdgpu_waves_per_eu(NBM == 2 ? 2 : 1, NBM == 2 ? 2 : 1)))
void f8_gemm_tile_kernel(MxGemmArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[KG * Geo<true, true, NBM, NBN>::kLds];
  run_tiles<true, true, kBf16, NBM, NBN, KG, kSplit>(p, smem);
}

template <bool kBf16, int NBM, int NBN>
static hipError_t tile_t(const MxGemmArgs& a, hipStream_t st) {
  using G = Geo<true, true, NBM, NBN>;
  const int64_t T = static_cast<int64_t>(tile_count(a.M, G::TM)) * tile_count(a.N, G::TN);
  if (T > INT32_MAX / 2) return hipErrorInvalidConfiguration;
  const int64_t most = static_cast<int64_t>(a.cus) * G::kWgs;
  const int64_t grid = ((T < most ? T : most) + kXcds - 1) / kXcds * kXcds;
  const dim3 wgs(static_cast<unsigned>(grid));
  if constexpr (NBM == 2) {
    if (T <= a.cus && a.K > 4096) {
      hipLaunchKernelGGL((f8_gemm_tile_kernel<kBf16, NBM, NBN, 2, false>), wgs, dim3(512), 0, st, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((f8_gemm_tile_kernel<kBf16, NBM, NBN, 1, false>), wgs, dim3(256), 0, st, a);
  return hipGetLastError();
}

// K in parts, one per blockIdx.y, into `sums` (parts x M rows of `pitch` values):
// every workgroup has at most one tile.
static hipError_t split_sums(const MxGemmArgs& a, int parts, float* sums, int64_t pitch, hipStream_t st) {
  using G = Geo<true, true, 1, 2>;
  MxGemmArgs p = a;
  p.C = p.bias = nullptr;
  p.D = sums;
  p.ldd = pitch;
  p.out_bf16 = 0;
  p.alpha = 1.0f;
  p.beta = 0.0f;
  const int64_t T = static_cast<int64_t>(tile_count(a.M, G::TM)) * tile_count(a.N, G::TN);
  const dim3 grid(static_cast<unsigned>((T + kXcds - 1) / kXcds * kXcds), static_cast<unsigned>(parts));
  hipLaunchKernelGGL((f8_gemm_tile_kernel<false, 1, 2, 1, true>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

// Adds the parts' sums, in their order, and finishes D: four columns of a row per thread.
template <bool kBf16>
__global__ __launch_bounds__(256) void f8_join_kernel(MxGemmArgs a, const float* sums, int parts, int32_t pitch) {
  const int32_t fours = pitch / 4;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x, row = i / static_cast<uint32_t>(fours);
  if (row >= static_cast<uint32_t>(a.M)) return;
  const int32_t col = static_cast<int32_t>(i - row * static_cast<uint32_t>(fours)) * 4;
  const float* s = sums + static_cast<int64_t>(row) * pitch + col;
  const int64_t next = static_cast<int64_t>(a.M) * pitch;
  f32x4 v = *reinterpret_cast<const f32x4*>(s);
#pragma unroll 4
  for (int k = 1; k < parts; ++k) v += *reinterpret_cast<const f32x4*>(s + k * next);
  store_four<kBf16>(a, 0, row, col, a.N - col, wide_rows<kBf16>(a), v);
}

}  // namespace f8

hipError_t launch_f8_gemm_split(const MxGemmArgs& a, int parts, float* sums, int64_t pitch, hipStream_t st) {
  // (a part without any K would not end)
  if (parts < 1 || (parts - 1) * f8_part(a.K, parts) >= a.K) return hipErrorInvalidValue;
  const hipError_t e = f8::split_sums(a, parts, sums, pitch, st);
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<unsigned>((a.M * (pitch / 4) + 255) / 256));
  if (a.out_bf16)
    hipLaunchKernelGGL((f8::f8_join_kernel<true>), grid, dim3(256), 0, st, a, sums, parts, static_cast<int32_t>(pitch));
  else
    hipLaunchKernelGGL((f8::f8_join_kernel<false>), grid, dim3(256), 0, st, a, sums, parts, static_cast<int32_t>(pitch));
  return hipGetLastError();
}

hipError_t launch_f8_gemm_tile(int size, const MxGemmArgs& a, hipStream_t st) {
  if (size == 64) return a.out_bf16 ? f8::tile_t<true, 1, 2>(a, st) : f8::tile_t<false, 1, 2>(a, st);
  if (size == 256) return a.out_bf16 ? f8::tile_t<true, 4, 4>(a, st) : f8::tile_t<false, 4, 4>(a, st);
  return a.out_bf16 ? f8::tile_t<true, 2, 2>(a, st) : f8::tile_t<false, 2, 2>(a, st);
}

}  // namespace dg
