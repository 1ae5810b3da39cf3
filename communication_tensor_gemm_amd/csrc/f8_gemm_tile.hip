// F8 product on square tiles, for many rows of A (mx_tile_loop.h has the main
// loop).
#include "f8_common.h"
#include "mx_tile_loop.h"

namespace dg {
namespace f8 {

template <bool kBf16, int NBM, int NBN, int KG>
__global__ __launch_bounds__(256 * KG) __attribute__((amdgpu_waves_per_eu(NBM* NBN == 16 ? 1 : 2, NBM* NBN == 16 ? 1 : 2)))
void f8_gemm_tile_kernel(MxGemmArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[KG * Geo<true, true, NBM, NBN>::kLds];
  run_tiles<true, true, kBf16, NBM, NBN, KG>(p, smem);
}

template <bool kBf16, int NBM, int NBN>
static hipError_t tile_t(const MxGemmArgs& a, hipStream_t st) {
  using G = Geo<true, true, NBM, NBN>;
  const int64_t T = static_cast<int64_t>(tile_count(a.M, G::TM)) * tile_count(a.N, G::TN);
  if (T > INT32_MAX / 2) return hipErrorInvalidConfiguration;
  const int64_t most = static_cast<int64_t>(a.cus) * G::kWgs;
  const int64_t grid = ((T < most ? T : most) + kXcds - 1) / kXcds * kXcds;
  const dim3 wgs(static_cast<unsigned>(grid));
  if constexpr (NBM * NBN < 16) {
    if (T <= a.cus && a.K > 4096) {
      hipLaunchKernelGGL((f8_gemm_tile_kernel<kBf16, NBM, NBN, 2>), wgs, dim3(512), 0, st, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((f8_gemm_tile_kernel<kBf16, NBM, NBN, 1>), wgs, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace f8

hipError_t launch_f8_gemm_tile(int size, const MxGemmArgs& a, hipStream_t st) {
  if (size == 256) return a.out_bf16 ? f8::tile_t<true, 4, 4>(a, st) : f8::tile_t<false, 4, 4>(a, st);
  return a.out_bf16 ? f8::tile_t<true, 2, 2>(a, st) : f8::tile_t<false, 2, 2>(a, st);
}

}  // namespace dg
