// MX product on square tiles, for many rows of A (mx_tile_loop.h has the main
// loop).
//
// Rates.  16384 x 13312 x 16384 E2M1: 1575 .. 1620 us, 4.4 .. 4.5 PFLOP/s, 70%
// of what MFMAs alone reach on random data (6.5): the MFMA pipe is busy 65% of
// the cycles at 1.8 GHz (power), waits take 24%.  E4M3: 2510 us, 2.85 PFLOP/s
// (MFMAs alone 4.0).  By group, 8192 rows x 16 x 4096 x 4096 E4M3: 148 us (E2M1
// 108); a round of tiles takes 47 and the last one, here half empty, as long as
// the others.  What is not whole bf16 columns without C goes four columns of a row
// at a time, C and bias by single elements: 4096 x 8192 x 4096 E2M1 76 us, with a
// bias 90, into fp32 109, with C 162 (171).
//
// Precision.  The matrix cores add the products of eight consecutive elements
// to 2^-13 of the largest one's power of two and cut off what lies below (measured
// on both MFMAs of these products); from there on sums are fp32.  E2M1 products,
// from 1/4 to 36, are all within that: exact.  E4M3 elements spread over 2^17, and
// their products' sums are off by 4e-6 to 6e-6 of the result's rms with normal data,
// 1.4e-5 to 2e-5 with one in a hundred columns of K 16 times as loud, for any
// K, without a bias to one side (an fp32 product: 3e-8).  It is the price
// of the 8-bit rate, a hundredth of what rounding D to bf16 costs.
#include "mx_tile_loop.h"

namespace dg {
namespace mx {

template <bool A8, bool kBf16, int NBM, int NBN, int KG>
__global__ __launch_bounds__(256 * KG) __attribute__((amdgpu_waves_per_eu(NBM* NBN == 16 ? 1 : 2, NBM* NBN == 16 ? 1 : 2)))
void mx_gemm_tile_kernel(MxGemmArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[KG * Geo<A8, false, NBM, NBN>::kLds];
  run_tiles<A8, false, kBf16, NBM, NBN, KG>(p, smem);
}

template <bool A8, bool kBf16, int NBM, int NBN>
static hipError_t tile_t(const MxGemmArgs& a, hipStream_t st) {
  using G = Geo<A8, false, NBM, NBN>;
  const int64_t row_tiles = a.offsets ? most_group_tiles(a.M, a.groups, G::TM) : tile_count(a.M, G::TM);
  const int64_t T = row_tiles * tile_count(a.N, G::TN);
  if (T > INT32_MAX / 2) return hipErrorInvalidConfiguration;
  const int64_t most = static_cast<int64_t>(a.cus) * G::kWgs;
  const int64_t grid = ((T < most ? T : most) + kXcds - 1) / kXcds * kXcds;
  const dim3 wgs(static_cast<unsigned>(grid));
  if constexpr (NBM * NBN < 16) {
    if (T <= a.cus && a.K > 4096) {  // "Few tiles" above
      hipLaunchKernelGGL((mx_gemm_tile_kernel<A8, kBf16, NBM, NBN, 2>), wgs, dim3(512), 0, st, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((mx_gemm_tile_kernel<A8, kBf16, NBM, NBN, 1>), wgs, dim3(256), 0, st, a);
  return hipGetLastError();
}

template <int NBM, int NBN>
static hipError_t tile_type(const MxGemmArgs& a, hipStream_t st) {
  if (a.a_format == MX_E4M3)
    return a.out_bf16 ? tile_t<true, true, NBM, NBN>(a, st) : tile_t<true, false, NBM, NBN>(a, st);
  return a.out_bf16 ? tile_t<false, true, NBM, NBN>(a, st) : tile_t<false, false, NBM, NBN>(a, st);
}

}  // namespace mx

hipError_t launch_mx_gemm_tile(int size, const MxGemmArgs& a, hipStream_t st) {
  return size == 256 ? mx::tile_type<4, 4>(a, st) : mx::tile_type<2, 2>(a, st);
}

}  // namespace dg
