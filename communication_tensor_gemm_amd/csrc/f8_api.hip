// Host side of the 8-bit training operators: argument checks and the C ABI
// declared in include/distgemm_f8.h.
#include "../../include/distgemm_f8.h"

#include <atomic>
#include <cmath>
#include <initializer_list>
#include <string>

#include "f8_common.h"

namespace {

thread_local std::string g_f8_error = "no error";

int fail(int code, const char* msg) {
  try {
    g_f8_error = std::string(dist_gemm_status_string(code)) + ": " + msg;
  } catch (...) {  // no memory for the message: the code still says what happened
  }
  return code;
}

int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return DIST_GEMM_OK;
  try {
    const std::string msg = std::string(what) + ": " + hipGetErrorName(e) + " (" + hipGetErrorString(e) + ")";
    return fail(DIST_GEMM_ERR_HIP, msg.c_str());
  } catch (...) {
    return DIST_GEMM_ERR_HIP;
  }
}

bool aligned(const void* p, uint64_t to) { return (reinterpret_cast<uint64_t>(p) & (to - 1)) == 0; }
bool is_elem(int e) { return e == DIST_GEMM_ELEM_F32 || e == DIST_GEMM_ELEM_BF16; }
uint64_t elem_bytes(int e) { return e == DIST_GEMM_ELEM_F32 ? 4 : 2; }

// Whether an output (not NULL) starts at another argument's address.
bool among(const void* out, std::initializer_list<const void*> others) {
  for (const void* p : others)
    if (out && p == out) return true;
  return false;
}

// CUs of the current device, asked for once per device.
int current_cus(int* cus) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return hip_status(e, "device query");
  if (device < kDevices && (*cus = known[device].load(std::memory_order_relaxed)) > 0) return DIST_GEMM_OK;
  e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, device);
  if (e != hipSuccess) return hip_status(e, "device query");
  if (device < kDevices) known[device].store(*cus, std::memory_order_relaxed);
  return DIST_GEMM_OK;
}

#define F8_INVALID(cond, msg) \
  if (cond) return fail(DIST_GEMM_ERR_INVALID_ARG, msg)
#define F8_SHAPE(cond, msg) \
  if (cond) return fail(DIST_GEMM_ERR_SHAPE, msg)

constexpr int64_t kMost = INT32_MAX / dg::kF8Block * dg::kF8Block;  // the widest row whose pitch is below 2^31

// the sizes of an F8 tensor and, with it, of its transpose
int check_size(int64_t rows, int64_t cols) {
  F8_INVALID(rows < 0 || cols < 1, "rows must be >= 0 and cols >= 1");
  F8_SHAPE(rows > kMost || cols > kMost, "rows and cols, rounded up to 128, must be < 2^31");
  F8_SHAPE(dg::f8_blocks(rows) * dg::f8_blocks(cols) > INT32_MAX, "2^31 or more blocks of 128 x 128");
  return DIST_GEMM_OK;
}

}  // namespace

extern "C" {

const char* dist_gemm_f8_last_error(void) { return g_f8_error.c_str(); }

int64_t dist_gemm_f8_pitch(int64_t cols) { return cols < 1 || cols > kMost ? 0 : dg::f8_pitch(cols); }

int64_t dist_gemm_f8_scale_pitch(int64_t cols) { return cols < 1 || cols > kMost ? 0 : dg::f8_scale_pitch(cols); }

int dist_gemm_f8_quantize(const void* x, int64_t ldx, int elem, int64_t rows, int64_t cols, int block_rows, void* codes,
                          void* scales, void* codes_t, void* scales_t, void* stream) {
  F8_INVALID(!is_elem(elem), "unknown element type");
  F8_INVALID(block_rows != 1 && block_rows != dg::kF8Block, "block_rows must be 1 or 128");
  const int rc = check_size(rows, cols);
  if (rc != DIST_GEMM_OK) return rc;
  F8_SHAPE(ldx < cols, "the leading dimension is smaller than cols");
  if (rows == 0) return DIST_GEMM_OK;
  F8_INVALID((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr),
             "codes and their scales go together");
  F8_INVALID(!x || (!codes && !codes_t), "null pointer");
  F8_INVALID(!aligned(x, elem_bytes(elem)), "x is not aligned to its element");
  F8_INVALID(!aligned(codes, 16) || !aligned(scales, 16) || !aligned(codes_t, 16) || !aligned(scales_t, 16),
             "codes and scales must be 16-byte aligned");
  F8_INVALID(among(codes, {x, scales, codes_t, scales_t}) || among(scales, {x, codes_t, scales_t}) ||
                 among(codes_t, {x, scales_t}) || among(scales_t, {x}),
             "codes, scales and x must not alias");
  dg::F8QuantizeArgs a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.cols = cols;
  a.codes = static_cast<uint8_t*>(codes); a.scales = static_cast<uint8_t*>(scales);
  a.codes_t = static_cast<uint8_t*>(codes_t); a.scales_t = static_cast<uint8_t*>(scales_t);
  a.square = block_rows != 1;
  return hip_status(dg::launch_f8_quantize(elem, a, static_cast<hipStream_t>(stream)), "quantize launch");
}

int dist_gemm_f8_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols, void* y, int64_t ldy,
                            int elem, void* stream) {
  F8_INVALID(!is_elem(elem), "unknown element type");
  const int rc = check_size(rows, cols);
  if (rc != DIST_GEMM_OK) return rc;
  F8_SHAPE(ldy < cols, "the leading dimension is smaller than cols");
  if (rows == 0) return DIST_GEMM_OK;
  F8_INVALID(!codes || !scales || !y, "null pointer");
  F8_INVALID(!aligned(y, elem_bytes(elem)), "y is not aligned to its element");
  F8_INVALID(!aligned(codes, 16) || !aligned(scales, 16), "codes and scales must be 16-byte aligned");
  F8_INVALID(among(y, {codes, scales}), "y must not alias codes or scales");
  const dg::F8DequantizeArgs a{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), rows, cols, y, ldy};
  return hip_status(dg::launch_f8_dequantize(elem, a, static_cast<hipStream_t>(stream)), "dequantize launch");
}

int dist_gemm_f8_transpose(const void* codes, const void* scales, int64_t rows, int64_t cols, void* codes_t,
                           void* scales_t, void* stream) {
  const int rc = check_size(rows, cols);
  if (rc != DIST_GEMM_OK) return rc;
  if (rows == 0) return DIST_GEMM_OK;
  F8_INVALID(!codes || !scales || !codes_t || !scales_t, "null pointer");
  F8_INVALID(!aligned(codes, 16) || !aligned(scales, 16) || !aligned(codes_t, 16) || !aligned(scales_t, 16),
             "codes and scales must be 16-byte aligned");
  F8_INVALID(among(codes_t, {codes, scales, scales_t}) || among(scales_t, {codes, scales}),
             "the transposed tensor must not alias the other");
  dg::F8QuantizeArgs a{};
  a.x = codes; a.x_scales = static_cast<const uint8_t*>(scales);
  a.ldx = dg::f8_pitch(cols); a.rows = rows; a.cols = cols;
  a.codes_t = static_cast<uint8_t*>(codes_t); a.scales_t = static_cast<uint8_t*>(scales_t);
  return hip_status(dg::launch_f8_transpose(a, static_cast<hipStream_t>(stream)), "transpose launch");
}

static bool product_size(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && M <= INT32_MAX && N >= 1 && N <= INT32_MAX && K >= dg::kF8Block && K % dg::kF8Block == 0 && K <= (1 << 22);
}

int64_t dist_gemm_f8_product_workspace(int64_t M, int64_t N, int64_t K) {
  int cus = 0;
  if (!product_size(M, N, K) || current_cus(&cus) != DIST_GEMM_OK) return 0;
  return dg::f8_gemm_workspace(M, N, K, cus);
}

int dist_gemm_f8_product(const void* A, const void* A_scales, const void* B, const void* B_scales, int64_t M, int64_t N,
                         int64_t K, const void* C, int64_t ldc, void* D, int64_t ldd, int out_elem, const void* bias,
                         float alpha, float beta, void* workspace, int64_t workspace_bytes, void* stream) {
  F8_INVALID(!is_elem(out_elem), "unknown element type");
  F8_INVALID(M < 0, "M must be >= 0");
  F8_SHAPE(!product_size(M, N, K), "M and N must be < 2^31, N at least 1, K a multiple of 128 in 128 .. 2^22");
  F8_INVALID(!std::isfinite(alpha) || !std::isfinite(beta), "alpha and beta must be finite");
  F8_SHAPE(ldd < N || (beta != 0.0f && ldc < N), "a leading dimension is smaller than N");
  if (M == 0) return DIST_GEMM_OK;
  F8_INVALID(!A || !A_scales || !B || !B_scales || !D, "null pointer");
  F8_INVALID(beta != 0.0f && !C, "C is NULL and beta is not 0");
  F8_INVALID(!aligned(A, 16) || !aligned(A_scales, 16) || !aligned(B, 16) || !aligned(B_scales, 16),
             "codes and scales must be 16-byte aligned");
  const uint64_t es = elem_bytes(out_elem);
  F8_INVALID(!aligned(D, es) || (beta != 0.0f && !aligned(C, es)) || !aligned(bias, es),
             "a pointer is not aligned to its element");
  F8_INVALID(among(D, {A, A_scales, B, B_scales, bias}), "D must not alias an operand");
  F8_INVALID(beta != 0.0f && C == D && ldc != ldd, "D on C needs its leading dimension");
  int cus = 0;
  const int rc = current_cus(&cus);
  if (rc != DIST_GEMM_OK) return rc;
  const int64_t need = dg::f8_gemm_workspace(M, N, K, cus);
  if (need > 0) {
    F8_INVALID(!workspace || !aligned(workspace, 16), "the workspace is null or misaligned");
    F8_INVALID(workspace_bytes < need, "the workspace is too small");
    F8_INVALID(among(workspace, {A, A_scales, B, B_scales, beta != 0.0f ? C : nullptr, D, bias}),
               "the workspace must not alias another argument");
  }
  dg::MxGemmArgs a{};
  a.A = static_cast<const uint8_t*>(A); a.As = static_cast<const uint8_t*>(A_scales);
  a.B = static_cast<const uint8_t*>(B); a.Bs = static_cast<const uint8_t*>(B_scales);
  a.C = beta != 0.0f ? C : nullptr; a.bias = bias; a.D = D;
  a.ldc = ldc; a.ldd = ldd;
  a.M = static_cast<int32_t>(M); a.N = static_cast<int32_t>(N); a.K = static_cast<int32_t>(K);
  a.a_format = dg::MX_E4M3; a.out_bf16 = out_elem == DIST_GEMM_ELEM_BF16;
  a.cus = cus;
  a.alpha = alpha; a.beta = beta;
  return hip_status(dg::launch_f8_gemm(a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream)), "product launch");
}

int dist_gemm_layer_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                         const void* bias, int elem, int64_t rows, int64_t cols, float eps, int out, float scale, void* y,
                         int64_t ldy, void* scales, void* h, int64_t ldh, float* mean, float* rstd, void* kept,
                         void* kept_scales, void* stream) {
  F8_INVALID(!is_elem(elem), "unknown element type");
  F8_INVALID(out < DIST_GEMM_LAYER_NORM_SAME || out > DIST_GEMM_LAYER_NORM_F8, "unknown output kind");
  F8_INVALID(rows < 0 || cols < 1, "rows must be >= 0 and cols >= 1");
  F8_INVALID(!(eps >= 0.0f) || !std::isfinite(eps), "eps must be finite and >= 0");
  F8_INVALID((residual == nullptr) != (h == nullptr), "residual and h go together");
  F8_INVALID((kept == nullptr) != (kept_scales == nullptr), "kept and kept_scales go together");
  const bool f8 = out == DIST_GEMM_LAYER_NORM_F8, same = out == DIST_GEMM_LAYER_NORM_SAME;
  F8_SHAPE(cols > dg::kNormMaxCols, "cols must be <= 32768");
  F8_SHAPE(rows > INT32_MAX, "rows must be < 2^31");
  F8_SHAPE(ldx < cols || (residual && (ldr < cols || ldh < cols)) || (!f8 && ldy < cols),
           "a leading dimension is smaller than cols");
  F8_INVALID(out == DIST_GEMM_LAYER_NORM_E4M3 &&
                 (!std::isfinite(scale) || !(scale > 0.0f) || !std::isfinite(1.0f / scale)),
             "scale and 1 / scale must be finite and positive");
  if (rows == 0) return DIST_GEMM_OK;
  F8_INVALID(!x || !weight || !y || (f8 && !scales), "null pointer");
  const uint64_t es = elem_bytes(elem);
  F8_INVALID(!aligned(x, es) || !aligned(weight, es) || !aligned(bias, es) || !aligned(residual, es) || !aligned(h, es) ||
                 !aligned(mean, 4) || !aligned(rstd, 4) || (same && !aligned(y, es)),
             "a pointer is not aligned to its element");
  F8_INVALID((f8 && (!aligned(y, 16) || !aligned(scales, 16))) || !aligned(kept, 16) || !aligned(kept_scales, 16),
             "codes and scales must be 16-byte aligned");
  F8_INVALID((h && h == x && ldh != ldx) || (h && h == residual && ldh != ldr) ||
                 (same && ((y == x && ldy != ldx) || (y == residual && ldy != ldr))),
             "an output that is an input needs its leading dimension");
  F8_INVALID(among(y, {weight, bias, h}) || among(h, {weight, bias}) || (!same && among(y, {x, residual})),
             "an output must not alias an input (but h and a plain y the stream), nor another output");
  const void* const s = f8 ? scales : nullptr;
  F8_INVALID(among(mean, {x, residual, weight, bias, y, h, rstd, s, kept, kept_scales}) ||
                 among(rstd, {x, residual, weight, bias, y, h, s, kept, kept_scales}) ||
                 among(s, {x, residual, weight, bias, y, h, kept, kept_scales}) ||
                 among(kept, {x, residual, weight, bias, y, h, kept_scales}) ||
                 among(kept_scales, {x, residual, weight, bias, y, h}),
             "mean, rstd, scales and what is kept must not alias another argument");
  dg::LayerNormArgs a{};
  a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.y = y; a.h = h; a.mean = mean; a.rstd = rstd;
  a.scales = static_cast<uint8_t*>(scales);
  a.kept = static_cast<uint8_t*>(kept); a.kept_scales = static_cast<uint8_t*>(kept_scales);
  a.ldx = ldx; a.ldr = ldr; a.ldy = ldy; a.ldh = ldh;
  a.rows = rows; a.cols = static_cast<int32_t>(cols);
  a.eps = eps; a.inv_scale = out == DIST_GEMM_LAYER_NORM_E4M3 ? 1.0f / scale : 1.0f;
  return hip_status(dg::launch_layer_norm(elem, out, a, static_cast<hipStream_t>(stream)), "layer_norm launch");
}

int64_t dist_gemm_layer_norm_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > dg::kNormMaxCols) return 0;
  // (at least one row, so that rows = 0 also has a place to pass)
  return dg::layer_norm_backward_blocks(rows < 1 ? 1 : rows, cols) * cols * 8;
}

int dist_gemm_layer_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* h_scales,
                                  const void* dh, int64_t lddh, const float* mean, const float* rstd, const void* weight,
                                  int elem, int64_t rows, int64_t cols, void* dx, int64_t lddx, float* dweight,
                                  float* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
  F8_INVALID(!is_elem(elem), "unknown element type");
  F8_INVALID(rows < 0 || cols < 1, "rows must be >= 0 and cols >= 1");
  F8_SHAPE(cols > dg::kNormMaxCols, "cols must be <= 32768");
  F8_SHAPE(rows > INT32_MAX, "rows must be < 2^31");
  F8_SHAPE(lddy < cols || (!h_scales && ldh < cols) || lddx < cols || (dh && lddh < cols),
           "a leading dimension is smaller than cols");
  F8_INVALID(!dweight || !aligned(dweight, 4) || !aligned(dbias, 4) || dweight == dbias,
             "dweight is null, or dweight or dbias misaligned, or both the same");
  const uint64_t es = elem_bytes(elem);
  if (rows > 0) {
    F8_INVALID(!dy || !h || !rstd || !weight || !dx || (!h_scales && !mean), "null pointer");
    F8_INVALID(!aligned(dy, es) || (!h_scales && !aligned(h, es)) || !aligned(dh, es) || !aligned(dx, es) ||
                   !aligned(weight, es) || !aligned(rstd, 4) || (!h_scales && !aligned(mean, 4)),
               "a pointer is not aligned to its element");
    F8_INVALID(h_scales && (!aligned(h, 16) || !aligned(h_scales, 16)), "codes and scales must be 16-byte aligned");
    F8_INVALID((dx == dy && lddx != lddy) || (!h_scales && dx == h && lddx != ldh) || (dh && dx == dh && lddx != lddh),
               "dx on an input needs its leading dimension");
    const void* const mu = h_scales ? nullptr : mean;
    F8_INVALID(among(dx, {weight, rstd, mu, h_scales}) || (h_scales && dx == h) ||
                   among(dweight, {dy, h, h_scales, dh, mu, rstd, weight, dx}) ||
                   among(dbias, {dy, h, h_scales, dh, mu, rstd, weight, dx}),
               "dweight and dbias must not alias an input, nor dx the weight, the statistics or what was kept");
    F8_INVALID(!workspace || !aligned(workspace, 16), "the workspace is null or misaligned");
    F8_INVALID(among(workspace, {dy, h, h_scales, dh, mu, rstd, weight, dx, dweight, dbias}),
               "the workspace must not alias another argument");
    F8_INVALID(workspace_bytes < dist_gemm_layer_norm_workspace(rows, cols), "the workspace is too small");
  }
  dg::LayerNormBackwardArgs a{};
  a.dy = dy; a.h = h; a.h_scales = static_cast<const uint8_t*>(h_scales); a.dh = dh; a.mean = mean; a.rstd = rstd;
  a.weight = weight; a.dx = dx; a.dweight = dweight; a.dbias = dbias;
  a.partial = static_cast<float*>(workspace);
  a.lddy = lddy; a.ldh = ldh; a.lddh = lddh; a.lddx = lddx;
  a.rows = rows; a.cols = static_cast<int32_t>(cols);
  return hip_status(dg::launch_layer_norm_backward(elem, a, static_cast<hipStream_t>(stream)), "layer_norm_backward launch");
}

}  // extern "C"
