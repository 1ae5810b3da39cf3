// Host side of the low-precision operators: argument checks and the C ABI
// declared in include/distgemm_mx.h.
#include "../../include/distgemm_mx.h"

#include <cmath>
#include <new>
#include <string>

#include "mx_common.h"

namespace {

thread_local std::string g_mx_error = "no error";

int fail(std::string* where, int code, const char* msg) {
  try {
    (where ? *where : g_mx_error) = std::string(dist_gemm_status_string(code)) + ": " + msg;
  } catch (...) {  // no memory for the message: the code still says what happened
  }
  return code;
}

int hip_status(std::string* where, hipError_t e, const char* what) {
  if (e == hipSuccess) return DIST_GEMM_OK;
  try {
    const std::string msg = std::string(what) + ": " + hipGetErrorName(e) + " (" + hipGetErrorString(e) + ")";
    return fail(where, DIST_GEMM_ERR_HIP, msg.c_str());
  } catch (...) {
    return DIST_GEMM_ERR_HIP;
  }
}

bool aligned(const void* p, uint64_t to) { return (reinterpret_cast<uint64_t>(p) & (to - 1)) == 0; }
bool is_elem(int e) { return e == DIST_GEMM_ELEM_F32 || e == DIST_GEMM_ELEM_BF16; }
bool is_format(int f) { return f == DIST_GEMM_MX_E2M1 || f == DIST_GEMM_MX_E4M3; }
uint64_t elem_bytes(int e) { return e == DIST_GEMM_ELEM_F32 ? 4 : 2; }

#define MX_INVALID(cond, msg) \
  if (cond) return fail(nullptr, DIST_GEMM_ERR_INVALID_ARG, msg)
#define MX_SHAPE(cond, msg) \
  if (cond) return fail(nullptr, DIST_GEMM_ERR_SHAPE, msg)

// the checks that quantising and dequantising share
int check_mx(const void* plain, int64_t ld, int elem, int64_t rows, int64_t cols, int format, const void* codes,
             const void* scales) {
  MX_INVALID(!is_elem(elem), "unknown element type");
  MX_INVALID(!is_format(format), "unknown MX format");
  MX_INVALID(rows < 0 || cols < 1, "rows must be >= 0 and cols >= 1");
  MX_SHAPE(cols % dg::kMxBlock != 0, "cols must be a multiple of 32");
  MX_SHAPE(rows > INT32_MAX || cols > INT32_MAX, "rows and cols must be < 2^31");
  MX_SHAPE(ld < cols, "the leading dimension is smaller than cols");
  if (rows == 0) return DIST_GEMM_OK;
  MX_INVALID(!plain || !codes || !scales, "null pointer");
  MX_INVALID(!aligned(plain, elem_bytes(elem)), "the plain matrix is not aligned to its element");
  MX_INVALID(!aligned(codes, 16) || !aligned(scales, 16), "codes and scales must be 16-byte aligned");
  MX_INVALID(codes == plain || scales == plain || codes == scales, "codes, scales and the plain matrix must not alias");
  return DIST_GEMM_OK;
}

}  // namespace

struct dist_gemm_mx_plan_s {
  int64_t M = 0, N = 0, K = 0, groups = 0;
  int a_format = 0, out_elem = 0;
  int device = 0, cus = 256;
  std::string err = "no error";
};

extern "C" {

const char* dist_gemm_mx_last_error(dist_gemm_mx_plan_t plan) { return plan ? plan->err.c_str() : g_mx_error.c_str(); }

int64_t dist_gemm_mx_scale_pitch(int64_t cols) {
  return cols < 1 || cols % dg::kMxBlock != 0 ? 0 : dg::scale_pitch(cols);
}

int dist_gemm_mx_quantize(const void* x, int64_t ldx, int elem, int64_t rows, int64_t cols, int format, void* codes,
                          void* scales, void* stream) {
  const int rc = check_mx(x, ldx, elem, rows, cols, format, codes, scales);
  if (rc != DIST_GEMM_OK || rows == 0) return rc;
  const dg::QuantizeArgs a{x, ldx, rows, cols, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales)};
  return hip_status(nullptr, dg::launch_mx_quantize(elem, format, a, static_cast<hipStream_t>(stream)), "quantize launch");
}

int dist_gemm_mx_dequantize(const void* codes, const void* scales, int format, int64_t rows, int64_t cols, void* y,
                            int64_t ldy, int elem, void* stream) {
  const int rc = check_mx(y, ldy, elem, rows, cols, format, codes, scales);
  if (rc != DIST_GEMM_OK || rows == 0) return rc;
  const dg::DequantizeArgs a{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), rows, cols, y, ldy};
  return hip_status(nullptr, dg::launch_mx_dequantize(elem, format, a, static_cast<hipStream_t>(stream)),
                    "dequantize launch");
}

int dist_gemm_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, int elem,
                       int64_t rows, int64_t cols, float eps, int out, float scale, void* y, int64_t ldy, void* scales,
                       void* h, int64_t ldh, float* rstd, void* stream) {
  MX_INVALID(!is_elem(elem), "unknown element type");
  MX_INVALID(out < DIST_GEMM_NORM_SAME || out > DIST_GEMM_NORM_MX_E4M3, "unknown output kind");
  MX_INVALID(rows < 0 || cols < 1, "rows must be >= 0 and cols >= 1");
  MX_INVALID(!(eps >= 0.0f) || !std::isfinite(eps), "eps must be finite and >= 0");
  MX_INVALID((residual == nullptr) != (h == nullptr), "residual and h go together");
  const bool mx = out == DIST_GEMM_NORM_MX_E2M1 || out == DIST_GEMM_NORM_MX_E4M3;
  MX_SHAPE(cols > dg::kNormMaxCols, "cols must be <= 32768");
  MX_SHAPE(rows > INT32_MAX, "rows must be < 2^31");
  MX_SHAPE(mx && cols % dg::kMxBlock != 0, "cols must be a multiple of 32 for an MX output");
  MX_SHAPE(ldx < cols || (residual && (ldr < cols || ldh < cols)) || (!mx && ldy < cols),
           "a leading dimension is smaller than cols");
  MX_INVALID(out == DIST_GEMM_NORM_E4M3 && (!std::isfinite(scale) || !(scale > 0.0f)), "scale must be finite and positive");
  MX_INVALID(out == DIST_GEMM_NORM_E4M3 && !std::isfinite(1.0f / scale), "1 / scale must be finite");
  if (rows == 0) return DIST_GEMM_OK;
  MX_INVALID(!x || !weight || !y || (mx && !scales), "null pointer");
  const uint64_t es = elem_bytes(elem);
  MX_INVALID(!aligned(x, es) || !aligned(weight, es) || !aligned(residual, es) || !aligned(h, es) || !aligned(rstd, 4) ||
                 (out == DIST_GEMM_NORM_SAME && !aligned(y, es)),
             "a pointer is not aligned to its element");
  MX_INVALID(mx && (!aligned(y, 16) || !aligned(scales, 16)), "codes and scales must be 16-byte aligned");
  MX_INVALID((h && h == x && ldh != ldx) || (h && h == residual && ldh != ldr) ||
                 (out == DIST_GEMM_NORM_SAME && ((y == x && ldy != ldx) || (y == residual && ldy != ldr))),
             "an output that is an input needs its leading dimension");
  MX_INVALID(y == weight || h == weight || (h && h == y), "outputs must not alias the weight or each other");
  MX_INVALID(out != DIST_GEMM_NORM_SAME && (y == x || y == residual), "an 8- or 4-bit output must not alias an input");
  const void* const others[] = {x, residual, weight, y, h};
  for (const void* p : others)
    MX_INVALID(p && (p == rstd || (mx && p == scales)), "rstd and scales must not alias another argument");
  MX_INVALID(mx && rstd && rstd == scales, "rstd must not alias the scales");
  dg::NormArgs a{};
  a.x = x; a.residual = residual; a.weight = weight; a.y = y; a.h = h; a.rstd = rstd;
  a.scales = static_cast<uint8_t*>(scales);
  a.ldx = ldx; a.ldr = ldr; a.ldy = ldy; a.ldh = ldh;
  a.rows = rows; a.cols = static_cast<int32_t>(cols);
  a.eps = eps; a.inv_scale = out == DIST_GEMM_NORM_E4M3 ? 1.0f / scale : 1.0f;
  return hip_status(nullptr, dg::launch_rms_norm(elem, out, a, static_cast<hipStream_t>(stream)), "rms_norm launch");
}

int64_t dist_gemm_rms_norm_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > dg::kNormMaxCols) return 0;
  // (at least one row, so that rows = 0 also has a place to pass)
  return dg::rms_norm_backward_blocks(rows < 1 ? 1 : rows, cols) * cols * 4;
}

int dist_gemm_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* dh, int64_t lddh,
                                const float* rstd, const void* weight, int elem, int64_t rows, int64_t cols, void* dx,
                                int64_t lddx, float* dweight, void* workspace, int64_t workspace_bytes, void* stream) {
  MX_INVALID(!is_elem(elem), "unknown element type");
  MX_INVALID(rows < 0 || cols < 1, "rows must be >= 0 and cols >= 1");
  MX_SHAPE(cols > dg::kNormMaxCols, "cols must be <= 32768");
  MX_SHAPE(rows > INT32_MAX, "rows must be < 2^31");
  MX_SHAPE(lddy < cols || ldh < cols || lddx < cols || (dh && lddh < cols), "a leading dimension is smaller than cols");
  MX_INVALID(!dweight || !aligned(dweight, 4), "dweight is null or misaligned");
  const uint64_t es = elem_bytes(elem);
  if (rows > 0) {
    MX_INVALID(!dy || !h || !rstd || !weight || !dx, "null pointer");
    MX_INVALID(!aligned(dy, es) || !aligned(h, es) || !aligned(dh, es) || !aligned(dx, es) || !aligned(weight, es) ||
                   !aligned(rstd, 4),
               "a pointer is not aligned to its element");
    MX_INVALID((dx == dy && lddx != lddy) || (dx == h && lddx != ldh) || (dh && dx == dh && lddx != lddh),
               "dx on an input needs its leading dimension");
    MX_INVALID(dx == weight || dx == rstd || dweight == rstd || dweight == weight || dweight == dx || dweight == dy ||
                   dweight == h || (dh && dweight == dh),
               "dweight must not alias an input, nor dx the weight or rstd");
    MX_INVALID(!workspace || !aligned(workspace, 16), "the workspace is null or misaligned");
    const void* const others[] = {dy, h, dh, rstd, weight, dx, dweight};
    for (const void* p : others) MX_INVALID(p == workspace, "the workspace must not alias another argument");
    MX_INVALID(workspace_bytes < dist_gemm_rms_norm_workspace(rows, cols), "the workspace is too small");
  }
  dg::NormBackwardArgs a{};
  a.dy = dy; a.h = h; a.dh = dh; a.rstd = rstd; a.weight = weight; a.dx = dx; a.dweight = dweight;
  a.partial = static_cast<float*>(workspace);
  a.lddy = lddy; a.ldh = ldh; a.lddh = lddh; a.lddx = lddx;
  a.rows = rows; a.cols = static_cast<int32_t>(cols);
  return hip_status(nullptr, dg::launch_rms_norm_backward(elem, a, static_cast<hipStream_t>(stream)),
                    "rms_norm_backward launch");
}

int dist_gemm_mx_plan(int64_t M, int64_t N, int64_t K, int64_t groups, int a_format, int out_elem,
                      dist_gemm_mx_plan_t* out) {
  MX_INVALID(!out, "out is NULL");
  *out = nullptr;
  MX_INVALID(M < 1 || N < 1 || K < 1 || groups < 0, "M, N, K must be >= 1 and groups >= 0");
  MX_INVALID(!is_format(a_format), "unknown MX format");
  MX_INVALID(!is_elem(out_elem), "unknown element type");
  MX_SHAPE(M > INT32_MAX || N > INT32_MAX, "M and N must be < 2^31");
  MX_SHAPE(K % dg::kMxBlock != 0, "K must be a multiple of 32");
  MX_SHAPE(K > (1 << 22), "K must be <= 2^22");
  MX_SHAPE(groups > 65535, "groups must be <= 65535");
  dist_gemm_mx_plan_s* p = new (std::nothrow) dist_gemm_mx_plan_s;
  if (!p) return fail(nullptr, DIST_GEMM_ERR_OOM, "no host memory for the plan");
  p->M = M; p->N = N; p->K = K; p->groups = groups; p->a_format = a_format; p->out_elem = out_elem;
  hipError_t e = hipGetDevice(&p->device);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&p->cus, hipDeviceAttributeMultiprocessorCount, p->device);
  if (e != hipSuccess) {
    delete p;
    return hip_status(nullptr, e, "device query");
  }
  *out = p;
  return DIST_GEMM_OK;
}

int dist_gemm_mx_run(dist_gemm_mx_plan_t P, int64_t rows, const void* A, const void* A_scales, const void* B,
                     const void* B_scales, const void* C, int64_t ldc, void* D, int64_t ldd, const void* bias,
                     const int32_t* offsets, float alpha, float beta, void* stream) {
  if (!P) return fail(nullptr, DIST_GEMM_ERR_INVALID_ARG, "plan is NULL");
  auto invalid = [&](const char* msg) { return fail(&P->err, DIST_GEMM_ERR_INVALID_ARG, msg); };
  auto shape = [&](const char* msg) { return fail(&P->err, DIST_GEMM_ERR_SHAPE, msg); };
  if (rows < 0) return invalid("rows must be >= 0");
  if (rows > P->M) return shape("more rows than the plan's M");
  if (!std::isfinite(alpha) || !std::isfinite(beta)) return invalid("alpha and beta must be finite");
  if (ldd < P->N || (beta != 0.0f && ldc < P->N)) return shape("a leading dimension is smaller than N");
  if ((offsets != nullptr) != (P->groups > 0)) return invalid("offsets go with a plan that has groups");
  if (rows == 0) return DIST_GEMM_OK;
  if (!A || !A_scales || !B || !B_scales || !D) return invalid("null pointer");
  if (beta != 0.0f && !C) return invalid("C is NULL and beta is not 0");
  if (!aligned(A, 16) || !aligned(A_scales, 16) || !aligned(B, 16) || !aligned(B_scales, 16))
    return invalid("codes and scales must be 16-byte aligned");
  const uint64_t es = elem_bytes(P->out_elem);
  if (!aligned(D, es) || (beta != 0.0f && !aligned(C, es)) || !aligned(bias, es) || !aligned(offsets, 4))
    return invalid("a pointer is not aligned to its element");
  if (D == A || D == A_scales || D == B || D == B_scales || D == bias || D == offsets)
    return invalid("D must not alias an operand");
  if (beta != 0.0f && C == D && ldc != ldd) return invalid("D on C needs its leading dimension");
  dg::MxGemmArgs a{};
  a.A = static_cast<const uint8_t*>(A); a.As = static_cast<const uint8_t*>(A_scales);
  a.B = static_cast<const uint8_t*>(B); a.Bs = static_cast<const uint8_t*>(B_scales);
  a.C = beta != 0.0f ? C : nullptr; a.bias = bias; a.D = D; a.offsets = offsets;
  a.ldc = ldc; a.ldd = ldd;
  a.M = static_cast<int32_t>(rows); a.N = static_cast<int32_t>(P->N); a.K = static_cast<int32_t>(P->K);
  a.groups = static_cast<int32_t>(P->groups);
  a.a_format = P->a_format; a.out_bf16 = P->out_elem == DIST_GEMM_ELEM_BF16;
  a.cus = P->cus;
  a.alpha = alpha; a.beta = beta;
  int prev = P->device;
  (void)hipGetDevice(&prev);
  if (prev != P->device) (void)hipSetDevice(P->device);
  const hipError_t e = dg::launch_mx_gemm(a, static_cast<hipStream_t>(stream));
  if (prev != P->device) (void)hipSetDevice(prev);
  return hip_status(&P->err, e, "mx product launch");
}

int dist_gemm_mx_destroy(dist_gemm_mx_plan_t plan) {
  delete plan;
  return DIST_GEMM_OK;
}

}  // extern "C"
