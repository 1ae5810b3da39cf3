/*
 * distgemm_mx.h -- C ABI of the low-precision operators of the MI355X
 * (gfx950) TP-step GEMM library: microscaled (MX) tensors, their products
 * (dense and by group of rows), and the RMS norm that feeds them and the
 * library's e4m3 GEMM.  Same library, status codes and conventions as
 * distgemm.h: device pointers owned by the caller, work enqueued on `stream`
 * (a hipStream_t; NULL = the null stream) and not waited for, no exit or
 * abort, and no device memory allocated by any call of this header.  Every
 * call here only launches kernels, so all of them can be captured into a HIP
 * graph.  Pointers belong to the current HIP device (a plan's: to the device
 * it was made on).  What a call writes must not overlap its other arguments
 * except where this header allows it; two that start at one address are
 * refused (INVALID_ARG).
 *
 * MX tensors (OCP Microscaling Formats v1.0 element and scale types).  A
 * matrix of `rows` x `cols` values, cols a multiple of 32, is
 *   codes : rows x cols elements, row-major without gaps.  E4M3: one byte
 *           each.  E2M1: two per byte, element 2i in the low nibble of byte
 *           i, so a row takes cols / 2 bytes.
 *   scales: one E8M0 byte b per 32 consecutive elements of a row, which
 *           multiplies them by 2^(b - 127); b = 255 makes them NaN.  A row
 *           of scales takes dist_gemm_mx_scale_pitch(cols) bytes: cols / 32
 *           rounded up to a multiple of 16 (for cols a multiple of 512, the
 *           plain rows x cols/32 matrix), so that 512 elements' scales are
 *           one aligned load.  The bytes past cols / 32 are written as zero
 *           and not used.
 * Both start at 16-byte aligned addresses.  Rows are independent, so a shard
 * of consecutive rows is a shard of both arrays, and an all-gather of row
 * shards is an all-gather of each.
 */
#ifndef DISTGEMM_MX_H_
#define DISTGEMM_MX_H_

#include <stdint.h>

#include "distgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Plain element types. */
enum dist_gemm_elem { DIST_GEMM_ELEM_F32 = 0, DIST_GEMM_ELEM_BF16 = 1 };

/* Element formats of an MX tensor. */
enum dist_gemm_mx_format { DIST_GEMM_MX_E2M1 = 0, DIST_GEMM_MX_E4M3 = 1 };

/* What dist_gemm_rms_norm writes to y. */
enum dist_gemm_norm_out {
  DIST_GEMM_NORM_SAME = 0,    /* the type of x */
  DIST_GEMM_NORM_E4M3 = 1,    /* e4m3fn bytes of y / scale, saturating at +-448 */
  DIST_GEMM_NORM_MX_E2M1 = 2, /* an MX tensor */
  DIST_GEMM_NORM_MX_E4M3 = 3
};

/* Bytes of one row of scales; 0 for cols < 1 or not a multiple of 32. */
int64_t dist_gemm_mx_scale_pitch(int64_t cols);

/* Quantise x (rows x cols of `elem`, rows ldx elements apart, ldx >= cols)
 * to an MX tensor.  Per block of 32 with largest magnitude m:
 *   X = max(floor(log2 m) - e, -127), e = 2 (E2M1) or 8 (E4M3),
 *   scale byte X + 127, element = x * 2^-X rounded to nearest even and
 *   saturated (at 6 or 448).
 * An all-zero block has scale byte 0; a block with an infinity or a NaN has
 * scale byte 255 and zero codes (all of its values are NaN).  rows = 0 does
 * nothing.  SHAPE: cols not a multiple of 32, ldx < cols, or a size past
 * 2^31 - 1; INVALID_ARG: a null or misaligned pointer, an unknown enum, a
 * negative size. */
int dist_gemm_mx_quantize(const void* x, int64_t ldx, int elem, int64_t rows, int64_t cols, int format,
                          void* codes, void* scales, void* stream);

/* The values of an MX tensor in `elem`, rows ldy elements apart; exact
 * except where they leave the range of the type (round to nearest even).
 * Errors as dist_gemm_mx_quantize. */
int dist_gemm_mx_dequantize(const void* codes, const void* scales, int format, int64_t rows, int64_t cols,
                            void* y, int64_t ldy, int elem, void* stream);

/* RMS norm of each row, after the residual's addition:
 *   h = x + residual, rounded to `elem` (without a residual, h = x)
 *   s = 1 / sqrt(mean(h^2) + eps)
 *   y = h * s * weight
 * in fp32, y rounded once to what `out` names (the sum of squares too: a row
 * whose sum overflows has s = 0, and with eps = 0 a row of zeros, or one whose
 * squares vanish, s = infinity).  x, residual and h hold
 * `rows` rows of `cols` values of `elem`, ldx, ldr and ldh elements apart,
 * weight `cols` values of `elem`.  residual and h go together (both NULL or
 * neither); h may be x or residual itself (then with the same leading
 * dimension), as may y with out = SAME.  rstd, if not NULL, receives s per
 * row (what the gradient needs).
 *   SAME:    y of `elem`, ldy elements apart.
 *   E4M3:    y bytes, ldy apart: cast_e4m3(y / scale), the operand of an
 *            E4M3 GEMM plan whose scale_a is `scale` (finite, positive).
 *   MX_*:    y the codes and `scales` the scales of an MX tensor (cols a
 *            multiple of 32; ldy is not used).
 * cols <= 32768.  rows = 0 does nothing.  Errors as dist_gemm_mx_quantize. */
int dist_gemm_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                       int elem, int64_t rows, int64_t cols, float eps, int out, float scale, void* y,
                       int64_t ldy, void* scales, void* h, int64_t ldh, float* rstd, void* stream);

/* Bytes of workspace that dist_gemm_rms_norm_backward needs (0 for sizes it
 * refuses). */
int64_t dist_gemm_rms_norm_workspace(int64_t rows, int64_t cols);

/* Gradient of dist_gemm_rms_norm (of the norm before any rounding to 8 or 4
 * bits): with g = dy * weight, n = h * rstd,
 *   dx      = rstd * (g - n * mean(g * n)) + dh      (rounded to `elem`)
 *   dweight = sum over rows of dy * n                (fp32)
 * h is what the forward pass normalised (x, or x + residual) and rstd what
 * it returned; dh, if not NULL, is the gradient that reaches h itself along
 * the residual stream.  dx is the gradient of x and of the residual alike.
 * dx may be dy, h or dh itself (same leading dimension).  workspace: at least
 * dist_gemm_rms_norm_workspace(rows, cols) bytes, 16-byte aligned, not shared
 * with work that may run at the same time.  The result does not depend on
 * timing: no atomics.  rows = 0 sets dweight to zero. */
int dist_gemm_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* dh,
                                int64_t lddh, const float* rstd, const void* weight, int elem, int64_t rows,
                                int64_t cols, void* dx, int64_t lddx, float* dweight, void* workspace,
                                int64_t workspace_bytes, void* stream);

/* Products of MX tensors:
 *   D = alpha * A * B^T + beta * C (+ bias[j])
 * A: rows x K in a_format; B: N x K in E2M1 (the logical K x N operand
 * stored K-contiguous, as in distgemm.h); C, D: rows x N of `out_elem`;
 * bias: N values of out_elem.  Sums are fp32; within eight consecutive
 * elements the matrix cores keep 2^-13 of the largest product's power of two,
 * which E2M1 products never leave (they are exact there) and which costs E4M3
 * ones about 2e-5 of the result's rms.
 *
 * groups > 0: the rows of A come in `groups` groups (a mixture of experts'
 * tokens sorted by expert), and group g is multiplied by its own B (N x K,
 * at B + g * N * K / 2 bytes; scales likewise) and bias (N values from g *
 * N).  `offsets` (device, int32, groups + 1 values) gives group g the rows
 * offsets[g] .. offsets[g + 1] - 1; any group may be empty.  Rows that no
 * group has are not written.  Offsets are read on the device and clamped
 * there to 0 .. rows and to be ascending (one below an earlier one counts as
 * that one: no row is in two groups); nothing waits for them on the host.
 *
 * A plan fixes the problem for calls with up to M rows.  Limits: 1 <= M, N
 * <= 2^31 - 1; K a multiple of 32, 32 <= K <= 2^22; 0 <= groups <= 65535. */
typedef struct dist_gemm_mx_plan_s* dist_gemm_mx_plan_t;

int dist_gemm_mx_plan(int64_t M, int64_t N, int64_t K, int64_t groups, int a_format, int out_elem,
                      dist_gemm_mx_plan_t* out);

/* Enqueue one product of `rows` rows (0 <= rows <= the plan's M; 0 does
 * nothing).  C may be NULL iff beta == 0 (C is not read then); D may be C
 * itself (same leading dimension); bias may be NULL; offsets is NULL iff the
 * plan has no groups.  ldc, ldd >= N (elements).  Errors: INVALID_ARG (null,
 * misaligned or aliased pointers, non-finite alpha / beta), SHAPE (rows,
 * leading dimensions), HIP. */
int dist_gemm_mx_run(dist_gemm_mx_plan_t plan, int64_t rows, const void* A, const void* A_scales, const void* B,
                     const void* B_scales, const void* C, int64_t ldc, void* D, int64_t ldd, const void* bias,
                     const int32_t* offsets, float alpha, float beta, void* stream);

/* Free the handle.  NULL is accepted (no-op). */
int dist_gemm_mx_destroy(dist_gemm_mx_plan_t plan);

/* Message of the last failure on `plan` (NULL: of a call of this header
 * without a plan, per thread).  Never NULL; valid until the next call. */
const char* dist_gemm_mx_last_error(dist_gemm_mx_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* DISTGEMM_MX_H_ */
