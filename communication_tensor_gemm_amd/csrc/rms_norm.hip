// Root-mean-square norm of rows, with the residual's addition before it and
// an 8-bit or MX output after it, and its gradient.
//
//   h = x + r (rounded to the type it is kept in),  s = 1 / sqrt(mean(h^2) + eps),
//   y = h * s * w
//   with g = dy * w and n = h * s:
//   dx = s * (g - n * mean(g * n)) + dh,   dw = sum over rows of dy * n
// All sums are fp32.  Both directions are bound by memory: every input is
// read once and every output written once, the row staying in registers
// between its sum and its use.  8192 x 16384 bf16 with residual into e4m3: 153
// us, 6.1 TB/s (a copy of the size: 6.2); 4 x 16384 into MX E4M3: 5 us, the
// latency of a load, two sums over 16 waves and a store; the gradient of 8192 x
// 8192 bf16 with dh: 95 us, 5.6 TB/s (its second kernel 4.4 of them), of 1021 x
// 5123 fp32 18 us, two launches.  Rows of few columns are bound by their waves: a
// row has one of its own, 262144 x 128 bf16 takes 71 us, 1.9 TB/s, with 16 of 64
// lanes at work (256 columns 74 us), its gradient 74.
//
// (The sum of squares is fp32: a row past 1.8e19 / sqrt(cols) overflows it.)
//
// A row belongs to W waves (W = 1 .. 16), each lane holding V pieces of eight
// consecutive elements, piece c of lane t of the row at 8 (c * 64 W + t): wide
// loads, and an MX block of 32 is four adjacent lanes.
#include "mx_common.h"
#include "mx_shape.h"

namespace dg {
namespace mx {

constexpr int kMaxWaves = 16;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sum over the W waves of a row; red: one slot per wave of the workgroup.
// Every wave of the workgroup calls it.
__device__ __forceinline__ float row_sum(float v, float* red, int W) {
  v = wave_sum(v);
  if (W == 1) return v;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) red[wave] = v;
  __syncthreads();
  float s = 0.0f;
  const int first = wave / W * W;
  for (int i = 0; i < W; ++i) s += red[first + i];
  return s;
}

// grid: the rows over workgroups of several rows (W waves each), along x and, past kGridX, y
template <int T, int OUT, int V, int A>
__global__ __launch_bounds__(1024) void rms_norm_kernel(NormArgs a, int W) {
  constexpr int kShared = A == ANY ? ANY : ALIGNED;  // what every row reads
  __shared__ float red[kMaxWaves];
  const int wave = threadIdx.x >> 6, groups = (blockDim.x >> 6) / W;
  const int t = static_cast<int>(threadIdx.x) - wave / W * W * 64, span = 64 * W;
  const int64_t row = (static_cast<int64_t>(blockIdx.y) * kGridX + blockIdx.x) * groups + wave / W;
  const bool live = row < a.rows;
  const int d = (a.cols + 7) / 8;
  Raw8<T> x[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int i = c * span + t;
    x[c].zero();
    if (live && i < d) x[c].template load<A>(a.x, row * a.ldx + 8 * i, a.cols - 8 * i);
  }
  if (a.residual) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int i = c * span + t;
      if (live && i < d) {
        Raw8<T> r;
        r.template load<A>(a.residual, row * a.ldr + 8 * i, a.cols - 8 * i);
        float f[8], g[8];
        x[c].get(f);
        r.get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += g[j];
        x[c].set(f);
        x[c].template store<A>(a.h, row * a.ldh + 8 * i, a.cols - 8 * i);
      }
    }
  }
  // the weight is on its way while the row is summed
  Raw8<T> wr[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int i = c * span + t;
    wr[c].zero();
    if (i < d) wr[c].template load<kShared>(a.weight, 8 * i, a.cols - 8 * i);
  }
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    float f[8];
    x[c].get(f);
    float s8 = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s8 = __builtin_fmaf(f[j], f[j], s8);
    ss += s8;
  }
  ss = row_sum(ss, red, W);
  if (!live) return;
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int i = c * span + t;
    if (i >= d) continue;
    const int n = a.cols - 8 * i;
    float f[8], w[8];
    x[c].get(f);
    wr[c].get(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];
    if constexpr (OUT == NO_SAME) {
      x[c].set(f);
      x[c].template store<A>(a.y, row * a.ldy + 8 * i, n);
    } else if constexpr (OUT == NO_E4M3) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= a.inv_scale;
      const u32x2 q = pack_e4m3<true>(f);
      uint8_t* y = static_cast<uint8_t*>(a.y) + row * a.ldy + 8 * i;
      if constexpr (A != ANY) {
        store_wide<A>(reinterpret_cast<u32x2*>(y), q);
      } else if (n >= 8) {
        *reinterpret_cast<u32x2_any*>(y) = q;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) y[j] = static_cast<uint8_t>(q[j / 4] >> (8 * (j & 3)));
      }
    } else {
      constexpr int FMT = OUT == NO_MX_E2M1 ? MX_E2M1 : MX_E4M3;
      store_block<FMT, A>(f, static_cast<uint8_t*>(a.y), row * mx_row_bytes(a.cols, FMT), i, a.scales,
                       row * scale_pitch(a.cols));
    }
  }
  if constexpr (OUT == NO_MX_E2M1 || OUT == NO_MX_E4M3) {
    const int blocks = a.cols / kMxBlock, pad = static_cast<int>(scale_pitch(a.cols)) - blocks;
    if (t < pad) a.scales[row * scale_pitch(a.cols) + blocks + t] = 0;
  }
}

// Waves of a row: the fewest that keep a lane's pieces at four, or, with too
// few rows to fill the chip, as many as have a piece each.
static int row_waves(int64_t rows, int d) {
  const int per_lane = rows >= 2048 ? 4 : 1;
  int W = 1;
  while (W < kMaxWaves && 64 * W * per_lane < d) W *= 2;
  return W;
}

template <int T, int OUT, int V>
static hipError_t norm_v(const NormArgs& a, int W, int access, hipStream_t st) {
  const int groups = W >= 4 ? 1 : 4 / W;
  const int64_t blocks = (a.rows + groups - 1) / groups;
  const dim3 grid(grid_x(blocks), grid_y(blocks)), block(64 * W * groups);
  if (access == STREAM)
    hipLaunchKernelGGL((rms_norm_kernel<T, OUT, V, STREAM>), grid, block, 0, st, a, W);
  else if (access == ALIGNED)
    hipLaunchKernelGGL((rms_norm_kernel<T, OUT, V, ALIGNED>), grid, block, 0, st, a, W);
  else
    hipLaunchKernelGGL((rms_norm_kernel<T, OUT, V, ANY>), grid, block, 0, st, a, W);
  return hipGetLastError();
}

template <int T, int OUT>
static hipError_t norm_t(const NormArgs& a, hipStream_t st) {
  const int es = T == PT_F32 ? 4 : 2, d = (a.cols + 7) / 8;
  const int W = row_waves(a.rows, d), v = (d + 64 * W - 1) / (64 * W);
  uint64_t m = reinterpret_cast<uint64_t>(a.x) | static_cast<uint64_t>(a.ldx * es) | reinterpret_cast<uint64_t>(a.weight);
  if (a.residual)
    m |= reinterpret_cast<uint64_t>(a.residual) | static_cast<uint64_t>(a.ldr * es) | reinterpret_cast<uint64_t>(a.h) |
         static_cast<uint64_t>(a.ldh * es);
  if (OUT == NO_SAME) m |= reinterpret_cast<uint64_t>(a.y) | static_cast<uint64_t>(a.ldy * es);
  if (OUT == NO_E4M3) m |= (reinterpret_cast<uint64_t>(a.y) | static_cast<uint64_t>(a.ldy)) << 1;  // 8-byte stores
  const int64_t bytes = a.rows * a.cols * ((a.residual ? 3 : 1) * es + (OUT == NO_SAME ? es : 1));
  const int access = (m & 15) != 0 || a.cols % 8 != 0 ? ANY : bytes < kLastLevelCache ? ALIGNED : STREAM;
  if (v <= 1) return norm_v<T, OUT, 1>(a, W, access, st);
  if (v <= 2) return norm_v<T, OUT, 2>(a, W, access, st);
  return norm_v<T, OUT, 4>(a, W, access, st);
}

template <int T>
static hipError_t norm_out(int out, const NormArgs& a, hipStream_t st) {
  switch (out) {
    case NO_SAME: return norm_t<T, NO_SAME>(a, st);
    case NO_E4M3: return norm_t<T, NO_E4M3>(a, st);
    case NO_MX_E2M1: return norm_t<T, NO_MX_E2M1>(a, st);
    default: return norm_t<T, NO_MX_E4M3>(a, st);
  }
}

// ---- gradient -------------------------------------------------------------
//
// dx needs one sum per row, dw one per column over all rows.  A fixed number
// of workgroups walks the rows, each keeping its columns' share of dw in
// registers (the row's lanes hold the same columns every time), and writes
// it out once as a row of `partial`; a second kernel adds those rows.  No
// atomics: the order of every sum is fixed, so the result is the same bit
// for bit from run to run.  With one piece per lane (of bf16, one or two; rows
// of up to 8192 and 16384 columns) the next row's loads are in flight while
// the current row's sum crosses the waves; longer rows have no registers for
// that, and above 16384 columns the row itself is read again (from the L2)
// after its sum.  There a lane's 32 column sums and the pieces do not fit 128
// registers either, and 164 to 276 bytes per lane go to scratch: 4096 x 32768 bf16
// with dh takes 452 us, 2.4 TB/s, 8192 x 16384 192 us, 5.6 TB/s (two pieces of
// bf16 keep 20 bytes of scratch, none of them in the loop over the rows).
template <int T, int V, int A>
__global__ __launch_bounds__(1024) void rms_norm_backward_kernel(NormBackwardArgs a, int W) {
  constexpr int kShared = A == ANY ? ANY : ALIGNED;
  __shared__ float red[2][kMaxWaves];
  const int wave = threadIdx.x >> 6, groups = (blockDim.x >> 6) / W;
  const int t = static_cast<int>(threadIdx.x) - wave / W * W * 64, span = 64 * W;
  const int d = (a.cols + 7) / 8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  constexpr bool kAhead = V == 1 || (V == 2 && T == PT_BF16), kHold = V <= 2;
  constexpr int H = kHold ? V : 1, N = kAhead ? V : 1;
  float dw[V][8];
#pragma unroll
  for (int c = 0; c < V; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[c][j] = 0.0f;
  Raw8<T> wr;  // the weight: kept if it is one piece
  auto weight = [&](int i) {
    wr.zero();
    if (i < d) wr.template load<kShared>(a.weight, 8 * i, a.cols - 8 * i);
  };
  if constexpr (V == 1) weight(t);
  // all groups of the workgroup make the same number of turns (they share the barrier)
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + wave / W;
  const int64_t turns = (a.rows - static_cast<int64_t>(blockIdx.x) * groups + step - 1) / step;
  Raw8<T> dy[H], h[H], dh[H], dy1[N], h1[N], dh1[N];
  float s = 0.0f, s1 = 0.0f;
  auto fetch = [&](int64_t r, int c, Raw8<T>& py, Raw8<T>& ph, Raw8<T>& pd) {
    const int i = c * span + t;
    py.zero();
    ph.zero();
    pd.zero();
    if (r < a.rows && i < d) {
      const int n = a.cols - 8 * i;
      py.template load<A>(a.dy, r * a.lddy + 8 * i, n);
      ph.template load<A>(a.h, r * a.ldh + 8 * i, n);
      if (a.dh) pd.template load<A>(a.dh, r * a.lddh + 8 * i, n);
    }
  };
  auto scale = [&](int64_t r) { return r < a.rows ? a.rstd[r] : 0.0f; };
  if constexpr (kAhead) {
    s1 = scale(row);
#pragma unroll
    for (int c = 0; c < V; ++c) fetch(row, c, dy1[c], h1[c], dh1[c]);
  }
  for (int64_t k = 0; k < turns; ++k) {
    if constexpr (kAhead) {
      s = s1;
      s1 = scale(row + step);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        dy[c] = dy1[c];
        h[c] = h1[c];
        dh[c] = dh1[c];
        fetch(row + step, c, dy1[c], h1[c], dh1[c]);
      }
    } else {
      s = scale(row);
      if constexpr (kHold) {
#pragma unroll
        for (int c = 0; c < V; ++c) fetch(row, c, dy[c], h[c], dh[c]);
      }
    }
    // g = y w and n = x s (y = dy, x = h): the row's sum is sum(g n), a column's
    // share of dw is y n, and dx = s (g - n mean(g n)) + dh.  No power of s is
    // formed: s^3 leaves fp32 from |h| about 1e13 up and 1e-13 down.
    float dot = 0.0f, yw[kHold ? V : 1][8], n[kHold ? V : 1][8];
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int q = kHold ? c : 0;
      if constexpr (!kHold) __builtin_amdgcn_sched_barrier(0);  // one piece in registers at a time
      if constexpr (!kHold) fetch(row, c, dy[0], h[0], dh[0]);
      if constexpr (V > 1) weight(c * span + t);
      float y[8], w[8];
      dy[q].get(y);
      h[q].get(n[q]);
      wr.get(w);
      float d8 = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        yw[q][j] = y[j] * w[j];
        n[q][j] *= s;
        d8 = __builtin_fmaf(yw[q][j], n[q][j], d8);
        dw[c][j] = __builtin_fmaf(y[j], n[q][j], dw[c][j]);
      }
      dot += d8;
    }
    // two sets of slots: a wave may be one turn ahead of another's reads
    const float mean = row_sum(dot, red[k & 1], W) * inv_n;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int i = c * span + t, q = kHold ? c : 0;
      if constexpr (!kHold) {
        __builtin_amdgcn_sched_barrier(0);
        fetch(row, c, dy[0], h[0], dh[0]);
        weight(i);
        float y[8], w[8];
        dy[0].get(y);
        h[0].get(n[0]);
        wr.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          yw[0][j] = y[j] * w[j];
          n[0][j] *= s;
        }
      }
      if (row >= a.rows || i >= d) continue;
      float e[8], o[8];
      dh[q].get(e);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __builtin_fmaf(s, __builtin_fmaf(n[q][j], -mean, yw[q][j]), e[j]);
      Raw8<T> out;
      out.set(o);
      out.template store<A>(a.dx, row * a.lddx + 8 * i, a.cols - 8 * i);
    }
    row += step;
  }
  // this workgroup's row of partial sums; several short rows' lanes are added through LDS
  __shared__ float sums[4][512];
  if (groups > 1) {
    // only rows of at most 512 columns come several to a workgroup
#pragma unroll
    for (int c = 0; c < V; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = 8 * (c * span + t) + j;
        if (col < 512) sums[wave / W][col] = dw[c][j];
      }
    __syncthreads();
    for (int col = threadIdx.x; col < a.cols; col += blockDim.x) {
      float v = 0.0f;
      for (int g = 0; g < groups; ++g) v += sums[g][col];
      a.partial[static_cast<int64_t>(blockIdx.x) * a.cols + col] = v;
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int i = c * span + t;
    if (i >= d) continue;
    Raw8<PT_F32> out;
    out.set(dw[c]);
    out.template store<ANY>(a.partial, static_cast<int64_t>(blockIdx.x) * a.cols + 8 * i, a.cols - 8 * i);
  }
}

// Adds the rows of `partial`: 64 columns per workgroup, 16 waves over the rows.
__global__ __launch_bounds__(1024) void rms_norm_dweight_kernel(const float* partial, float* dweight, int blocks,
                                                               int cols) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = static_cast<int>(blockIdx.x) * 64 + lane;
  float v = 0.0f;
  if (col < cols)
#pragma unroll 8
    for (int b = wave; b < blocks; b += 16) v += partial[static_cast<int64_t>(b) * cols + col];
  sums[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && col < cols) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sums[w][lane];
    dweight[col] = s;
  }
}

// One row per workgroup of W waves, or four rows of one wave each where a row
// has at most 512 columns.  bf16 rows take two pieces to a lane, so that two
// workgroups of half the threads share a CU and one moves data while the
// other's sum crosses its waves; fp32 has the registers for one.  As many
// workgroups as the chip holds at a time.
static void backward_shape(int type, int64_t rows, int64_t cols, int* W, int* groups, int64_t* blocks) {
  const int d = static_cast<int>((cols + 7) / 8), pieces = type == PT_BF16 && d > 64 ? 2 : 1;
  *W = 1;
  while (*W < kMaxWaves && 64 * *W * pieces < d) *W *= 2;
  *groups = cols <= 512 ? 4 : 1;
  const int waves = *W * *groups, fit = waves >= 16 ? 1 : (waves >= 8 ? 2 : 4);
  const int64_t want = (rows + *groups - 1) / *groups, cap = 256 * fit;
  *blocks = want < cap ? want : cap;
}

template <int T, int V>
static void backward_v(const NormBackwardArgs& a, int W, int groups, int64_t blocks, int access, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * W * groups);
  constexpr int kStream = V <= 2 ? STREAM : ALIGNED;  // (a row that is read twice does not go past the caches)
  if (access == STREAM)
    hipLaunchKernelGGL((rms_norm_backward_kernel<T, V, kStream>), grid, block, 0, st, a, W);
  else if (access == ALIGNED)
    hipLaunchKernelGGL((rms_norm_backward_kernel<T, V, ALIGNED>), grid, block, 0, st, a, W);
  else
    hipLaunchKernelGGL((rms_norm_backward_kernel<T, V, ANY>), grid, block, 0, st, a, W);
}

template <int T>
static hipError_t backward_t(const NormBackwardArgs& a, hipStream_t st) {
  const uint64_t es = T == PT_F32 ? 4 : 2;
  uint64_t m = reinterpret_cast<uint64_t>(a.dy) | reinterpret_cast<uint64_t>(a.h) | reinterpret_cast<uint64_t>(a.dx) |
               reinterpret_cast<uint64_t>(a.weight) | static_cast<uint64_t>(a.lddy) * es |
               static_cast<uint64_t>(a.ldh) * es | static_cast<uint64_t>(a.lddx) * es;
  if (a.dh) m |= reinterpret_cast<uint64_t>(a.dh) | static_cast<uint64_t>(a.lddh) * es;
  const int64_t bytes = a.rows * a.cols * static_cast<int64_t>(es) * (a.dh ? 4 : 3);
  int W, groups;
  int64_t blocks;
  backward_shape(T, a.rows, a.cols, &W, &groups, &blocks);
  const int d = (a.cols + 7) / 8, v = (d + 64 * W - 1) / (64 * W);
  const int access = (m & 15) != 0 || a.cols % 8 != 0 ? ANY : bytes < kLastLevelCache ? ALIGNED : STREAM;
  if (blocks == 0)
    ;  // no rows: the second kernel writes zeros
  else if (v <= 1)
    backward_v<T, 1>(a, W, groups, blocks, access, st);
  else if (v <= 2)
    backward_v<T, 2>(a, W, groups, blocks, access, st);
  else
    backward_v<T, 4>(a, W, groups, blocks, access, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(rms_norm_dweight_kernel, dim3(static_cast<unsigned>((a.cols + 63) / 64)), dim3(1024), 0, st,
                     a.partial, a.dweight, static_cast<int>(blocks), a.cols);
  return hipGetLastError();
}

}  // namespace mx

hipError_t launch_rms_norm(int type, int out, const NormArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  return type == PT_F32 ? mx::norm_out<PT_F32>(out, a, st) : mx::norm_out<PT_BF16>(out, a, st);
}

int64_t rms_norm_backward_blocks(int64_t rows, int64_t cols) {
  int W, groups;
  int64_t f32, bf16;
  mx::backward_shape(PT_F32, rows, cols, &W, &groups, &f32);
  mx::backward_shape(PT_BF16, rows, cols, &W, &groups, &bf16);
  return f32 > bf16 ? f32 : bf16;
}

hipError_t launch_rms_norm_backward(int type, const NormBackwardArgs& a, hipStream_t st) {
  return type == PT_F32 ? mx::backward_t<PT_F32>(a, st) : mx::backward_t<PT_BF16>(a, st);
}

}  // namespace dg
