// Layer norm of rows, with the residual's addition before it, an 8-bit output
// and an 8-bit checkpoint behind it, and its gradient.
//
//   h = x + r (rounded to the type it is kept in),  mu = mean(h),
//   s = 1 / sqrt(mean((h - mu)^2) + eps),  n = (h - mu) s,  y = n w + b
//   with g = dy w:
//   dx = s (g - mean(g) - n mean(g n)) + dh,   dw = sum dy n,  db = sum dy
// All sums are fp32.  Both directions are bound by memory: every input is
// read once and every output written once, the row staying in registers
// between its sums and its use.  8192 x 8192 bf16 with residual into F8 with the
// checkpoint: 95 us, 5.7 TB/s (a copy: 6.2); 4 x 16384 into F8: 5.9 us, the latency
// of loads one behind another (x; per piece the residual, before h is stored; the
// weights behind those stores), two sums over 16 waves and a store; the gradient of
// 8192 x 8192 bf16 from the checkpoint with dh: 91 us, 5.2 TB/s (its second kernel 6.4
// of them), from the stream 100; of 1021 x 5123 fp32 19.7 us, two dependent launches
// (16.7 and 3.9), the first one's four rows to a workgroup a memory latency each.
//
// The variance is of the differences from a mean, never a difference of two
// sums: each wave sums its part of the row and the squares around its own
// mean, and the parts (count, mean, M2) are joined by
//   mean = sum n_i mean_i / n,   M2 = sum M2_i + n_i (mean_i - mean)^2,
// so one exchange between the waves does for both statistics.
//
// A row belongs to W waves (W = 1 .. 16), each lane holding V pieces of eight
// consecutive elements, piece c of lane t of the row at 8 (c * 64 W + t): wide
// loads, and an F8 block of 128 is 16 adjacent lanes.  Rows of up to 128 and 256
// columns have 16 and 32 lanes, four or two rows to a wave (262144 x 128 bf16: 25 us,
// with a wave to a row 90; its gradient 41 and 75).
#include "f8_common.h"

namespace dg {
namespace f8 {

constexpr int kMaxWaves = 16;

// Sum over the wave's lanes (or each 16 or 32 of them), in all of them: within 16 lanes by DPP, over the four rows by
// lane swaps.
template <int LANES = 64>
__device__ __forceinline__ float wave_total(float v) {
  auto add = [](float x, int y) { return x + __builtin_bit_cast(float, y); };
  v = add(v, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, true));
  v = add(v, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4E, 0xf, 0xf, true));
  v = add(v, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x141, 0xf, 0xf, true));
  v = add(v, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x140, 0xf, 0xf, true));
  if constexpr (LANES == 16) return v;
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t a0 = a[0], a1 = a[1];
  v = __builtin_bit_cast(float, a0) + __builtin_bit_cast(float, a1);
  if constexpr (LANES == 32) return v;
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  const uint32_t b0 = b[0], b1 = b[1];
  return __builtin_bit_cast(float, b0) + __builtin_bit_cast(float, b1);
}

// Eight e4m3 bytes of a row, n of them inside it.
template <int A>
__device__ __forceinline__ void store_bytes(uint8_t* y, u32x2 q, int n) {
  if constexpr (A != ANY) {
    store_wide<A>(reinterpret_cast<u32x2*>(y), q);
  } else if (n >= 8) {
    *reinterpret_cast<u32x2_any*>(y) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) y[j] = static_cast<uint8_t>(q[j / 4] >> (8 * (j & 3)));
  }
}

// grid: the rows over workgroups of several rows (W waves each, or LANES lanes of
// one), along x and, past kGridX, y
template <int T, int OUT, int V, int A, int LANES>
__global__ __launch_bounds__(1024) void layer_norm_kernel(LayerNormArgs a, int W) {
  constexpr int kShared = A == ANY ? ANY : ALIGNED;  // what every row reads
  __shared__ f32x2 parts[kMaxWaves];
  constexpr bool kWhole = LANES == 64;  // whole waves to a row
  // (a whole wave's row is one: kept in scalar registers, with its addresses)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = kWhole ? wave % W : 0;
  const int groups = kWhole ? (blockDim.x >> 6) / W : blockDim.x / LANES;
  const int t = kWhole ? part * 64 + (threadIdx.x & 63) : threadIdx.x % LANES, span = kWhole ? 64 * W : LANES;
  const int64_t row = (static_cast<int64_t>(blockIdx.y) * kGridX + blockIdx.x) * groups +
                      (kWhole ? wave / W : static_cast<int>(threadIdx.x) / LANES);
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
  // (behind the stores of h, which the compiler cannot tell apart from them, and waited for with x before the sums:
  // loads under branches are not counted)
  Raw8<T> wr[V], br[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int i = c * span + t;
    wr[c].zero();
    br[c].zero();
    if (i < d) {
      wr[c].template load<kShared>(a.weight, 8 * i, a.cols - 8 * i);
      if (a.bias) br[c].template load<kShared>(a.bias, 8 * i, a.cols - 8 * i);
    }
  }
  // elements of piece i inside the row
  auto inside = [&](int i) { return min(max(a.cols - 8 * i, 0), 8); };
  float sum = 0.0f;
  int count = kWhole ? 0 : a.cols;  // elements of this wave, or of the row
#pragma unroll
  for (int c = 0; c < V; ++c) {
    float f[8];
    x[c].get(f);
    float s8 = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s8 += f[j];  // (zeros past the end)
    sum += s8;
    if constexpr (kWhole) count += min(max(a.cols - 8 * (c * span + part * 64), 0), 512);
  }
  float mean = wave_total<LANES>(sum) / static_cast<float>(max(count, 1));
  float m2 = 0.0f;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int in = inside(c * span + t);
    float f[8];
    x[c].get(f);
    float s8 = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float e = j < in ? f[j] - mean : 0.0f;
      s8 = __builtin_fmaf(e, e, s8);
    }
    m2 += s8;
  }
  m2 = wave_total<LANES>(m2);
  if (kWhole && W > 1) {
    if ((threadIdx.x & 63) == 0) parts[wave] = f32x2{mean, m2};
    __syncthreads();
    // a part to a lane (a loop over the parts would wait for LDS once per part)
    const int i = threadIdx.x & 63;
    int n = 0;
#pragma unroll
    for (int c = 0; c < V; ++c) n += min(max(a.cols - 8 * (c * span + i * 64), 0), 512);
    n = i < W ? n : 0;
    const f32x2 p = n > 0 ? parts[wave - part + i] : f32x2{0.0f, 0.0f};
    const float count_i = static_cast<float>(n);
    mean = wave_total(count_i * p[0]) / static_cast<float>(a.cols);
    const float e = p[0] - mean;
    m2 = wave_total(n > 0 ? __builtin_fmaf(count_i * e, e, p[1]) : 0.0f);
  }
  if (!live) return;
  const float rstd = 1.0f / sqrtf(m2 / static_cast<float>(a.cols) + a.eps);
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  const int pitch8 = static_cast<int>(f8_pitch(a.cols) / 8);
  const int64_t pitch = f8_pitch(a.cols), spitch = f8_scale_pitch(a.cols);
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int i = c * span + t;
    // (whole blocks of 16 lanes go on: an F8 row is written to its pitch)
    if (i >= pitch8) continue;
    const int n = a.cols - 8 * i, in = inside(i);
    float f[8], w[8], b[8];
    x[c].get(f);
    wr[c].get(w);
    br[c].get(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < in ? (f[j] - mean) * rstd : 0.0f;
    if (a.kept) store_block8<A>(f, a.kept, row * pitch, i, a.kept_scales, row * spitch);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf(f[j], w[j], b[j]);
    if constexpr (OUT == LO_F8) {
      store_block8<A>(f, static_cast<uint8_t*>(a.y), row * pitch, i, a.scales, row * spitch);
    } else {
      if (i >= d) continue;
      if constexpr (OUT == LO_SAME) {
        x[c].set(f);
        x[c].template store<A>(a.y, row * a.ldy + 8 * i, n);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= a.inv_scale;
        store_bytes<A>(static_cast<uint8_t*>(a.y) + row * a.ldy + 8 * i, pack_e4m3<true>(f), n);
      }
    }
  }
  const int blocks = pitch8 / 16, pad = static_cast<int>(spitch) - blocks;
  if (t < pad) {
    if constexpr (OUT == LO_F8) a.scales[row * spitch + blocks + t] = 0;
    if (a.kept) a.kept_scales[row * spitch + blocks + t] = 0;
  }
}

// How the rows are reached.  fp32 stays in the caches: a lane's 32 bytes are two
// accesses to half of each line's bytes, and past the caches lines move twice
// (norm 8192 x 8192 115 us, so 104; with residual 220 and 200; gradient from
// the checkpoint with dh 178 and 163).
template <int T>
static int access_of(uint64_t misaligned, int64_t cols, int64_t bytes) {
  if ((misaligned & 15) != 0 || cols % 8 != 0) return ANY;
  return T == PT_F32 || bytes < kLastLevelCache ? ALIGNED : STREAM;
}

// Waves of a row: the fewest that keep a lane's pieces at two (8192 x 8192 bf16
// into F8 with the checkpoint: 97 us; four pieces 102, one 116), or, with too
// few rows to fill the chip, as many as have a piece each.
static int row_waves(int64_t rows, int d) {
  const int per_lane = rows >= 2048 ? 2 : 1;
  int W = 1;
  while (W < kMaxWaves && 64 * W * per_lane < d) W *= 2;
  return W;
}

template <int T, int OUT, int V, int LANES = 64>
static void norm_v(const LayerNormArgs& a, int W, int access, hipStream_t st) {
  const int groups = LANES < 64 ? 256 / LANES : W >= 4 ? 1 : 4 / W;
  const int64_t blocks = (a.rows + groups - 1) / groups;
  const dim3 grid(grid_x(blocks), grid_y(blocks)), block(LANES < 64 ? 256 : 64 * W * groups);
  constexpr int kStream = T == PT_F32 ? ALIGNED : STREAM;
  if (access == STREAM)
    hipLaunchKernelGGL((layer_norm_kernel<T, OUT, V, kStream, LANES>), grid, block, 0, st, a, W);
  else if (access == ALIGNED)
    hipLaunchKernelGGL((layer_norm_kernel<T, OUT, V, ALIGNED, LANES>), grid, block, 0, st, a, W);
  else
    hipLaunchKernelGGL((layer_norm_kernel<T, OUT, V, ANY, LANES>), grid, block, 0, st, a, W);
}

template <int T, int OUT>
static void norm_t(const LayerNormArgs& a, hipStream_t st) {
  const int es = T == PT_F32 ? 4 : 2, d = static_cast<int>(f8_pitch(a.cols) / 8);
  const int W = row_waves(a.rows, d), v = (d + 64 * W - 1) / (64 * W);
  uint64_t m = reinterpret_cast<uint64_t>(a.x) | static_cast<uint64_t>(a.ldx * es) | reinterpret_cast<uint64_t>(a.weight) |
               reinterpret_cast<uint64_t>(a.bias);
  if (a.residual)
    m |= reinterpret_cast<uint64_t>(a.residual) | static_cast<uint64_t>(a.ldr * es) | reinterpret_cast<uint64_t>(a.h) |
         static_cast<uint64_t>(a.ldh * es);
  if (OUT == LO_SAME) m |= reinterpret_cast<uint64_t>(a.y) | static_cast<uint64_t>(a.ldy * es);
  if (OUT == LO_E4M3) m |= (reinterpret_cast<uint64_t>(a.y) | static_cast<uint64_t>(a.ldy)) << 1;  // 8-byte stores
  const int64_t bytes = a.rows * a.cols * ((a.residual ? 3 : 1) * es + (OUT == LO_SAME ? es : 1) + (a.kept ? 1 : 0));
  const int access = access_of<T>(m, a.cols, bytes);
  // (few columns: four or two rows to a wave)
  if (d <= 16)
    norm_v<T, OUT, 1, 16>(a, 1, access, st);
  else if (d <= 32)
    norm_v<T, OUT, 1, 32>(a, 1, access, st);
  else if (v <= 1)
    norm_v<T, OUT, 1>(a, W, access, st);
  else if (v <= 2)
    norm_v<T, OUT, 2>(a, W, access, st);
  else
    norm_v<T, OUT, 4>(a, W, access, st);
}

template <int T>
static void norm_out(int out, const LayerNormArgs& a, hipStream_t st) {
  switch (out) {
    case LO_SAME: return norm_t<T, LO_SAME>(a, st);
    case LO_E4M3: return norm_t<T, LO_E4M3>(a, st);
    default: return norm_t<T, LO_F8>(a, st);
  }
}

// ---- gradient -------------------------------------------------------------
//
// dx needs two sums per row, dw and db one each per column over all rows.  A
// fixed number of workgroups walks the rows, each keeping its columns' share
// of dw and db in registers (the row's lanes hold the same columns every
// time), and writes it out once as a row of `partial`; a second kernel adds
// those rows.  No atomics: the order of every sum is fixed.
//
// The next row's loads are issued before the current row's sums, where the
// registers allow it (one piece to a lane, and two of bf16).  They hide the row's
// arithmetic and not much more: the compiler does not count loads under branches,
// so it waits for all that are under way, in fp32 before the sums cross the waves,
// at the latest before dx is stored.  A turn then costs a memory latency, which
// the CU's other workgroups have to cover.  Spills: none with one piece to a lane,
// nor with two from the stream on aligned rows; from the checkpoint two pieces
// spill one register of bf16 (11 of unaligned rows) and 11 to 15 of fp32, four
// pieces up to 50.
//
// Rows of more than 16384 columns have no registers for the columns' sums: there a
// kernel of its own walks down the columns first (4096 x 32768 bf16 from the
// checkpoint with dh 272 us, 2048 x 32768 fp32 332: half of the bytes are read twice).

// Eight elements of a row's dy and n (or h), as loaded.
template <int T, bool KEPT>
struct Pair {
  Raw8<T> dy, h;
  u32x2 code;
  uint32_t byte;
  template <int A>
  __device__ __forceinline__ void load(const LayerNormBackwardArgs& a, int64_t row, int i, bool in) {
    const int n = a.cols - 8 * i;
    dy.zero();
    if constexpr (KEPT) {
      code = u32x2{0, 0};
      byte = 0;
    } else {
      h.zero();
    }
    if (!in) return;
    dy.template load<A>(a.dy, row * a.lddy + 8 * i, n);
    if constexpr (KEPT) {
      code = load_wide<A>(reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.h) + row * f8_pitch(a.cols) + 8 * i));
      byte = a.h_scales[row * f8_scale_pitch(a.cols) + (i >> 4)];
    } else {
      h.template load<A>(a.h, row * a.ldh + 8 * i, n);
    }
  }
  // g = dy w (w of zeros past the columns) and n
  __device__ __forceinline__ void get(float mean, float s, float (&y)[8], float (&n)[8]) const {
    dy.get(y);
    if constexpr (KEPT) {
      unpack8(code, block_factor(byte), n);
      if (byte == 255u) {
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = __builtin_nanf("");
      }
    } else {
      h.get(n);
#pragma unroll
      for (int j = 0; j < 8; ++j) n[j] = (n[j] - mean) * s;
    }
  }
};

// (LANES: of a row, as in the forward kernel)
template <int T, bool KEPT, int V, int A, int LANES>
__global__ __launch_bounds__(1024) void layer_norm_backward_kernel(LayerNormBackwardArgs a, int W) {
  constexpr int kShared = A == ANY ? ANY : ALIGNED;
  constexpr bool kSums = V <= 2, kAhead = V == 1 || (V == 2 && T == PT_BF16);
  constexpr int N = kAhead ? V : 1;
  __shared__ f32x2 red[2][kMaxWaves];
  constexpr bool kWhole = LANES == 64;
  // (a whole wave's row is one: kept in scalar registers, with its addresses)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = kWhole ? wave % W : 0;
  const int groups = kWhole ? (blockDim.x >> 6) / W : blockDim.x / LANES;
  const int group = kWhole ? wave / W : static_cast<int>(threadIdx.x) / LANES;
  const int t = kWhole ? part * 64 + (threadIdx.x & 63) : threadIdx.x % LANES, span = kWhole ? 64 * W : LANES;
  const int d = (a.cols + 7) / 8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  float dw[kSums ? V : 1][8], db[kSums ? V : 1][8];
#pragma unroll
  for (int c = 0; c < (kSums ? V : 1); ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[c][j] = db[c][j] = 0.0f;
  Raw8<T> wr[kSums ? V : 1];
  auto weight = [&](int c, Raw8<T>& w) {
    const int i = c * span + t;
    w.zero();
    if (i < d) w.template load<kShared>(a.weight, 8 * i, a.cols - 8 * i);
  };
  if constexpr (kSums) {
#pragma unroll
    for (int c = 0; c < V; ++c) weight(c, wr[c]);
  }
  // all groups of the workgroup make the same number of turns (they share the barrier)
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t turns = (a.rows - static_cast<int64_t>(blockIdx.x) * groups + step - 1) / step;
  Pair<T, KEPT> in[V], ahead[N];
  Raw8<T> dh[kSums ? V : 1];
  auto fetch_dh = [&](int64_t r, int c, Raw8<T>& e) {
    const int i = c * span + t;
    e.zero();
    if (a.dh && r < a.rows && i < d) e.template load<A>(a.dh, r * a.lddh + 8 * i, a.cols - 8 * i);
  };
  float s = 0.0f, s1 = 0.0f, mu = 0.0f, mu1 = 0.0f;
  auto fetch = [&](int64_t r, int c, Pair<T, KEPT>& p) {
    const int i = c * span + t;
    p.template load<A>(a, r, i, r < a.rows && i < d);
  };
  auto statistics = [&](int64_t r, float& m, float& v) {
    v = r < a.rows ? a.rstd[r] : 0.0f;
    m = !KEPT && r < a.rows ? a.mean[r] : 0.0f;
  };
  if constexpr (kAhead) {
    statistics(row, mu1, s1);
#pragma unroll
    for (int c = 0; c < V; ++c) fetch(row, c, ahead[c]);
  }
  for (int64_t k = 0; k < turns; ++k) {
    // (dh is used behind the sums: asked for now, it needs no registers a row ahead)
    if constexpr (kSums) {
#pragma unroll
      for (int c = 0; c < V; ++c) fetch_dh(row, c, dh[c]);
    }
    if constexpr (kAhead) {
      s = s1;
      mu = mu1;
      statistics(row + step, mu1, s1);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        in[c] = ahead[c];
        fetch(row + step, c, ahead[c]);
      }
    } else {
      statistics(row, mu, s);
#pragma unroll
      for (int c = 0; c < V; ++c) fetch(row, c, in[c]);
    }
    float sg = 0.0f, sgn = 0.0f;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      float y[8], n[8], w[8];
      in[c].get(mu, s, y, n);
      if constexpr (kSums) {
        wr[c].get(w);
      } else {
        Raw8<T> r;
        weight(c, r);
        r.get(w);
      }
      float g8 = 0.0f, gn8 = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = y[j] * w[j];
        g8 += g;
        gn8 = __builtin_fmaf(g, n[j], gn8);
        if constexpr (kSums) {
          dw[c][j] = __builtin_fmaf(y[j], n[j], dw[c][j]);
          db[c][j] += y[j];
        }
      }
      sg += g8;
      sgn += gn8;
    }
    sg = wave_total<LANES>(sg);
    sgn = wave_total<LANES>(sgn);
    if (kWhole && W > 1) {
      // two sets of slots: a wave may be one turn ahead of another's reads
      if ((threadIdx.x & 63) == 0) red[k & 1][wave] = f32x2{sg, sgn};
      __syncthreads();
      // a wave's sums to a lane (a loop over them would wait for LDS once per wave)
      const int i = threadIdx.x & 63;
      const f32x2 p = i < W ? red[k & 1][wave - part + i] : f32x2{0.0f, 0.0f};
      sg = wave_total(p[0]);
      sgn = wave_total(p[1]);
    }
    sg *= inv_n;
    sgn *= inv_n;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int i = c * span + t;
      if (row >= a.rows || i >= d) continue;
      float y[8], n[8], w[8], e[8], o[8];
      in[c].get(mu, s, y, n);
      if constexpr (kSums) {
        wr[c].get(w);
      } else {
        Raw8<T> r;
        weight(c, r);
        r.get(w);
      }
      if constexpr (!kSums) fetch_dh(row, c, dh[0]);
      dh[kSums ? c : 0].get(e);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __builtin_fmaf(s, __builtin_fmaf(n[j], -sgn, __builtin_fmaf(y[j], w[j], -sg)), e[j]);
      Raw8<T> out;
      out.set(o);
      out.template store<A>(a.dx, row * a.lddx + 8 * i, a.cols - 8 * i);
    }
    row += step;
  }
  if constexpr (kSums) {
    // this workgroup's two rows of partial sums; several short rows' lanes are added through LDS
    float* const to = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    __shared__ float sums[2][4 * 512 * V];  // of four waves' columns
    if (groups > 1) {
      const int of_group = 8 * V * span, first = group * of_group;
#pragma unroll
      for (int c = 0; c < V; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sums[0][first + 8 * (c * span + t) + j] = dw[c][j];
          sums[1][first + 8 * (c * span + t) + j] = db[c][j];
        }
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * a.cols; i += blockDim.x) {
        const int which = i >= a.cols, col = i - which * a.cols;
        float v = 0.0f;
        for (int g = 0; g < groups; ++g) v += sums[which][g * of_group + col];
        to[i] = v;
      }
      return;
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int i = c * span + t;
      if (i >= d) continue;
      Raw8<PT_F32> out;
      out.set(dw[c]);
      out.template store<ANY>(to, 8 * i, a.cols - 8 * i);
      out.set(db[c]);
      out.template store<ANY>(to + a.cols, 8 * i, a.cols - 8 * i);
    }
  }
}

// The columns' sums by themselves: a workgroup has 512 columns (blockIdx.x) and
// every gridDim.y-th four rows, a wave to a row.
template <int T, bool KEPT, int A>
__global__ __launch_bounds__(256) void layer_norm_columns_kernel(LayerNormBackwardArgs a) {
  __shared__ float sums[2][4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = static_cast<int>(blockIdx.x) * 64 + lane;
  const bool in = 8 * i < a.cols;
  float dw[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.0f;
#pragma unroll 4
  for (int64_t row = static_cast<int64_t>(blockIdx.y) * 4 + wave; row < a.rows; row += static_cast<int64_t>(gridDim.y) * 4) {
    Pair<T, KEPT> p;
    p.template load<A>(a, row, i, in);
    float y[8], n[8];
    p.get(KEPT ? 0.0f : a.mean[row], a.rstd[row], y, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] = __builtin_fmaf(y[j], n[j], dw[j]);
      db[j] += y[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sums[0][wave][8 * lane + j] = dw[j];
    sums[1][wave][8 * lane + j] = db[j];
  }
  __syncthreads();
  float* const to = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
  for (int q = threadIdx.x; q < 1024; q += 256) {
    const int which = q >> 9, col = q & 511, at = static_cast<int>(blockIdx.x) * 512 + col;
    if (at < a.cols)
      to[static_cast<int64_t>(which) * a.cols + at] =
          (sums[which][0][col] + sums[which][1][col]) + (sums[which][2][col] + sums[which][3][col]);
  }
}

// Adds the rows of `partial` (dw's and db's columns side by side): 64 columns per workgroup, 16 waves over the rows.
__global__ __launch_bounds__(1024) void layer_norm_dweight_kernel(const float* partial, float* dweight, float* dbias,
                                                                 int blocks, int cols) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = static_cast<int>(blockIdx.x) * 64 + lane, all = 2 * cols;
  float v = 0.0f;
  if (col < all)
#pragma unroll 8
    for (int b = wave; b < blocks; b += 16) v += partial[static_cast<int64_t>(b) * all + col];
  sums[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && col < all) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sums[w][lane];
    if (col < cols)
      dweight[col] = s;
    else if (dbias)
      dbias[col - cols] = s;
  }
}

// Workgroups of one row of W waves, or of 4 / W rows where W is less than four
// (65536 x 1000 bf16 with dh: 128 us with one row of one wave to each, 95 with
// four); as many workgroups as the chip holds at a time.
static int row_lanes(int64_t cols) { return cols <= 128 ? 16 : cols <= 256 ? 32 : 64; }
static void backward_shape(int type, int64_t rows, int64_t cols, int* W, int* groups, int64_t* blocks) {
  const int d = static_cast<int>((cols + 7) / 8), pieces = type == PT_BF16 && d > 64 ? 2 : 1;
  *W = 1;
  while (*W < kMaxWaves && 64 * *W * pieces < d) *W *= 2;
  *groups = cols <= 256 ? 256 / row_lanes(cols) : *W < 4 ? 4 / *W : 1;
  const int waves = cols <= 256 ? 4 : *W * *groups, fit = waves >= 16 ? 1 : (waves >= 8 ? 2 : 4);
  const int64_t want = (rows + *groups - 1) / *groups, cap = 256 * fit;
  *blocks = want < cap ? want : cap;
}

// Rows of `partial`: one per workgroup, or of the columns' own kernel one per split of the rows.
constexpr int kSumCols = 16384, kSplits = 32;
static int64_t partial_rows(int64_t rows, int64_t cols, int64_t blocks) {
  if (cols <= kSumCols) return blocks;
  const int64_t fours = (rows + 3) / 4;
  return fours < kSplits ? fours : kSplits;
}

template <int T, bool KEPT, int V, int A>
static void backward_launch(const LayerNormBackwardArgs& a, int W, int groups, int64_t blocks, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(blocks));
  if constexpr (V == 1) {
    // (few columns: four or two rows to a wave)
    const int lanes = row_lanes(a.cols);
    if (lanes == 16)
      hipLaunchKernelGGL((layer_norm_backward_kernel<T, KEPT, V, A, 16>), grid, dim3(256), 0, st, a, W);
    if (lanes == 32)
      hipLaunchKernelGGL((layer_norm_backward_kernel<T, KEPT, V, A, 32>), grid, dim3(256), 0, st, a, W);
    if (lanes < 64) return;
  }
  hipLaunchKernelGGL((layer_norm_backward_kernel<T, KEPT, V, A, 64>), grid, dim3(64 * W * groups), 0, st, a, W);
}

template <int T, bool KEPT, int V>
static void backward_v(const LayerNormBackwardArgs& a, int W, int groups, int64_t blocks, int access, hipStream_t st) {
  if constexpr (V > 2) {
    // the columns' kernel reads dy and the rows first: dx may be one of them
    const int64_t splits = partial_rows(a.rows, a.cols, blocks);
    const dim3 grid(static_cast<unsigned>((a.cols + 511) / 512), static_cast<unsigned>(splits));
    if (access == ANY)
      hipLaunchKernelGGL((layer_norm_columns_kernel<T, KEPT, ANY>), grid, dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((layer_norm_columns_kernel<T, KEPT, ALIGNED>), grid, dim3(256), 0, st, a);
  }
  constexpr int kStream = T == PT_F32 ? ALIGNED : STREAM;
  if (access == STREAM)
    backward_launch<T, KEPT, V, kStream>(a, W, groups, blocks, st);
  else if (access == ALIGNED)
    backward_launch<T, KEPT, V, ALIGNED>(a, W, groups, blocks, st);
  else
    backward_launch<T, KEPT, V, ANY>(a, W, groups, blocks, st);
}

template <int T, bool KEPT>
static hipError_t backward_t(const LayerNormBackwardArgs& a, hipStream_t st) {
  const uint64_t es = T == PT_F32 ? 4 : 2;
  uint64_t m = reinterpret_cast<uint64_t>(a.dy) | reinterpret_cast<uint64_t>(a.dx) | reinterpret_cast<uint64_t>(a.weight) |
               static_cast<uint64_t>(a.lddy) * es | static_cast<uint64_t>(a.lddx) * es;
  if (!KEPT) m |= reinterpret_cast<uint64_t>(a.h) | static_cast<uint64_t>(a.ldh) * es;
  if (a.dh) m |= reinterpret_cast<uint64_t>(a.dh) | static_cast<uint64_t>(a.lddh) * es;
  const int64_t bytes = a.rows * a.cols * (static_cast<int64_t>(es) * (a.dh ? 3 : 2) + (KEPT ? 1 : es));
  int W, groups;
  int64_t blocks;
  backward_shape(T, a.rows, a.cols, &W, &groups, &blocks);
  const int d = (a.cols + 7) / 8, v = (d + 64 * W - 1) / (64 * W);
  const int access = access_of<T>(m, a.cols, bytes);
  if (blocks == 0)
    ;  // no rows: the second kernel writes zeros
  else if (v <= 1)
    backward_v<T, KEPT, 1>(a, W, groups, blocks, access, st);
  else if (v <= 2)
    backward_v<T, KEPT, 2>(a, W, groups, blocks, access, st);
  else
    backward_v<T, KEPT, 4>(a, W, groups, blocks, access, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(layer_norm_dweight_kernel, dim3(static_cast<unsigned>((2 * a.cols + 63) / 64)), dim3(1024), 0, st,
                     a.partial, a.dweight, a.dbias, static_cast<int>(partial_rows(a.rows, a.cols, blocks)), a.cols);
  return hipGetLastError();
}

}  // namespace f8

hipError_t launch_layer_norm(int type, int out, const LayerNormArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (type == PT_F32)
    f8::norm_out<PT_F32>(out, a, st);
  else
    f8::norm_out<PT_BF16>(out, a, st);
  return hipGetLastError();
}

int64_t layer_norm_backward_blocks(int64_t rows, int64_t cols) {
  int W, groups;
  int64_t f32, bf16;
  f8::backward_shape(PT_F32, rows, cols, &W, &groups, &f32);
  f8::backward_shape(PT_BF16, rows, cols, &W, &groups, &bf16);
  return f8::partial_rows(rows, cols, f32 > bf16 ? f32 : bf16);
}

hipError_t launch_layer_norm_backward(int type, const LayerNormBackwardArgs& a, hipStream_t st) {
  if (type == PT_F32) return a.h_scales ? f8::backward_t<PT_F32, true>(a, st) : f8::backward_t<PT_F32, false>(a, st);
  return a.h_scales ? f8::backward_t<PT_BF16, true>(a, st) : f8::backward_t<PT_BF16, false>(a, st);
}

}  // namespace dg
