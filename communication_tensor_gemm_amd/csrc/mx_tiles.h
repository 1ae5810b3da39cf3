// Device helpers of the MX product kernels: buffer loads, the groups' tile
// search and the element epilogue.
#pragma once
#include "mx_common.h"
#include "mx_shape.h"

namespace dg {
namespace mx {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;

// A pointer into global memory, said so in its type: where it was read from
// memory, the compiler cannot know, and flat accesses (which also occupy the
// LDS counter) would be the result.
template <typename T>
using global_ptr = __attribute__((address_space(1))) T*;

constexpr uint32_t kOutOfRange = 0x80000000u;  // an offset past every descriptor's end: the load gives zeros

// Buffer descriptor of a wave-uniform base and byte count (below 2^31).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), (short)0,
                                           static_cast<int>(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000);
}

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff = 0) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
}

// The rows of one group tile.
struct GroupTile {
  int32_t group;  // -1: there is no such tile
  int32_t row0;   // first row of the tile
  int32_t rows;   // rows left in the group from there
  int32_t index;  // the tile's place in the group, of `tiles`
  int32_t tiles;
};

// Row tile u (of height tm) of the groups' rows, groups in order, each with
// ceil(rows / tm) tiles.  Offsets are clamped to [0, M] and to be ascending (one
// below an earlier one counts as that one), so that wrong ones cannot reach past
// the operands, no row is in two groups, and the tiles are no more than the
// launch was made for.  The wave's 64 lanes take 64 groups at a time: a scan of
// their tile counts, then a ballot.
// Every lane of the wave calls it with the same arguments.  total: all tiles.
__device__ __forceinline__ int32_t group_bound(const int32_t* offsets, int32_t i, int32_t M) {
  return min(max(((global_ptr<const int32_t>)offsets)[i], 0), M);
}

// 64 groups, one per lane: their rows lo .. hi - 1 and the tiles of the
// groups up to and including the lane's.  from: the end of the groups before.
struct GroupLanes {
  int32_t lo, hi, incl;
};
__device__ __forceinline__ GroupLanes load_groups(const int32_t* offsets, int32_t groups, int32_t M, int32_t tm,
                                                  int32_t base = 0, int32_t from = 0) {
  const int lane = threadIdx.x & 63;
  GroupLanes g;
  // (past the last group: no rows, from its end on)
  g.lo = max(group_bound(offsets, min(base + lane, groups), M), from);
  g.hi = group_bound(offsets, min(base + lane + 1, groups), M);
  // an offset falls: the running maximum instead (rolled and out of the way: 64 rows
  // over 32 groups 22 us, as without it; in line 23)
  if (__builtin_expect(__ballot(g.hi < g.lo) != 0, 0)) {
#pragma unroll 1
    for (int s = 1; s < 64; s <<= 1) {
      const int32_t v = __shfl_up(g.lo, s);
      if (lane >= s) g.lo = max(g.lo, v);
    }
    g.hi = max(g.lo, g.hi);
  }
  g.incl = tile_count(g.hi - g.lo, tm);
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int32_t v = __shfl_up(g.incl, s);
    if (lane >= s) g.incl += v;
  }
  return g;
}

// Row tile u among these 64 groups, `before` tiles and `base` groups before them.
__device__ __forceinline__ GroupTile group_tile_of(const GroupLanes& g, int32_t base, int32_t before, int32_t tm,
                                                   int32_t u) {
  const uint64_t past = __ballot(before + g.incl > u);
  if (past == 0) return GroupTile{-1, 0, 0, 0, 0};
  const int first = __builtin_ctzll(past);
  const int32_t lo = __builtin_amdgcn_readlane(g.lo, first), hi = __builtin_amdgcn_readlane(g.hi, first);
  GroupTile t;
  t.group = base + first;
  t.tiles = tile_count(hi - lo, tm);
  t.index = u - (before + __builtin_amdgcn_readlane(g.incl, first) - t.tiles);
  t.row0 = lo + t.index * tm;
  t.rows = hi - t.row0;
  return t;
}

__device__ __forceinline__ GroupTile find_group_tile(const int32_t* offsets, int32_t groups, int32_t M, int32_t tm,
                                                     int32_t u) {
  int32_t before = 0, from = 0;  // tiles and end of the groups already passed
  for (int32_t base = 0; base < groups; base += 64) {
    const GroupLanes g = load_groups(offsets, groups, M, tm, base, from);
    const GroupTile t = group_tile_of(g, base, before, tm, u);
    if (t.group >= 0) return t;
    before += __builtin_amdgcn_readlane(g.incl, 63);
    from = __builtin_amdgcn_readlane(g.hi, 63);
  }
  return GroupTile{-1, 0, 0, 0, 0};
}

// All row tiles of height tm.
__device__ __forceinline__ int32_t count_group_tiles(const int32_t* offsets, int32_t groups, int32_t M, int32_t tm) {
  const int lane = threadIdx.x & 63;
  int32_t n = 0;
  bool falls = false;
  for (int32_t g = lane; g < groups; g += 64) {
    const int32_t lo = group_bound(offsets, g, M), hi = group_bound(offsets, g + 1, M);
    falls |= hi < lo;
    n += tile_count(max(hi, lo) - lo, tm);
  }
  if (__ballot(falls) != 0) {
    int32_t all = 0, from = 0;
    for (int32_t base = 0; base < groups; base += 64) {
      const GroupLanes g = load_groups(offsets, groups, M, tm, base, from);
      all += __builtin_amdgcn_readlane(g.incl, 63);
      from = __builtin_amdgcn_readlane(g.hi, 63);
    }
    return all;
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) n += __shfl_xor(n, s);
  return __builtin_amdgcn_readfirstlane(n);
}

// Row tiles that `groups` groups with M rows together can have at most.
inline int64_t most_group_tiles(int64_t M, int64_t groups, int64_t tm) {
  const int64_t some = groups < M ? groups : M;  // groups that can have a row
  return some + (M - some) / tm;
}

template <bool kBf16>
__device__ __forceinline__ float load_value(const void* p, int64_t i) {
  if constexpr (kBf16)
    return __builtin_bit_cast(float, static_cast<uint32_t>(((global_ptr<const uint16_t>)p)[i]) << 16);
  else
    return ((global_ptr<const float>)p)[i];
}

// Four neighbouring values of row `row` from column `col`: alpha * v + beta *
// C + bias, rounded once.  n values are inside D; wide: the row's 4-element
// pieces are aligned for one store.
template <bool kBf16>
__device__ __forceinline__ void store_four(const MxGemmArgs& a, int64_t bias0, int64_t row, int32_t col, int32_t n,
                                           bool wide, f32x4 v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float o = a.alpha * v[e];
    if (e < n) {
      if (a.beta != 0.0f) o = __builtin_fmaf(a.beta, load_value<kBf16>(a.C, row * a.ldc + col + e), o);
      if (a.bias) o += load_value<kBf16>(a.bias, bias0 + col + e);
    }
    v[e] = o;
  }
  const int64_t at = row * a.ldd + col;
  if constexpr (kBf16) {
    const auto d = (global_ptr<uint16_t>)a.D + at;
    if (wide && n >= 4) {
      *(global_ptr<u32x2>)d = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) d[e] = static_cast<uint16_t>(pack_bf16(v[e], 0.0f));
    }
  } else {
    const auto d = (global_ptr<float>)a.D + at;
    if (wide && n >= 4) {
      *(global_ptr<f32x4>)d = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) d[e] = v[e];
    }
  }
}

// Four neighbouring values at p + at, all inside and aligned for one load.
template <bool kBf16>
__device__ __forceinline__ f32x4 load_four(const void* p, int64_t at) {
  if constexpr (kBf16) {
    const u32x2 w = *(global_ptr<const u32x2>)((global_ptr<const uint16_t>)p + at);
    return f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
  } else {
    return *(global_ptr<const f32x4>)((global_ptr<const float>)p + at);
  }
}

// Whether D's rows allow a store of four values at once.
template <bool kBf16>
__device__ __forceinline__ bool wide_rows(const MxGemmArgs& a) {
  constexpr uint64_t es = kBf16 ? 2 : 4;
  return ((reinterpret_cast<uint64_t>(a.D) | static_cast<uint64_t>(a.ldd) * es) & (4 * es - 1)) == 0;
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// The caller has waited for what the other waves must see; no memory fence.
__device__ __forceinline__ void barrier_only() { asm volatile("s_barrier" ::: "memory"); }

}  // namespace mx
}  // namespace dg
