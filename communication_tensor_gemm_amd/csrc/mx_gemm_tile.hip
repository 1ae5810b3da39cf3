// MX product on square tiles, for many rows of A.
//
// Tiling.  A workgroup of four waves, 2 x 2, computes a tile of 64 NBM x 64
// NBN of D, each wave NBM x NBN blocks of 32 x 32 with
// v_mfma_scale_f32_32x32x64_f8f6f4, its accumulators in AGPRs.  The first
// MFMA operand is B and the second A, so a lane ends with four neighbouring
// columns of a row of D.
//
// K is walked in slabs of 128 bytes per row of A: 256 elements of E2M1 (128
// bytes per row of B too) or 128 of E4M3 (64 bytes per row of B), each in two
// halves.  Slabs go from memory straight into LDS (buffer_load_dwordx4 ...
// lds, 1 KiB per wave instruction, whole lines of 128 bytes where the rows
// allow it: slabs of 64 bytes per row, twice as many of them, measured 13%
// slower), two stages of E2M1 or three of E4M3; the scales in chunks of 512
// elements (16 bytes per row), two buffers.  While half a slab is multiplied
// from one set of registers, the next half is read from LDS into the other.
// One barrier per slab, between its halves, says that every wave has read
// the second half, which frees the slab's stage for the loads of the slab two
// (E4M3: three) further on, and that the next slab has landed.  MFMAs, reads
// and loads alternate in a fixed order (scheduling barriers keep it).  The
// scales' loads touch a line per lane, so they are placed in the half without
// other loads.
//
// Tile boundaries.  The launch is persistent: a workgroup's slabs form one
// stream over all of its tiles, and the loads, reads and scales of the next
// tile's first slabs are issued during the current tile's last ones, so a
// tile begins without waiting.  Its first MFMAs take 0 for their C operand.
// With one workgroup per CU, prologue and epilogue of a tile took 18 us of
// 127 (E2M1, K = 16384) when nothing overlapped them.
//
// Few tiles.  Where no CU has a second tile, a slab's 16 or so MFMAs per wave
// do not cover its loads' latency and its other instructions (0.7 us per slab,
// deeper stages or not).  With a long K, two groups of four waves then compute
// half of a tile's K each, with stages of their own, and the second group's
// sums go to the first through LDS at the end: 128 x 13312 x 16384 E2M1 69 -> 60
// us (E4M3 72 -> 70), 256 x 8192 x 8192 28 -> 25 (36 -> 34).  That end costs 1.5
// us, so for K up to 4096 one group is as fast or faster (256 x 8192 x 3584: 14.9
// us, with two 16.1; E4M3 19.1 and 20.7; at 200 x 8192 x 4096 two gain 3%, at 512 x
// 4096 x 4608 they lose 5% of E4M3).
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
// their products' sums are off by 1.7e-5 of the result's rms with normal data, for
// any K, without a bias to one side (an fp32 product: 3e-8).  It is the price
// of the 8-bit rate, a hundredth of what rounding D to bf16 costs.
//
// Operand layout (see mx_gemm_rows.hip for the other MFMA's): lane l has row
// l % 32 and, with h = l / 32, an E2M1 block of 32 elements, or of E4M3
// elements 16 h .. + 15 and 32 + 16 h .. + 15 of 64.  Its scale is that of
// block h of the 64, in both cases: of a dword of scales (four blocks, 128
// elements), byte h for the first 64 and 2 + h for the second, so the dword is
// shifted by h bytes once and op_sel takes bytes 0 and 2.
//
// LDS layout.  128-byte rows: blocks of 8 rows (1 KiB), half row s at + 512 s,
// row r at + 64 (r % 8), 16-byte piece q of the half at + 16 (q ^ f(r)), f(r) =
// ((r >> 1) ^ (r >> 2)) & 3: the 16 rows that one LDS cycle serves then fall
// on distinct banks.  64-byte rows: blocks of 16 rows, the same with one half.
//
// K past the end (K is a multiple of 32, not of the slab): the lanes whose
// piece of the last slab lies past K get an out-of-range offset for that
// slab's loads, and receive zeros; all other slabs are loaded unmasked.
#include "mx_tiles.h"

namespace dg {
namespace mx {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(2))) int i32x2;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kXcds = 8;

__device__ __forceinline__ int row_perm(int row) { return ((row >> 1) ^ (row >> 2)) & 3; }

__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8)); }

// acc += B block x A block, the scales' byte J of both dwords.  Inline asm
// with the accumulator tied to its AGPRs: the builtin's accumulators are
// copied between MFMAs when all 256 are in use.
#define DG_MX_MFMA(SELHI, FORMATS)                                                                               \
  asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:" SELHI " " FORMATS \
               : "+a"(acc)                                                                                       \
               : "v"(b), "v"(a), "v"(sb), "v"(sa))
template <int J>
__device__ __forceinline__ void mfma(f32x16& acc, const i32x4& b, const i32x4& a, int sb, int sa) {
  static_assert(J == 0 || J == 2, "scale byte");
  if constexpr (J == 0)
    DG_MX_MFMA("[0,0,0]", "cbsz:4 blgp:4");
  else
    DG_MX_MFMA("[1,1,0]", "cbsz:4 blgp:4");
}
template <int J>
__device__ __forceinline__ void mfma(f32x16& acc, const i32x4& b, const i32x8& a, int sb, int sa) {
  static_assert(J == 0 || J == 2, "scale byte");
  if constexpr (J == 0)
    DG_MX_MFMA("[0,0,0]", "cbsz:4");
  else
    DG_MX_MFMA("[1,1,0]", "cbsz:4");
}
#undef DG_MX_MFMA

template <bool A8, int NBM, int NBN>
struct Geo {
  typedef std::conditional_t<A8, i32x8, i32x4> AFrag;
  static constexpr int TM = 64 * NBM, TN = 64 * NBN;
  static constexpr int kSlabK = A8 ? 128 : 256;
  static constexpr int kRowB = A8 ? 64 : 128;  // bytes of a row of B per slab
  static constexpr int SA = TM * 128, SB = TN * kRowB, kStage = SA + SB;
  static constexpr int kStages = A8 ? 3 : 2;
  static constexpr int kScales = (TM + TN) * 16;
  static constexpr int kLds = kStages * kStage + 2 * kScales;
  static constexpr int LA = SA / 4096, LB = SB / 4096, LS = kScales / 4096;  // loads per wave
  static constexpr int kPerChunk = 512 / kSlabK;                             // slabs per chunk of scales
  static constexpr int kSteps = A8 ? 1 : 2;                                  // MFMAs of a block per half slab
  static constexpr int kWgs = NBM * NBN == 16 ? 1 : 2;                       // workgroups per CU
  static constexpr int kStores = NBM * NBN * 2;                              // of a whole bf16 wave block
};

// One tile's place.
struct Place {
  int32_t row0, rows;  // first row of A and D, rows from there on (0: no tile)
  int32_t n0, cols;
  int64_t b_row0;      // row of B that holds its group's column 0
};

// Height, in tiles, of a band of tile rows that is walked column by column.
constexpr int kBand = 4;

// Place w of the order of a tiles_m x tiles_n grid.
__device__ __forceinline__ void order_tile(int32_t w, int32_t tiles_m, int32_t tiles_n, int32_t& tm, int32_t& tn) {
  const int32_t band = w / (kBand * tiles_n), first = band * kBand;
  const int32_t high = min(kBand, tiles_m - first), in = w - band * kBand * tiles_n;
  tm = first + in % high;
  tn = in / high;
}

// The tiles of a launch in their order: workgroup b runs on XCD b mod 8, and
// each XCD takes one contiguous range of the order, its workgroups in turn.
struct Tiles {
  int32_t tiles_n, row_tiles, begin, end, step;
  GroupLanes groups;
};

// The launch's arguments read again where they are needed (scalar loads from
// the kernel's argument segment, which starts with them): held over the main
// loop they, and what the compiler derives from them ahead of it, would push
// the loop's own scalars out of the SGPRs.
__device__ __forceinline__ MxGemmArgs fresh_args() {
  typedef __attribute__((address_space(4))) const uint32_t* words_t;
  words_t q = (words_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(q));
  struct Words {
    uint32_t w[sizeof(MxGemmArgs) / 4];
  } a;
  static_assert(sizeof(MxGemmArgs) % 4 == 0, "whole words");
#pragma unroll
  for (size_t i = 0; i < sizeof(MxGemmArgs) / 4; ++i) a.w[i] = q[i];
  return __builtin_bit_cast(MxGemmArgs, a);
}

template <typename G>
__device__ __forceinline__ Tiles all_tiles(const MxGemmArgs& p) {
  Tiles t;
  t.tiles_n = tile_count(p.N, G::TN);
  if (p.offsets) {
    t.groups = load_groups(p.offsets, p.groups, p.M, G::TM);
    t.row_tiles = p.groups <= 64 ? __builtin_amdgcn_readlane(t.groups.incl, 63)
                                 : count_group_tiles(p.offsets, p.groups, p.M, G::TM);
  } else {
    t.row_tiles = tile_count(p.M, G::TM);
  }
  const int32_t T = t.row_tiles * t.tiles_n;
  const int32_t x = static_cast<int32_t>(blockIdx.x) % kXcds, each = T / kXcds, more = T % kXcds;
  t.begin = x * each + min(x, more) + static_cast<int32_t>(blockIdx.x) / kXcds;
  t.end = (x + 1) * each + min(x + 1, more);
  t.step = static_cast<int32_t>(gridDim.x) / kXcds;
  return t;
}

template <typename G>
__device__ __forceinline__ Place place_of(Tiles t, int32_t at) {
  const MxGemmArgs p = fresh_args();
  asm volatile("" : "+s"(t.tiles_n), "+s"(t.row_tiles));  // nothing of the divisions ahead of the loop either
  Place q{0, 0, 0, 0, 0};
  if (at >= t.end) return q;
  int32_t tm, tn, row0 = 0, rows = p.M;
  if (p.offsets) {
    const int32_t u = at / t.tiles_n;
    const GroupTile g = p.groups <= 64 ? group_tile_of(t.groups, 0, 0, G::TM, u)
                                       : find_group_tile(p.offsets, p.groups, p.M, G::TM, u);
    if (g.group < 0) return q;
    // the group's tiles are a grid of their own, from its first row tile on
    row0 = g.row0 - g.index * G::TM;
    rows = g.rows + g.index * G::TM;
    q.b_row0 = static_cast<int64_t>(g.group) * p.N;
    order_tile(at - (u - g.index) * t.tiles_n, g.tiles, t.tiles_n, tm, tn);
  } else {
    order_tile(at, t.row_tiles, t.tiles_n, tm, tn);
  }
  q.row0 = row0 + tm * G::TM;
  q.rows = min(rows - tm * G::TM, G::TM);
  q.n0 = tn * G::TN;
  q.cols = min(p.N - q.n0, G::TN);
  return q;
}

// The wave's block of D from its accumulators.  A lane holds, of block (i,
// j), row l % 32 and columns 8 g + 4 h + 0 .. 3 (g = 0 .. 3).  Whole columns of
// bf16 without C: the two halves of the wave exchange their fours of g and
// g + 1, so that each lane has eight neighbouring columns and an instruction
// stores 32 rows of 32 bytes, those past the last row out of the descriptor's
// range (kStores instructions in all, and true is returned); else four columns
// at a time.  No LDS: the next tile's slabs are in it.
template <bool kBf16, int NBM, int NBN>
__device__ __forceinline__ bool store_block_of(const MxGemmArgs& p, const Place& at, int wm, int wn, int lane,
                                               f32x16 (&acc)[NBM][NBN]) {
  constexpr int WM = 32 * NBM, WN = 32 * NBN;
  const int32_t wrow = wm * WM, wcol = wn * WN;
  // (a tile's rows within 2 GiB: offsets of 32 bits)
  const bool whole = kBf16 && at.cols - wcol >= WN && p.beta == 0.0f && p.ldd < (1 << 22) &&
                     ((reinterpret_cast<uint64_t>(p.D) | (static_cast<uint64_t>(p.ldd) * 2)) & 15) == 0;
  const bool wide = wide_rows<kBf16>(p);
  const uint32_t pitch = whole ? static_cast<uint32_t>(p.ldd) * 2 : 0;
  const auto rD = make_rsrc(static_cast<uint8_t*>(p.D) + (static_cast<int64_t>(at.row0) * p.ldd + at.n0) * 2, at.rows * pitch);
#pragma unroll
  for (int i = 0; i < NBM; ++i)
#pragma unroll
    for (int j = 0; j < NBN; ++j) {
      // one block at a time, its addresses from a lane index of its own, so that
      // nothing is computed ahead for all of them: the registers hold the loop's state
      __builtin_amdgcn_sched_barrier(0);
      int l = lane;
      asm volatile("" : "+v"(l));
      asm volatile("" : "+a"(acc[i][j]));
      const int el = l & 31, eh = l >> 5;
      const int32_t r = wrow + 32 * i + el, c0 = wcol + 32 * j;
      if (whole) {
        u32x2 w[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = p.alpha * acc[i][j][4 * g + e];
          if (p.bias) {  // N values per group, as B's rows
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += load_value<true>(p.bias, at.b_row0 + at.n0 + c0 + 8 * g + 4 * eh + e);
          }
          w[g] = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        }
        const uint32_t d = r * pitch + (c0 + 8 * eh) * 2;
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
          // the upper half's fours of g against the lower half's of g + 1
          const auto x = __builtin_amdgcn_permlane32_swap(w[g][0], w[g + 1][0], false, false);
          const auto y = __builtin_amdgcn_permlane32_swap(w[g][1], w[g + 1][1], false, false);
          __builtin_amdgcn_raw_buffer_store_b128(u32x4{x[0], y[0], x[1], y[1]}, rD, d + 16 * g, 0, 0);
        }
      } else if (r < at.rows) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int32_t c = c0 + 8 * g + 4 * eh;
          if (c < at.cols)
            store_four<kBf16>(p, at.b_row0, at.row0 + r, at.n0 + c, at.cols - c, wide,
                              f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]});
        }
      }
    }
  return whole;
}

// A workgroup's share of the launch.  KG = 2: of its one tile, two groups of four
// waves compute half of K each.
template <bool A8, bool kBf16, int NBM, int NBN, int KG>
__device__ __forceinline__ void run_tiles(const MxGemmArgs& p, uint8_t* const all_smem) {
  using G = Geo<A8, NBM, NBN>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  uint8_t* const smem = all_smem + kg * G::kLds;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5;
  const Tiles tiles = all_tiles<G>(p);
  int32_t at = tiles.begin;
  if (at >= tiles.end) return;

  Place cur = place_of<G>(tiles, at), next = place_of<G>(tiles, at + tiles.step);
  const uint32_t lda = static_cast<uint32_t>(A8 ? p.K : p.K / 2), ldb = static_cast<uint32_t>(p.K / 2);
  const uint32_t pitch = static_cast<uint32_t>(scale_pitch(p.K));
  // KG = 2: the first group takes whole chunks of scales, the second what is
  // left, K elements from kfrom on, and slabs of zeros up to the first one's number
  const int each = (p.K + 512 * KG - 1) / (512 * KG) * 512, kfrom = kg * each;
  const int K = KG == 1 ? static_cast<int>(p.K) : min(static_cast<int>(p.K) - kfrom, each);
  const int KT = ((KG == 1 ? K : each) + G::kSlabK - 1) / G::kSlabK, KC = ((KG == 1 ? K : each) + 511) / 512;
  const bool partial = KT * G::kSlabK != K;
  const uint32_t afrom = A8 ? kfrom : kfrom / 2, bfrom = kfrom / 2, sfrom = kfrom / kMxBlock;  // bytes of a row
  uint8_t* const scales = smem + G::kStages * G::kStage;

  // ---- loads.  The loader walks the workgroup's stream of slabs; lkt is its
  // slab of the tile that rA and rB describe.  (No tile: no bytes, all zeros.)
  __amdgpu_buffer_rsrc_t rA, rB, rS;
  auto slabs_of = [&](const Place& q) {
    const MxGemmArgs p = fresh_args();
    // no tile: no bytes, also with the second half's offset
    rA = make_rsrc(p.A + static_cast<int64_t>(q.row0) * lda + afrom, KG == 1 || q.rows ? q.rows * lda - afrom : 0);
    rB = make_rsrc(p.B + (q.b_row0 + q.n0) * ldb + bfrom, KG == 1 || q.rows ? q.cols * ldb - bfrom : 0);
  };
  // waves 0, 1 load scales of A, 2, 3 of B
  const bool scale_a = wave < 2;
  auto scales_of = [&](const Place& q) {
    const MxGemmArgs p = fresh_args();
    rS = make_rsrc((scale_a ? p.As + static_cast<int64_t>(q.row0) * pitch : p.Bs + (q.b_row0 + q.n0) * pitch) + sfrom,
                   KG == 1 || q.rows ? (scale_a ? q.rows : q.cols) * pitch - sfrom : 0);
  };
  // lane offsets: 128-byte rows in even and odd blocks of 8 rows, 64-byte rows in blocks of 16
  const int piece = lane & 3, r16 = lane >> 2;
  auto byte_in_slab = [&](int odd) { return 16 * (4 * (lane >> 5) + (piece ^ row_perm(8 * odd + (r16 & 7)))); };
  uint32_t ga[2], gb[2];
#pragma unroll
  for (int odd = 0; odd < 2; ++odd) {
    ga[odd] = (8 * G::LA * wave + 8 * odd + (r16 & 7)) * lda + byte_in_slab(odd);
    gb[odd] = A8 ? (16 * G::LB * wave + r16) * ldb + 16 * (piece ^ row_perm(r16))
                 : (8 * G::LB * wave + 8 * odd + (r16 & 7)) * ldb + byte_in_slab(odd);
  }
  const uint32_t gs = static_cast<uint32_t>((scale_a ? wave : wave - 2) * 64 * G::LS + lane) * pitch;
  int lkt = 0;
  // before the loads of slab lkt, K not a multiple of the slab: the last
  // slabs' pieces past K out of range, the first slab's back in
  auto mask = [&]() {
    const bool last = KG == 1 ? lkt == KT - 1 : (lkt + 1) * G::kSlabK > K;
    if (!partial || (lkt != 0 && !last)) return;
    const int k0 = lkt * G::kSlabK;
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      const int ka = k0 + byte_in_slab(odd) * (A8 ? 1 : 2);
      const int kb = A8 ? k0 + 32 * (piece ^ row_perm(r16)) : ka;
      ga[odd] = (ga[odd] & ~kOutOfRange) | (last && ka >= K ? kOutOfRange : 0u);
      gb[odd] = (gb[odd] & ~kOutOfRange) | (last && kb >= K ? kOutOfRange : 0u);
    }
  };
  constexpr int kLoads = G::LA + G::LB;
  // load d of the wave's of the loader's slab, into the stage at st
  auto load = [&](uint8_t* st, int d) {
    if (d < G::LA) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_ptr_t)(st + (wave * G::LA + d) * 1024), 16,
                                               ga[d & 1] + (d >> 1) * 16 * lda, lkt * 128, 0, 0);
    } else {
      const int e = d - G::LA;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr_t)(st + G::SA + (wave * G::LB + e) * 1024), 16,
                                               A8 ? gb[0] + e * 16 * ldb : gb[e & 1] + (e >> 1) * 16 * ldb,
                                               lkt * G::kRowB, 0, 0);
    }
  };
  // the loader's next slab, of its next tile past the last (with few slabs to
  // a tile, the loader is more than one tile ahead)
  int32_t lat = at;
  auto advance = [&]() {
    lkt = __builtin_amdgcn_readfirstlane(lkt + 1);
    if (lkt == KT) {
      lkt = 0;
      lat += tiles.step;
      slabs_of(place_of<G>(tiles, lat));
    }
  };
  auto load_scales = [&](int c, int buf, int d) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rS, (lds_ptr_t)(scales + buf * G::kScales + (wave * G::LS + d) * 1024), 16,
                                             gs + d * 64 * pitch, c * 16, 0, 0);
  };

  // ---- reads: lane bases within a stage, per 16-byte piece (E4M3's B: per half)
  uint32_t fa[2], fb[2];
  {
    const int ra = wm * 32 * NBM + (lane & 31), rb = wn * 32 * NBN + (lane & 31);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      fa[u] = (ra >> 3) * 1024 + (ra & 7) * 64 + 16 * ((2 * u + h) ^ row_perm(ra));
      fb[u] = G::SA + (A8 ? (rb >> 4) * 1024 + (rb & 15) * 64 : (rb >> 3) * 1024 + (rb & 7) * 64) +
              16 * ((2 * u + h) ^ row_perm(rb));
    }
  }
  const uint32_t sa_at = (wm * 32 * NBM + (lane & 31)) * 16, sb_at = (G::TM + wn * 32 * NBN + (lane & 31)) * 16;
  struct Frags {
    typename G::AFrag a[NBM][G::kSteps];
    i32x4 b[NBN][G::kSteps];
  };
  constexpr int kReads = 2 * NBM + G::kSteps * NBN;
  // read r of half hs of the slab in st
  auto read = [&](const uint8_t* st, int hs, int r, Frags& F) {
    if constexpr (A8) {
      if (r < 2 * NBM) {
        const int blk = r >> 1, u = r & 1;
        const i32x4 v = *reinterpret_cast<const i32x4*>(st + fa[u] + 512 * hs + 4096 * blk);
        if (u == 0)
          F.a[blk][0].lo = v;
        else
          F.a[blk][0].hi = v;
      } else {
        const int blk = r - 2 * NBM;
        F.b[blk][0] = *reinterpret_cast<const i32x4*>(st + fb[hs] + 2048 * blk);
      }
    } else {
      // A and B blocks in turn, the piece of the half's first MFMAs before the second's
      static_assert(NBM == NBN || A8, "reads in turn");
      const int u = r / (NBM + NBN), in = r % (NBM + NBN), blk = in >> 1;
      if ((in & 1) == 0)
        F.a[blk][u] = *reinterpret_cast<const i32x4*>(st + fa[u] + 512 * hs + 4096 * blk);
      else
        F.b[blk][u] = *reinterpret_cast<const i32x4*>(st + fb[u] + 512 * hs + 4096 * blk);
    }
  };
  // slab kt's scales (one dword of E4M3, two of E2M1) of the wave's row block r: A's, then B's
  i32x2 raw[NBM + NBN];
  auto read_scales = [&](int kt, int buf, int r) {
    const uint8_t* const q = scales + buf * G::kScales + (kt % G::kPerChunk) * (A8 ? 4 : 8) +
                             (r < NBM ? sa_at + 512 * r : sb_at + 512 * (r - NBM));
    if constexpr (A8)
      raw[r][0] = *reinterpret_cast<const int*>(q);
    else
      raw[r] = *reinterpret_cast<const i32x2*>(q);
  };
  // S: the dwords of scales in use, shifted so that bytes 0 and 2 are this
  // lane's: per half of an E2M1 slab, or (one set) of an E4M3 slab with the
  // next slab's in the other set.  Each is made from raw during the half
  // before its use, in the shadow of the MFMAs.
  int S[2][NBM + NBN];
  // a scale byte past K may hold anything, also the NaN scale: the bytes of
  // dword `dword` of slab kt that count
  auto keep_of = [&](int kt, int dword) -> uint32_t {
    if (!partial || (KG == 1 ? kt != KT - 1 : (kt + 1) * G::kSlabK <= K)) return ~0u;
    const int left = K - kt * G::kSlabK - 128 * dword;
    return left >= 128 ? ~0u : left <= 0 ? 0u : (1u << (left / 4)) - 1u;
  };
  auto make_scale = [&](int set, int r, int dword, uint32_t keep) {
    S[set][r] = static_cast<int>((static_cast<uint32_t>(raw[r][dword]) & keep) >> (8 * h));
  };
  // The MFMAs are opaque to the compiler's hazard tracking: the wait states
  // between a VALU write of an operand and its MFMA are given here, behind the
  // definition of every S that the half uses.
  auto settle_scales = [&](int set) {
#pragma unroll
    for (int r = 0; r < NBM + NBN; ++r) asm volatile("" : "+v"(S[set][r]));
    asm volatile("s_nop 1" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  f32x16 acc[NBM][NBN];
  constexpr int kBlocks = NBM * NBN, kMfmas = kBlocks * G::kSteps;
  Frags F0, F1;
  // Half hs of a slab on F: its MFMAs, and placed behind given ones the reads
  // of the next half slab (at st) into Fn; in the first half, LS loads of the
  // scale chunk c into buffer sbuf (c < 0: none); in the second, the reads of
  // the next slab's scales and the loads of the loader's slab into `to`; in
  // the last quarter, the next half's scales from raw (`keep` of them).
  auto half_step = [&](auto hs_c, const uint8_t* st, uint8_t* to, int kt_next, int buf_next, int c, int sbuf, uint32_t keep,
                       const Frags& F, Frags& Fn) {
    constexpr int hs = decltype(hs_c)::value;
    constexpr int kSet = A8 ? 0 : hs, kMake = A8 ? 1 : hs ^ 1;
    constexpr int kAll = kReads + (hs == 1 ? NBM + NBN : 0);
    // reads fill the first half of the MFMAs, loads all of them
    constexpr int kReadsPer = (kAll * 2 + kMfmas - 1) / kMfmas;
    constexpr int kLoadsPer = (kLoads + kMfmas - 1) / kMfmas, kLoadEvery = kMfmas / kLoads > 0 ? kMfmas / kLoads : 1;
    constexpr int kMakeAt = kMfmas * 3 / 4, kMakePer = (NBM + NBN) / (kMfmas - kMakeAt);
    static_assert(kMakePer * (kMfmas - kMakeAt) == NBM + NBN, "scales in the last quarter");
#pragma unroll
    for (int m = 0; m < kMfmas; ++m) {
      const int u = m / kBlocks, i = m / NBN % NBM, j = m % NBN;
      if constexpr (A8)
        mfma<2 * hs>(acc[i][j], F.b[j][0], F.a[i][0], S[kSet][NBM + j], S[kSet][i]);
      else if (u == 0)
        mfma<0>(acc[i][j], F.b[j][0], F.a[i][0], S[kSet][NBM + j], S[kSet][i]);
      else
        mfma<2>(acc[i][j], F.b[j][G::kSteps - 1], F.a[i][G::kSteps - 1], S[kSet][NBM + j], S[kSet][i]);
#pragma unroll
      for (int v = 0; v < kReadsPer; ++v) {
        const int r = m * kReadsPer + v;
        if (r < kReads)
          read(st, hs ^ 1, r, Fn);
        else if (r < kAll)
          read_scales(kt_next, buf_next, r - kReads);
      }
      if constexpr (hs == 1) {
        if (m % kLoadEvery == 0) {
#pragma unroll
          for (int v = 0; v < kLoadsPer; ++v)
            if (m / kLoadEvery * kLoadsPer + v < kLoads) load(to, m / kLoadEvery * kLoadsPer + v);
        }
      } else {
#pragma unroll
        for (int d = 0; d < G::LS; ++d)
          if (m == kMfmas / 8 + d * kMfmas / G::LS && c >= 0) load_scales(c, sbuf, d);
      }
      if constexpr (hs == 1 || !A8) {
        if (m >= kMakeAt) {
#pragma unroll
          for (int v = 0; v < kMakePer; ++v) make_scale(kMake, (m - kMakeAt) * kMakePer + v, hs == 1 ? 0 : 1, keep);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // The accumulators to zero, by MFMAs of zeros without a C operand: tied in
  // place like all their other writes, and half the cycles of 256 VALU writes.
  auto clear = [&]() {
    i32x4 zero = {0, 0, 0, 0};
    asm volatile("" : "+v"(zero));
    asm volatile("s_nop 3");
#pragma unroll
    for (int i = 0; i < NBM; ++i)
#pragma unroll
      for (int j = 0; j < NBN; ++j)
        asm volatile("v_mfma_f32_32x32x64_f8f6f4 %0, %1, %1, 0 cbsz:4 blgp:4" : "+a"(acc[i][j]) : "v"(zero));
  };
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};

  // ---- the stream's first stages and its first chunk of scales
  slabs_of(cur);
  scales_of(cur);
#pragma unroll
  for (int d = 0; d < G::LS; ++d) load_scales(0, 0, d);
#pragma unroll
  for (int t = 0; t < G::kStages; ++t) {
    mask();
#pragma unroll
    for (int d = 0; d < kLoads; ++d) load(smem + t * G::kStage, d);
    advance();
  }
  clear();
  wait_vmcnt<(G::kStages - 1) * kLoads>();
  barrier_only();
  uint8_t *s0 = smem, *s1 = smem + G::kStage;  // stages of this slab and the next
#pragma unroll
  for (int r = 0; r < kReads; ++r) read(s0, 0, r, F0);
#pragma unroll
  for (int r = 0; r < NBM + NBN; ++r) read_scales(0, 0, r);

#pragma unroll
  for (int r = 0; r < NBM + NBN; ++r) make_scale(A8 ? 1 : 0, r, 0, keep_of(0, 0));

  int buf = 0, kv = 0;   // buffer of the current chunk of scales; slab of the current tile
  bool behind = false;   // kStores stores were issued since the last loads of a slab
  for (;;) {
    const int kt = __builtin_amdgcn_readfirstlane(kv);
    const bool last = kt + 1 == KT;
    const int kt_next = last ? 0 : kt + 1;
    // the chunk of scales after this one, loaded at its first slab: what its
    // buffer held was used up before the last barrier
    int c = -1;
    if (kt % G::kPerChunk == 0) {
      c = kt / G::kPerChunk + 1;
      if (c == KC) {
        c = 0;
        scales_of(next);
      }
    }
    // what the barrier waits for: the next slab has landed, and so has the next
    // chunk of scales if it is read now.  Operations retire in order, and behind
    // the next slab's loads are those of the slabs after it, a tile's stores
    // and the scales' loads.
    const int wait = last && kt % G::kPerChunk == 0 ? 2 : kt == 0 && behind ? 1 : 0;
    wait_lgkmcnt0();
    if constexpr (A8) {
#pragma unroll
      for (int r = 0; r < NBM + NBN; ++r) S[0][r] = S[1][r];
    }
    settle_scales(0);
    half_step(first, s0, nullptr, 0, 0, c, buf ^ 1, A8 ? 0u : keep_of(kt, 1), F0, F1);
    wait_lgkmcnt0();
    if constexpr (!A8) settle_scales(1);
    if (wait == 0)
      wait_vmcnt<(G::kStages - 2) * kLoads>();
    else if (wait == 1)
      wait_vmcnt<(G::kStages - 2) * kLoads + G::kStores + G::LS>();
    else
      wait_vmcnt<0>();
    barrier_only();
    if (kt_next % G::kPerChunk == 0) buf ^= 1;
    mask();
    half_step(second, s1, s0, kt_next, buf, -1, 0, keep_of(kt_next, 0), F1, F0);
    advance();
    s0 = s1;
    s1 = s1 + G::kStage == scales ? smem : s1 + G::kStage;
    kv = kt_next;
    if (last) {
      // the last MFMAs' result latency, then every accumulator redefined behind it
      asm volatile("s_nop 7\n s_nop 7\n s_nop 7\n s_nop 7" ::: "memory");
#pragma unroll
      for (int i = 0; i < NBM; ++i)
#pragma unroll
        for (int j = 0; j < NBN; ++j) asm volatile("" : "+a"(acc[i][j]));
      if constexpr (KG == 2) {
        // the second group's sums to the first, through the second's stages: all
        // of its slabs have been read, and no load into them is under way
        static_assert(G::kStages * G::kStage >= NBM * NBN * 4 * 4096, "room for the sums");
        wait_vmcnt<0>();
        barrier_only();
        f32x4* const sums = reinterpret_cast<f32x4*>(all_smem + G::kLds) + wave * NBM * NBN * 4 * 64 + lane;
        if (kg == 1) {
#pragma unroll
          for (int b = 0; b < NBM * NBN; ++b)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const f32x16& v = acc[b / NBN][b % NBN];
              sums[(b * 4 + g) * 64] = f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
            }
        }
        wait_lgkmcnt0();
        barrier_only();
        if (kg == 1) return;
#pragma unroll
        for (int b = 0; b < NBM * NBN; ++b)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 v = sums[(b * 4 + g) * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b / NBN][b % NBN][4 * g + e] += v[e];
          }
      }
      int elane = lane;  // the epilogue's addresses are not hoisted above the loop
      asm volatile("" : "+v"(elane));
      behind = store_block_of<kBf16, NBM, NBN>(fresh_args(), cur, wm, wn, elane, acc);
      if (KG == 2 || next.rows == 0) return;
      clear();
      at += tiles.step;
      cur = next;
      next = place_of<G>(tiles, at + tiles.step);
      // the next tile's first fragments once more: kept in registers over the
      // epilogue they would push others out to memory, and every slab's waits
      // would then include those
#pragma unroll
      for (int r = 0; r < kReads; ++r) read(s0, 0, r, F0);
#pragma unroll
      for (int r = 0; r < NBM + NBN; ++r) read_scales(0, buf, r);
#pragma unroll
      for (int r = 0; r < NBM + NBN; ++r) make_scale(A8 ? 1 : 0, r, 0, keep_of(0, 0));
    }
  }
}

template <bool A8, bool kBf16, int NBM, int NBN, int KG>
__global__ __launch_bounds__(256 * KG) __attribute__((amdgpu_waves_per_eu(NBM* NBN == 16 ? 1 : 2, NBM* NBN == 16 ? 1 : 2)))
void mx_gemm_tile_kernel(MxGemmArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[KG * Geo<A8, NBM, NBN>::kLds];
  run_tiles<A8, kBf16, NBM, NBN, KG>(p, smem);
}

template <bool A8, bool kBf16, int NBM, int NBN>
static hipError_t tile_t(const MxGemmArgs& a, hipStream_t st) {
  using G = Geo<A8, NBM, NBN>;
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
