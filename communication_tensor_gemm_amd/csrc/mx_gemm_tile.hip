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
// half slabs.  Slabs go from memory straight into LDS (buffer_load_dwordx4
// ... lds, 1 KiB per wave instruction, whole rows of the slab), two stages of
// E2M1 or three of E4M3; the scales in chunks of 512 elements (16 bytes per
// row), two buffers.  While a half slab is multiplied from one set of
// registers, the next is read from LDS into the other; one barrier per slab
// says that every wave has read its second half, which frees the slab's
// stage for the loads of the slab two (E4M3: three) further on.
//
// Operand layout (see mx_gemm_rows.hip for the MFMA's): lane l has row l % 32
// and, with h = l / 32, an E2M1 block of 32 elements, or of E4M3 elements 16 h
// .. + 15 and 32 + 16 h .. + 15 of 64.  E2M1 x E2M1 takes the K order freely
// (both operands alike): half h of the lanes works on the h-th 128 elements of
// the slab, so that the four MFMAs of a slab use the four bytes of one dword
// of scales per lane, by op_sel.  With E4M3 the order is fixed inside 64, and
// the lane's dword of scales (four blocks, a slab) is shifted by h bytes once.
//
// LDS layout.  128-byte rows: blocks of 8 rows (1 KiB), half row s at + 512 s,
// row r at + 64 (r % 8), 16-byte piece q of the half at + 16 (q ^ f(r)), f(r) =
// ((r >> 1) ^ (r >> 2)) & 3: the 16 rows that one LDS cycle serves then fall
// on distinct banks.  64-byte rows: blocks of 16 rows, the same with one half.
//
// K past the end (K is a multiple of 32, not of the slab): the lanes whose
// piece of the last slab lies past K get an out-of-range offset once, before
// that slab's loads, and receive zeros; all earlier slabs are loaded unmasked.
#include "mx_tiles.h"

namespace dg {
namespace mx {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kXcds = 8;
constexpr int kChunkK = 512;  // elements of K per chunk of scales

__device__ __forceinline__ int row_perm(int row) { return ((row >> 1) ^ (row >> 2)) & 3; }

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8)); }
// The caller has waited for what the other waves must see; no memory fence.
__device__ __forceinline__ void barrier_only() { asm volatile("s_barrier" ::: "memory"); }

// acc += B block x A block, the scales' byte J of both dwords.  Inline asm
// with the accumulator tied to its AGPRs: the builtin's accumulators are
// copied between MFMAs when all 256 are in use.
template <int J>
__device__ __forceinline__ void mfma(f32x16& acc, const i32x4& b, const i32x4& a, int sb, int sa) {
#define DG_MX_MFMA(SEL, SELHI, FORMATS)                                                                              \
  asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:" SEL " op_sel_hi:" SELHI " " FORMATS \
               : "+a"(acc)                                                                                           \
               : "v"(b), "v"(a), "v"(sb), "v"(sa))
#define DG_MX_MFMA_BYTE(FORMATS)                       \
  if constexpr (J == 0)                                \
    DG_MX_MFMA("[0,0,0]", "[0,0,0]", FORMATS);         \
  else if constexpr (J == 1)                           \
    DG_MX_MFMA("[1,1,0]", "[0,0,0]", FORMATS);         \
  else if constexpr (J == 2)                           \
    DG_MX_MFMA("[0,0,0]", "[1,1,0]", FORMATS);         \
  else                                                 \
    DG_MX_MFMA("[1,1,0]", "[1,1,0]", FORMATS)
  DG_MX_MFMA_BYTE("cbsz:4 blgp:4");
}
template <int J>
__device__ __forceinline__ void mfma(f32x16& acc, const i32x4& b, const i32x8& a, int sb, int sa) {
  DG_MX_MFMA_BYTE("cbsz:4");
}
#undef DG_MX_MFMA_BYTE
#undef DG_MX_MFMA

template <bool A8, int NBM, int NBN>
struct Geo {
  typedef std::conditional_t<A8, i32x8, i32x4> AFrag;
  static constexpr int TM = 64 * NBM, TN = 64 * NBN;
  static constexpr int kSlabK = A8 ? 128 : 256;
  static constexpr int kRowB = A8 ? 64 : 128;  // bytes of a row of B per slab
  static constexpr int SA = TM * 128, SB = TN * kRowB;
  static constexpr int kStages = A8 ? 3 : 2;
  static constexpr int kScales = (TM + TN) * 16;
  static constexpr int kLds = kStages * (SA + SB) + 2 * kScales;
  static constexpr int LA = SA / 4096, LB = SB / 4096, LS = kScales / 4096;  // loads per wave
  static constexpr int kPerChunk = kChunkK / kSlabK;                         // slabs per chunk of scales
  static constexpr int kSteps = A8 ? 1 : 2;                                  // MFMAs of a block per half slab
};

// One tile: rows row0 .. + rows_left of A (and D), columns n0 .. of the B at
// row b_row0 + n0.  Every argument is workgroup-uniform.
template <bool A8, bool kBf16, int NBM, int NBN>
__device__ __forceinline__ void mx_tile(const MxGemmArgs& p, int32_t row0, int32_t rows_left, int32_t n0,
                                        int64_t b_row0, uint8_t* smem) {
  using G = Geo<A8, NBM, NBN>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5;
  const int32_t rows = min(rows_left, G::TM), cols = min(p.N - n0, G::TN);
  const uint32_t lda = static_cast<uint32_t>(A8 ? p.K : p.K / 2), ldb = static_cast<uint32_t>(p.K / 2);
  const uint32_t lds_pitch = static_cast<uint32_t>(scale_pitch(p.K));
  const auto rA = make_rsrc(p.A + static_cast<int64_t>(row0) * lda, rows * lda);
  const auto rB = make_rsrc(p.B + (b_row0 + n0) * ldb, cols * ldb);
  // this wave loads scales of A (waves 0, 1) or of B (2, 3)
  const bool scale_a = wave < 2;
  const auto rS = make_rsrc(scale_a ? p.As + static_cast<int64_t>(row0) * lds_pitch : p.Bs + (b_row0 + n0) * lds_pitch,
                            (scale_a ? rows : cols) * lds_pitch);
  const int KT = (p.K + G::kSlabK - 1) / G::kSlabK, KC = (p.K + kChunkK - 1) / kChunkK;

  // loads: lane offsets.  128-byte rows: even / odd blocks of 8 rows.
  uint32_t ga[2], gb[2];
  {
    const int half = lane >> 5, brow = (lane >> 2) & 7, piece = lane & 3;
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      const int r16 = 8 * odd + brow, at = 16 * (4 * half + (piece ^ row_perm(r16)));
      ga[odd] = (8 * G::LA * wave + r16) * lda + at;
      if constexpr (!A8) gb[odd] = (8 * G::LB * wave + r16) * ldb + at;
    }
    if constexpr (A8) {
      const int r16 = lane >> 2;
      gb[0] = gb[1] = (16 * G::LB * wave + r16) * ldb + 16 * (piece ^ row_perm(r16));
    }
  }
  const uint32_t gs = static_cast<uint32_t>((scale_a ? wave : wave - 2) * 64 * G::LS + lane) * lds_pitch;
  // the last slab's pieces past K
  const bool partial = KT * G::kSlabK != p.K;
  auto mask_last = [&]() {
    const int k0 = (KT - 1) * G::kSlabK;
    const int half = lane >> 5, brow = (lane >> 2) & 7, piece = lane & 3;
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      const int byte = 16 * (4 * half + (piece ^ row_perm(8 * odd + brow)));
      if (k0 + (A8 ? byte : 2 * byte) >= p.K) ga[odd] |= kOutOfRange;
      if constexpr (!A8)
        if (k0 + 2 * byte >= p.K) gb[odd] |= kOutOfRange;
    }
    if constexpr (A8)
      if (k0 + 32 * (piece ^ row_perm(lane >> 2)) >= p.K) gb[0] |= kOutOfRange;
  };
  auto stage = [&](int slab) { return smem + (slab % G::kStages) * (G::SA + G::SB); };
  uint8_t* const scales = smem + G::kStages * (G::SA + G::SB);
  // load d of the wave's LA + LB of slab kt
  auto load_slab = [&](uint8_t* st, int kt, int d) {
    if (d < G::LA) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_ptr_t)(st + (wave * G::LA + d) * 1024), 16,
                                               ga[d & 1] + (d >> 1) * 16 * lda, kt * 128, 0, 0);
    } else {
      const int e = d - G::LA;
      uint8_t* const to = st + G::SA + (wave * G::LB + e) * 1024;
      if constexpr (A8)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr_t)to, 16, gb[0] + e * 16 * ldb, kt * 64, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_ptr_t)to, 16, gb[e & 1] + (e >> 1) * 16 * ldb, kt * 128, 0, 0);
    }
  };
  auto load_scales = [&](int c) {
#pragma unroll
    for (int d = 0; d < G::LS; ++d)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rS, (lds_ptr_t)(scales + (c & 1) * G::kScales + (wave * G::LS + d) * 1024), 16,
                                               gs + d * 64 * lds_pitch, c * 16, 0, 0);
  };

  // fragment reads: lane bases within a stage
  uint32_t fa[4], fb[4];  // E2M1: piece 2 hs + odd; E4M3: A low / high half, B per half slab
  {
    const int ra = wm * 32 * NBM + (lane & 31), rb = wn * 32 * NBN + (lane & 31);
    const uint32_t a0 = (ra >> 3) * 1024 + (ra & 7) * 64;
    if constexpr (A8) {
      const uint32_t b0 = (rb >> 4) * 1024 + (rb & 15) * 64;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        fa[u] = a0 + 16 * ((2 * u + h) ^ row_perm(ra));
        fb[u] = G::SA + b0 + 16 * ((2 * u + h) ^ row_perm(rb));
        fa[2 + u] = fb[2 + u] = 0;
      }
    } else {
      const uint32_t b0 = (rb >> 3) * 1024 + (rb & 7) * 64;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        fa[q] = a0 + 512 * h + 16 * (q ^ row_perm(ra));
        fb[q] = G::SA + b0 + 512 * h + 16 * (q ^ row_perm(rb));
      }
    }
  }
  const uint32_t sa_at = (wm * 32 * NBM + (lane & 31)) * 16 + (A8 ? 0 : 4 * h);
  const uint32_t sb_at = (G::TM + wn * 32 * NBN + (lane & 31)) * 16 + (A8 ? 0 : 4 * h);

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
      const int odd = r / (NBM + NBN), in = r % (NBM + NBN);
      const int least = NBM < NBN ? NBM : NBN;
      const bool is_a = in < 2 * least ? (in & 1) == 0 : NBM > NBN;
      const int blk = in < 2 * least ? in >> 1 : in - least;
      if (is_a)
        F.a[blk][odd] = *reinterpret_cast<const i32x4*>(st + fa[2 * hs + odd] + 4096 * blk);
      else
        F.b[blk][odd] = *reinterpret_cast<const i32x4*>(st + fb[2 * hs + odd] + 4096 * blk);
    }
  };
  // dword r of slab kt's scales
  auto read_scale = [&](int kt, int r, int (&S)[NBM + NBN]) {
    const uint8_t* const at = scales + (kt / G::kPerChunk & 1) * G::kScales + (kt % G::kPerChunk) * (A8 ? 4 : 8);
    S[r] = *reinterpret_cast<const int*>(at + (r < NBM ? sa_at + 512 * r : sb_at + 512 * (r - NBM)));
  };

  f32x16 acc[NBM][NBN];
#pragma unroll
  for (int i = 0; i < NBM; ++i)
#pragma unroll
    for (int j = 0; j < NBN; ++j) acc[i][j] = f32x16{};

  constexpr int kMfmas = NBM * NBN * G::kSteps;  // per half slab
  constexpr int kLoads = G::LA + G::LB;
  Frags F0, F1;
  int S[NBM + NBN], Sn[NBM + NBN];

  // Half hs of slab kt on F: its MFMAs, with the reads of the next half slab
  // into Fn (kRead) and, in the second half, of the next slab's scales, and the
  // loads of slab kt_load (kLoad) placed behind given MFMAs.
  auto half_step = [&](auto hs_c, auto read_c, auto load_c, int kt, int kt_load, const Frags& F, Frags& Fn) {
    constexpr int hs = decltype(hs_c)::value;
    constexpr bool kRead = decltype(read_c)::value, kLoad = decltype(load_c)::value;
    const uint8_t* const from = stage(hs == 0 ? kt : kt + 1);
    uint8_t* const to = stage(kt_load);
    constexpr int kScaleReads = hs == 1 ? NBM + NBN : 0;
    constexpr int kAllReads = kReads + kScaleReads;
    // reads fill the first half of the MFMAs, loads all of them
    constexpr int kReadsPer = (kAllReads * 2 + kMfmas - 1) / kMfmas;
    constexpr int kLoadsPer = (kLoads + kMfmas - 1) / kMfmas;
    constexpr int kLoadEvery = kMfmas / kLoads > 0 ? kMfmas / kLoads : 1;
#pragma unroll
    for (int m = 0; m < kMfmas; ++m) {
      const int step = m / (NBM * NBN), i = m / NBN % NBM, j = m % NBN;
      if constexpr (A8) {
        mfma<2 * hs>(acc[i][j], F.b[j][0], F.a[i][0], S[NBM + j], S[i]);
      } else {
        if (step == 0)
          mfma<2 * hs>(acc[i][j], F.b[j][0], F.a[i][0], S[NBM + j], S[i]);
        else
          mfma<2 * hs + 1>(acc[i][j], F.b[j][G::kSteps - 1], F.a[i][G::kSteps - 1], S[NBM + j], S[i]);
      }
      if constexpr (kRead) {
#pragma unroll
        for (int u = 0; u < kReadsPer; ++u) {
          const int r = m * kReadsPer + u;
          if (r < kReads)
            read(from, hs ^ 1, r, Fn);
          else if (r < kAllReads)
            read_scale(kt + 1, r - kReads, Sn);
        }
      }
      if constexpr (kLoad) {
        if (m % kLoadEvery == 0) {
#pragma unroll
          for (int u = 0; u < kLoadsPer; ++u) {
            const int d = m / kLoadEvery * kLoadsPer + u;
            if (d < kLoads) load_slab(to, kt_load, d);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // the scales of the coming slab, from their reads; the MFMAs are opaque to
  // the compiler's hazard tracking, so the wait states between a VALU write of
  // an operand and its MFMA are given here
  auto take_scales = [&]() {
#pragma unroll
    for (int r = 0; r < NBM + NBN; ++r) {
      S[r] = A8 ? static_cast<int>(static_cast<uint32_t>(Sn[r]) >> (8 * h)) : Sn[r];
      asm volatile("" : "+v"(S[r]));
    }
    asm volatile("s_nop 3" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};
  constexpr std::true_type yes{};
  constexpr std::false_type no{};

  // prologue: the first stages, chunks 0 and 1 of the scales
  load_scales(0);
  if (KC > 1) load_scales(1);
#pragma unroll
  for (int t = 0; t < G::kStages; ++t) {
    if (t < KT) {
      if (partial && t == KT - 1) mask_last();
#pragma unroll
      for (int d = 0; d < kLoads; ++d) load_slab(stage(t), t, d);
    }
  }
  wait_vmcnt<0>();
  barrier_only();
#pragma unroll
  for (int r = 0; r < kReads; ++r) read(stage(0), 0, r, F0);
#pragma unroll
  for (int r = 0; r < NBM + NBN; ++r) read_scale(0, r, Sn);

  int kt = 0;
  for (; kt + G::kStages < KT; ++kt) {
    wait_lgkmcnt0();
    take_scales();
    half_step(first, yes, no, kt, 0, F0, F1);
    wait_lgkmcnt0();
    // slab kt + 1 has landed; E4M3: slab kt + 2 may still be on its way
    wait_vmcnt<(G::kStages - 2) * kLoads>();
    barrier_only();
    // this slab's stage is free, and so is its chunk's buffer after its last slab
    if (kt % G::kPerChunk == G::kPerChunk - 1 && kt / G::kPerChunk + 2 < KC) load_scales(kt / G::kPerChunk + 2);
    if (partial && kt + G::kStages == KT - 1) mask_last();
    half_step(second, yes, yes, kt, kt + G::kStages, F1, F0);
  }
  for (; kt + 1 < KT; ++kt) {  // nothing left to load
    wait_lgkmcnt0();
    take_scales();
    half_step(first, yes, no, kt, 0, F0, F1);
    wait_lgkmcnt0();
    wait_vmcnt<0>();
    barrier_only();
    half_step(second, yes, no, kt, 0, F1, F0);
  }
  wait_lgkmcnt0();
  take_scales();
  half_step(first, yes, no, kt, 0, F0, F1);
  wait_lgkmcnt0();
  half_step(second, no, no, kt, 0, F1, F0);
  // the last MFMAs' result latency, then every accumulator redefined behind it
  asm volatile("s_nop 7\n s_nop 7\n s_nop 7\n s_nop 7" ::: "memory");
#pragma unroll
  for (int i = 0; i < NBM; ++i)
#pragma unroll
    for (int j = 0; j < NBN; ++j) asm volatile("" : "+a"(acc[i][j]));

  // Epilogue.  A lane holds, of block (i, j), row l % 32 and columns 8 (r / 4)
  // + 4 h + r % 4.  A whole bf16 wave block without C goes through LDS, so
  // that a row is stored in 16-byte pieces; else four columns at a time.
  constexpr int WM = 32 * NBM, WN = 32 * NBN;
  const int32_t wrow = wm * WM, wcol = wn * WN;
  const int64_t bias0 = b_row0 + n0 + wcol;  // p.bias: N values per group, as B's rows
  int elane = lane;  // the epilogue's addresses are not hoisted above the loop
  asm volatile("" : "+v"(elane));
  const int el = elane & 31, eh = elane >> 5;
  if constexpr (kBf16) {
    constexpr int kPitch = WN * 2 + 16;  // padded: rows start on different banks
    static_assert(4 * WM * kPitch <= G::kLds, "epilogue LDS");
    const bool whole = rows - wrow >= WM && cols - wcol >= WN && p.beta == 0.0f &&
                       ((reinterpret_cast<uint64_t>(p.D) | (static_cast<uint64_t>(p.ldd) * 2)) & 15) == 0;
    barrier_only();  // every wave is past its reads of the stages
    if (whole) {
      uint8_t* const w = smem + wave * WM * kPitch;
#pragma unroll
      for (int i = 0; i < NBM; ++i)
#pragma unroll
        for (int j = 0; j < NBN; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int c = 32 * j + 8 * g + 4 * eh;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[e] = p.alpha * acc[i][j][4 * g + e];
              if (p.bias) v[e] += load_value<true>(p.bias, bias0 + c + e);
            }
            *reinterpret_cast<u32x2*>(w + (32 * i + el) * kPitch + 2 * c) =
                u32x2{bf16_rne(v[0]) | (bf16_rne(v[1]) << 16), bf16_rne(v[2]) | (bf16_rne(v[3]) << 16)};
          }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's own area: no barrier
      constexpr int kLanes = WN / 8, kRowsPer = 64 / kLanes;  // lanes per row, rows per instruction
      const int er = elane / kLanes, ec = elane % kLanes;
      uint16_t* const d = static_cast<uint16_t*>(p.D) + static_cast<int64_t>(row0 + wrow + er) * p.ldd + n0 + wcol + 8 * ec;
#pragma unroll
      for (int t = 0; t < WM / kRowsPer; ++t)
        *reinterpret_cast<u32x4*>(d + static_cast<int64_t>(t * kRowsPer) * p.ldd) =
            *reinterpret_cast<const u32x4*>(w + (t * kRowsPer + er) * kPitch + 16 * ec);
      return;
    }
  }
  const bool wide = wide_rows<kBf16>(p);
#pragma unroll
  for (int i = 0; i < NBM; ++i) {
    const int32_t r = wrow + 32 * i + el;
    if (r >= rows) continue;
#pragma unroll
    for (int j = 0; j < NBN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int32_t c = wcol + 32 * j + 8 * g + 4 * eh;
        if (c < cols)
          store_four<kBf16>(p, b_row0, row0 + r, n0 + c, cols - c, wide,
                            f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]});
      }
  }
}

// Height, in tiles, of a band of tile rows that is walked column by column.
constexpr int kBand = 4;

// Place w of the order of a tiles_m x tiles_n grid.
__device__ __forceinline__ void order_tile(int32_t w, int32_t tiles_m, int32_t tiles_n, int32_t& tm, int32_t& tn) {
  const int32_t band = w / (kBand * tiles_n), first = band * kBand;
  const int32_t high = min(kBand, tiles_m - first), in = w - band * kBand * tiles_n;
  tm = first + in % high;
  tn = in / high;
}

template <bool A8, bool kBf16, int NBM, int NBN>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(NBM* NBN == 16 ? 1 : 2, NBM* NBN == 16 ? 1 : 2)))
void mx_gemm_tile_kernel(MxGemmArgs p) {
  using G = Geo<A8, NBM, NBN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[G::kLds];
  const int32_t tiles_n = (p.N + G::TN - 1) / G::TN;
  const int32_t row_tiles = p.offsets ? count_group_tiles(p.offsets, p.groups, p.M, G::TM) : (p.M + G::TM - 1) / G::TM;
  // workgroup b runs on XCD b mod 8: each XCD takes one contiguous range of the tile order
  const int32_t T = row_tiles * tiles_n, x = static_cast<int32_t>(blockIdx.x) % kXcds, i = static_cast<int32_t>(blockIdx.x) / kXcds;
  const int32_t each = T / kXcds, more = T % kXcds;
  if (i >= each + (x < more ? 1 : 0)) return;
  const int32_t t = x * each + min(x, more) + i;
  int32_t tm, tn, row0 = 0, rows = p.M;
  int64_t b_row0 = 0;
  if (p.offsets) {
    const GroupTile g = find_group_tile(p.offsets, p.groups, p.M, G::TM, t / tiles_n);
    if (g.group < 0) return;
    // the group's tiles are a grid of their own, from its first row tile on
    row0 = g.row0 - g.index * G::TM;
    rows = g.rows + g.index * G::TM;
    b_row0 = static_cast<int64_t>(g.group) * p.N;
    order_tile(t - (t / tiles_n - g.index) * tiles_n, g.tiles, tiles_n, tm, tn);
  } else {
    order_tile(t, row_tiles, tiles_n, tm, tn);
  }
  mx_tile<A8, kBf16, NBM, NBN>(p, row0 + tm * G::TM, rows - tm * G::TM, tn * G::TN, b_row0, smem);
}

template <bool A8, bool kBf16, int NBM, int NBN>
static hipError_t tile_t(const MxGemmArgs& a, hipStream_t st) {
  using G = Geo<A8, NBM, NBN>;
  const int64_t row_tiles = a.offsets ? most_group_tiles(a.M, a.groups, G::TM) : (a.M + G::TM - 1) / G::TM;
  const int64_t T = row_tiles * ((a.N + G::TN - 1) / G::TN);
  if (T > INT32_MAX / 2) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((mx_gemm_tile_kernel<A8, kBf16, NBM, NBN>), dim3(static_cast<unsigned>((T + kXcds - 1) / kXcds * kXcds)),
                     dim3(256), 0, st, a);
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
