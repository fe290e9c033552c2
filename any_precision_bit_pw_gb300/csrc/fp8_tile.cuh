// Products of e4m3 matrices with a scale per row and 128 columns of the
// activations and per 128 x 128 block of the weights, on tcgen05 tiles: the kernel
// of fp8_linear.cu (one weight) and of fp8_gated.cu (two, with the activation and the
// product of both in its epilogue), and the loads of their kernels for few tokens.
#pragma once

#include <type_traits>

#include "ops_common.cuh"
#include "umma.cuh"

namespace pw_fp8 {

struct LinearParams {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  void* y;
  int64_t lda, ldb, ldy, sa_stride, sb_stride;
  int M, N, K, KB;
  int splits;       // CTAs of a cluster that share a tile's groups
  int32_t* status;
  bool wide_b;      // rows of b start at 32-byte addresses
  bool wide_y;      // rows of y start at 16-byte addresses
  bool wide_scales; // scales through tensor maps
};

// The gated block: b and sb are the gate's weight, h = act(a b^T) * (a u^T) goes to y
// and / or to e4m3 codes q with a scale per 128 columns.
struct GatedParams : LinearParams {
  const uint8_t* u;
  const float* su;
  uint8_t* q;
  float* scale;
  int64_t ldu, su_stride, ldq, scale_stride;
  int act;          // PW_ACT_*
  bool wide_q;      // rows of q start at 16-byte addresses
};

// act(g) * u, of two columns.  Both activations are g / (1 + 2^-t): t is g log2(e)
// for SiLU, and for GELU by its tanh form 1/2 g (1 + tanh x) the same with 2 x for g,
// which does not cancel for negative g.  (2^-t may be an infinity: the quotient is 0.)
__device__ __forceinline__ uint64_t gated2(uint64_t g, uint64_t u, int act) {
  constexpr float kLog2e = 1.4426950408889634f, kGelu = -2.0f * 0.7978845608028654f * kLog2e;
  uint64_t t;   // -t
  if (act == PW_ACT_SILU) {
    t = pw::mul_f32x2(g, pw::twice(-kLog2e));
  } else {
    const uint64_t square = pw::mul_f32x2(g, g);
    t = pw::mul_f32x2(g, pw::fma_f32x2(square, pw::twice(0.044715f * kGelu), pw::twice(kGelu)));
  }
  float lo, hi;
  pw::unpack_f32x2(t, lo, hi);
  const uint64_t e = pw::pack_f32x2(__float_as_uint(pw::exp2_fast(lo)), __float_as_uint(pw::exp2_fast(hi)));
  pw::unpack_f32x2(pw::add_f32x2(e, pw::twice(1.0f)), lo, hi);
  const uint64_t r = pw::pack_f32x2(__float_as_uint(pw::reciprocal_fast(lo)), __float_as_uint(pw::reciprocal_fast(hi)));
  return pw::mul_f32x2(pw::mul_f32x2(g, r), u);
}
__device__ __forceinline__ float gated(float g, float u, int act) {
  float lo, hi;
  pw::unpack_f32x2(gated2(pw::twice(g), pw::twice(u), act), lo, hi);
  return lo;
}

// 16 bytes at column k of a row; columns from K on are 0.
__device__ __forceinline__ uint4 load16(const uint8_t* row, int k, int K, bool valid) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (!valid || k >= K) return v;
  if (k + 16 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 15; ++i)
    if (k + i < K) w[i / 4] |= static_cast<uint32_t>(row[k + i]) << (8 * (i % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 32 bytes at column k, by one load where `wide`.
__device__ __forceinline__ void load32(const uint8_t* row, int k, int K, bool valid, bool wide, uint32_t (&v)[8]) {
  if (wide && valid && k + 32 <= K) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(row + k));
    return;
  }
  const uint4 lo = load16(row, k, K, valid), hi = load16(row, k + 16, K, valid);
  v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
  v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
}

// ---------------------------------------------------------------------------
// More tokens: tiles on the tcgen05 tensor cores.  The MMAs of one 128-column
// group write a fresh accumulator in Tensor Memory; eight warps read it,
// multiply by the group's scales and add to sums in registers, while the next
// group's MMAs fill the other accumulator.  Tokens are the lanes of Tensor
// Memory, so a thread owns one token and has one scale product per group.
//
//  kPair: 256 tokens x 256 weight rows by a pair of CTAs, persistent.  Each
//    CTA holds half of both operands, so a group costs its shared memory 32 KB
//    in and 32 KB out for 512 cycles of matrix work: at 128 bytes a cycle both
//    are busy to the end.  (128 x 128 by one CTA move twice that for the same
//    work: 406 us instead of 310 for 8192 x 8192 x 6144.)
//  otherwise: 128 x 128 by one CTA, for fewer tokens; with few tiles the groups
//    are split among the CTAs of a cluster, which add their sums through
//    distributed shared memory, in the order of their ranks.
// ---------------------------------------------------------------------------
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr int kBoxBytes = 128;      // one group of columns: a swizzled row
constexpr int kSumWarps = 8;
constexpr int kCopyWarp = kSumWarps, kMmaWarp = kSumWarps + 1;

constexpr int kOutBytes = 32 * 64 * 2;     // 32 rows x 64 columns of 16-bit results on their way out, of one warp
constexpr int kScaleSlots = 8;
constexpr int kTokenScaleBytes = 128 * 16;             // the token scales of four groups
constexpr int kScaleBytes = kTokenScaleBytes + 128;    // and the weight scales of the tile's 128-row blocks
constexpr int kGatedScaleBytes = kTokenScaleBytes + 256;   // of both weights, each at a copy's alignment

template <int kTokens, int kWide, bool kGated>
struct Tile {
  static constexpr bool kPair = kTokens == 256;
  static constexpr int kM = kTokens;                  // tokens
  static constexpr int kN = kWide;                    // weight rows
  static constexpr int kRowsA = kPair ? 128 : kM;     // of both, in one CTA's shared memory
  static constexpr int kRowsB = kPair ? kN / 2 : kN;
  static constexpr int kCols = kN / 2;                // of one warpgroup's sums
  static constexpr int kQuarters = kRowsA / 32;       // warps of a warpgroup with tokens
  // 32 KB (pairs: half of both operands) and 24 KB a stage; single CTAs with 256 weight rows 48 and 40 KB
  static constexpr int kStages = kN == 256 && !kPair ? (kRowsA == 128 ? 3 : 4) : kRowsA == 128 ? 5 : 7;
  static constexpr int kAccs = 512 / kN;              // accumulators in Tensor Memory
  static constexpr bool kMove = kN == 256;            // registers move to the sums
  static constexpr int kThreads = kMove ? 384 : 320;  // whole warpgroups for that
  static constexpr int kStageBytes = (kRowsA + kRowsB) * kBoxBytes;
  static constexpr int kSlotBytes = kGated ? kGatedScaleBytes : kScaleBytes;
  static constexpr int kSmem = kStages * kStageBytes + kSumWarps * kOutBytes + kScaleSlots * kSlotBytes + 1024;
  static constexpr int kPartRow = kN + 4;   // floats of a row of sums in shared memory: 16-byte lanes on distinct banks
  static constexpr int kOutN = kGated ? kN / 2 : kN;   // columns of the result
  static_assert(kSmem <= 227 * 1024 && (kPair || kRowsA * kPartRow * 4 <= kStages * kStageBytes), "shared memory");
  static constexpr bool kCodes = kGated && kOutN == 128;   // a tile has whole groups of the result's scales
  static constexpr int kHalf = kGated ? kCols / 2 : kCols;  // of the result's columns a thread has
};
template <bool kGated>
using Params = typename std::conditional<kGated, GatedParams, LinearParams>::type;
template <bool kGated>
struct Maps {
  CUtensorMap a, b, y, sa, sb;
};
template <>
struct Maps<true> {
  CUtensorMap a, b, y, sa, sb, u, su;
};

struct alignas(8) TileShared {
  uint64_t full[7], empty[7], done[4], read[4], scales[kScaleSlots], drained;
  uint32_t tmem;
  int dead;   // a wait ran out: everybody leaves
};
// The largest magnitudes of 64 columns of the result, of each row: the two warps
// that have a row's 128 exchange them.
struct alignas(8) GatedShared {
  uint64_t met[4];        // a barrier a pair of warps
  float top[2][2][128];   // [tile's parity][side][row]
};

__device__ __forceinline__ bool wait(const uint64_t& bar, uint32_t parity, TileShared& sh, const LinearParams& p) {
  return pw::warp_wait(&bar, parity, &sh.dead, p.status);
}

// A warp's 32 rows of kW 16-bit results (a thread has a row, in pairs) to rows of y at
// any address: through shared memory, so that a store covers neighbouring columns of a
// row (value by value from its owner, a store touches 32 rows: 8192 x 8191 x 6144 takes
// 839 us, 324 so; gated 2000 x 1500 x 256 36 and 11).  Columns from
// `left` and rows from `rows` on are not written.
template <typename T, int kW>
__device__ __forceinline__ void store_rows(const uint64_t* sum, T* y, int64_t ldy, int rows, int left, unsigned char* out) {
  constexpr int kUnits = kW / 8, kRow = 2 * kW;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      pw::unpack_f32x2(sum[4 * i + j], lo, hi);
      w[j] = pw::pack2<T>(lo, hi);
    }
    *reinterpret_cast<uint4*>(out + lane * kRow + ((i ^ (lane & (kUnits - 1))) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  // two columns a lane; 64 columns take a warp, 32 half of one
  constexpr int kAtOnce = 64 / kW;
  const int col = 2 * (lane % (kW / 2)), unit = col >> 3;
  const bool pairs = (reinterpret_cast<uintptr_t>(y) & 3) == 0 && ldy % 2 == 0;
#pragma unroll 4
  for (int r0 = 0; r0 < 32; r0 += kAtOnce) {
    const int r = r0 + lane / (kW / 2);
    if (r >= rows || col >= left) continue;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(out + r * kRow + ((unit ^ (r & (kUnits - 1))) << 4) + 2 * (col & 7));
    uint16_t* to = reinterpret_cast<uint16_t*>(y + r * ldy + col);
    if (pairs && col + 1 < left) {
      *reinterpret_cast<uint32_t*>(to) = w;
    } else {
      to[0] = static_cast<uint16_t>(w);
      if (col + 1 < left) to[1] = static_cast<uint16_t>(w >> 16);
    }
  }
  __syncwarp();   // the memory is free again
}

// Tiles in strips of 2048 tokens, so that the CTAs that run at the same time
// share both operands through L2.
template <int kM>
__device__ __forceinline__ void tile_at(int tile, int tiles_m, int tiles_n, int& mt, int& nt) {
  constexpr int kStrip = 2048 / kM;
  const int per_strip = kStrip * tiles_n, strip = tile / per_strip, r = tile - strip * per_strip;
  const int height = min(kStrip, tiles_m - strip * kStrip);
  nt = r / height;
  mt = strip * kStrip + r - nt * height;
}

//
// Gated: a tile's weight rows are 128 (or 64, for 16-bit results only) of the gate's and
// the same of the other weight (of a pair, a CTA loads one of them); a thread sums 64
// (32) columns of each, so that the activation and the product are its own.
//
// kRagged: rows of y do not start at 16-byte addresses.  (Apart, because the other
// kernel is 4 % slower with those stores in it: 8192 x 8192 x 6144 281 and 294 us.)
template <typename T, int kTokens, int kWide, bool kGated, bool kRagged>
__global__ void __launch_bounds__(Tile<kTokens, kWide, kGated>::kThreads, 1)
    linear_tile_kernel(const __grid_constant__ Params<kGated> p, const __grid_constant__ Maps<kGated> maps) {
  using C = Tile<kTokens, kWide, kGated>;
  constexpr bool kPair = C::kPair;
  extern __shared__ unsigned char smem_raw[];
  __shared__ TileShared sh;
  __shared__ typename std::conditional<kGated, GatedShared, char>::type gsh;
  unsigned char* smem = smem_raw + ((1024u - (pw::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t stages = pw::smem_u32(smem);
  const int warp = pw::uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int tiles_m = (p.M + C::kM - 1) / C::kM, tiles_n = (p.N + C::kOutN - 1) / C::kOutN, tiles = tiles_m * tiles_n;
  // the CTA's place: rank in its pair, or its share of the groups
  const int rank = kPair || p.splits > 1 ? static_cast<int>(pw::cluster_rank()) : 0;
  const int group_size = kPair ? 2 : p.splits;
  const int first_tile = blockIdx.x / group_size, tile_step = gridDim.x / group_size;
  const int kb0 = kPair ? 0 : p.KB * rank / p.splits, kb1 = kPair ? p.KB : p.KB * (rank + 1) / p.splits;
  const uint32_t scale_smem = stages + C::kStages * C::kStageBytes + kSumWarps * kOutBytes;
  // Copies of one group (the copy warp).
  pw::Ring<C::kStages> stage;
  pw::Ring<kScaleSlots> slot;
  uint32_t x = 0, fours = 0;   // groups, and fours of groups, started
  auto start_group = [&](int kb, int mt, int nt) {
    const int row_a = mt * C::kM + (kPair ? 128 * rank : 0), row_b = nt * C::kOutN + (kPair && !kGated ? C::kRowsB * rank : 0);
    const uint32_t bar = pw::smem_u32(&sh.full[stage.at]), dst = stages + stage.at * C::kStageBytes;
    if (p.wide_scales && (kb == kb0 || (kb & 3) == 0)) {
      // The slot is free: the MMAs of group x - kStages are done, they were
      // issued after every warp had read the accumulator of group x - kStages -
      // kAccs (at most 11 back), and the slot's last user is at least 14 back
      // (seven fours of a tile of two groups or more).
      const uint32_t sbar = pw::smem_u32(&sh.scales[slot.at]), sdst = scale_smem + slot.at * C::kSlotBytes;
      if (pw::elect_one()) {
        pw::mbar_arrive_expect_tx(sbar, 16 * (C::kRowsA + (kGated ? 2 : C::kN / 128)));
        pw::tma_load_2d(sdst, &maps.sa, kb & ~3, row_a, sbar);
        pw::tma_load_2d(sdst + kTokenScaleBytes, &maps.sb, kb & ~3, nt * C::kOutN / 128, sbar);
        if constexpr (kGated) pw::tma_load_2d(sdst + kTokenScaleBytes + 128, &maps.su, kb & ~3, nt * C::kOutN / 128, sbar);
      }
      ++fours;
      slot.next();
      __syncwarp();
    }
    if (pw::elect_one()) {
      if constexpr (kPair) {
        // both CTAs' copies complete on the first one's barrier
        if (rank == 0) pw::mbar_arrive_expect_tx(bar, 2 * C::kStageBytes);
        const uint32_t lead = pw::map_shared(bar, 0);
        pw::tma_load_2d_pair(dst, &maps.a, kb * pw::kGroup, row_a, lead);
        const CUtensorMap* mine = &maps.b;
        if constexpr (kGated) mine = rank ? &maps.u : &maps.b;
        pw::tma_load_2d_pair(dst + C::kRowsA * kBoxBytes, mine, kb * pw::kGroup, row_b, lead);
      } else {
        pw::mbar_arrive_expect_tx(bar, C::kStageBytes);
        pw::tma_load_2d(dst, &maps.a, kb * pw::kGroup, row_a, bar);
        pw::tma_load_2d(dst + C::kRowsA * kBoxBytes, &maps.b, kb * pw::kGroup, row_b, bar);
        if constexpr (kGated) pw::tma_load_2d(dst + (C::kRowsA + C::kOutN) * kBoxBytes, &maps.u, kb * pw::kGroup, row_b, bar);
      }
    }
    stage.next();
    ++x;
    __syncwarp();
  };
  int kb_early = kb0;   // groups of the first tile that are under way before the set-up is done
  if (warp == kCopyWarp) {
    if (pw::elect_one()) {
      pw::prefetch_tmap(&maps.a);
      pw::prefetch_tmap(&maps.b);
      if constexpr (kGated) pw::prefetch_tmap(&maps.u);
      for (int i = 0; i < C::kStages; ++i) {
        pw::mbar_init(pw::smem_u32(&sh.full[i]), 1);
        pw::mbar_init(pw::smem_u32(&sh.empty[i]), 1);
      }
      for (int i = 0; i < C::kAccs; ++i) {
        pw::mbar_init(pw::smem_u32(&sh.done[i]), 1);
        pw::mbar_init(pw::smem_u32(&sh.read[i]), 2 * C::kQuarters * (kPair ? 2 : 1));
      }
      for (int i = 0; i < kScaleSlots; ++i) pw::mbar_init(pw::smem_u32(&sh.scales[i]), 1);
      pw::mbar_init(pw::smem_u32(&sh.drained), 1);
      if constexpr (kGated)
        for (int i = 0; i < 4; ++i) pw::mbar_init(pw::smem_u32(&gsh.met[i]), 2);
      sh.dead = 0;
      pw::mbar_init_fence();
    }
    __syncwarp();
    // A single CTA's copies need its own barriers only: they start here, while
    // the others set up Tensor Memory.
    if constexpr (!kPair) {
      int mt, nt;
      tile_at<C::kM>(first_tile, tiles_m, tiles_n, mt, nt);
      for (; kb_early < kb1 && x < C::kStages; ++kb_early) start_group(kb_early, mt, nt);
    }
  }
  if (warp == kMmaWarp) {
    if constexpr (kPair) {
      pw::tmem_alloc_pair(pw::smem_u32(&sh.tmem), 512);
    } else {
      pw::tmem_alloc(pw::smem_u32(&sh.tmem), 512);
      pw::tmem_relinquish();
    }
  }
  pw::tc_fence_before();
  __syncthreads();
  if constexpr (kPair) pw::cluster_sync();   // the other CTA's barriers are set up
  pw::tc_fence_after();
  const uint32_t tmem = pw::uniform(sh.tmem);

  if (warp == kCopyWarp) {
    if constexpr (C::kMove) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    bool ok = true;
    for (int tile = first_tile; ok && tile < tiles; tile += tile_step) {
      int mt, nt;
      tile_at<C::kM>(tile, tiles_m, tiles_n, mt, nt);
      for (int kb = tile == first_tile ? kb_early : kb0; kb < kb1; ++kb) {
        if (x >= C::kStages && !(ok = wait(sh.empty[stage.at], stage.parity ^ 1u, sh, p))) break;
        start_group(kb, mt, nt);
      }
    }
    // No copy may be in flight when the CTA leaves.  A pair's second CTA leaves
    // after the first (cluster barrier below), which sees both CTAs' copies.
    if (!ok && (!kPair || rank == 0))
      for (uint32_t i = x > C::kStages ? x - C::kStages : 0; i < x; ++i)
        pw::mbar_wait(pw::smem_u32(&sh.full[i % C::kStages]), (i / C::kStages) & 1u, kDrainNs);
    if (!ok)
      for (uint32_t i = fours > kScaleSlots ? fours - kScaleSlots : 0; i < fours; ++i)
        pw::mbar_wait(pw::smem_u32(&sh.scales[i % kScaleSlots]), (i / kScaleSlots) & 1u, kDrainNs);
  } else if (warp == kMmaWarp) {
    if constexpr (C::kMove) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (!kPair || rank == 0) {
      // (fewer tokens than the 128 lanes: the rows after them are those of the
      // weights, in lanes that nobody reads)
      constexpr uint32_t kIdesc = pw::idesc_f32(kPair ? 256 : 128, C::kN, false, false);
      pw::Ring<C::kStages> stage;
      pw::Ring<C::kAccs> acc;
      bool ok = true;
      for (int tile = first_tile; ok && tile < tiles; tile += tile_step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          // (an accumulator's first use waits for the phase before the first: passed)
          if (!(ok = pw::warp_wait2(&sh.full[stage.at], stage.parity, &sh.read[acc.at], acc.parity ^ 1u, &sh.dead,
                                    p.status)))
            break;
          pw::tc_fence_after();
          const uint32_t s = stage.at, buf = acc.at;
          const uint64_t a = pw::sdesc_kmajor_sw128(stages + s * C::kStageBytes);
          const uint64_t b = pw::sdesc_kmajor_sw128(stages + s * C::kStageBytes + C::kRowsA * kBoxBytes);
          if (pw::elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // 32 columns a step: 2 units of 16 bytes
              if constexpr (kPair)
                pw::tc_mma_f8_pair(tmem + buf * C::kN, a + 2 * i, b + 2 * i, kIdesc, i);
              else
                pw::tc_mma_f8(tmem + buf * C::kN, a + 2 * i, b + 2 * i, kIdesc, i);
            }
            if constexpr (kPair) {
              pw::tc_commit_pair(pw::smem_u32(&sh.empty[s]));
              pw::tc_commit_pair(pw::smem_u32(&sh.done[buf]));
            } else {
              pw::tc_commit(pw::smem_u32(&sh.empty[s]));
              pw::tc_commit(pw::smem_u32(&sh.done[buf]));
            }
          }
          stage.next();
          acc.next();
          __syncwarp();
        }
      }
      if (!ok) {   // the accumulators go back only when nothing writes them
        if (pw::elect_one()) {
          if constexpr (kPair)
            pw::tc_commit_pair(pw::smem_u32(&sh.drained));
          else
            pw::tc_commit(pw::smem_u32(&sh.drained));
        }
        __syncwarp();
        pw::mbar_wait(pw::smem_u32(&sh.drained), 0, kDrainNs);
      }
    }
  } else if (warp > kMmaWarp) {
    if constexpr (C::kMove) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");   // a warpgroup gives as a whole
  } else if ((warp & 3) >= C::kQuarters) {
    if constexpr (C::kMove) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");  // and takes as a whole
  } else {
    // sums; registers: 256 threads x 208 and 128 x 88 are the pair kernel's 384 x 168
    if constexpr (C::kMove) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int quarter = warp & 3, side = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t read0 = kPair ? pw::map_shared(pw::smem_u32(&sh.read[0]), 0) : pw::smem_u32(&sh.read[0]);
    unsigned char* out = smem + C::kStages * C::kStageBytes + warp * kOutBytes;
    pw::Ring<C::kAccs> acc;
    pw::Ring<kScaleSlots> slot;
    bool ok = true;
    uint32_t turn = 0, turn_parity = 0;   // of the exchange of largest magnitudes
    for (int tile = first_tile; ok && tile < tiles; tile += tile_step) {
      int mt, nt;
      tile_at<C::kM>(tile, tiles_m, tiles_n, mt, nt);
      const int m0 = mt * C::kM + (kPair ? 128 * rank : 0) + 32 * quarter, m = m0 + lane;
      const int n0 = nt * C::kOutN + C::kOutN / 2 * side;
      const float* sa = p.sa + static_cast<int64_t>(m < p.M ? m : 0) * p.sa_stride;
      const float* sb = p.sb + static_cast<int64_t>(min(n0, p.N - 1) / pw::kGroup) * p.sb_stride;
      const float* su = nullptr;
      if constexpr (kGated) su = p.su + static_cast<int64_t>(min(n0, p.N - 1) / pw::kGroup) * p.su_stride;
      uint64_t sum[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) sum[i] = 0;
      // Scales, four groups at a time, through shared memory where their layout
      // allows: a load from here would queue behind the ring's copies, 160 KB
      // of them, and hold up the sums for 450 cycles at every fourth group.
      const unsigned char* scales = smem + (scale_smem - stages);
      for (int kb = kb0; kb < kb1; ++kb) {
        const uint32_t buf = acc.at;
        float sc, sc_u = 0.0f;
        if (p.wide_scales) {
          if (kb == kb0 || (kb & 3) == 0) {
            if (!(ok = wait(sh.scales[slot.at], slot.parity, sh, p))) break;
            scales = smem + (scale_smem - stages) + slot.at * C::kSlotBytes;
            slot.next();
          }
          const float token = *reinterpret_cast<const float*>(scales + (32 * quarter + lane) * 16 + 4 * (kb & 3));
          sc = token * *reinterpret_cast<const float*>(scales + kTokenScaleBytes + (C::kN == 256 && !kGated ? 16 * side : 0) +
                                                       4 * (kb & 3));
          if constexpr (kGated) sc_u = token * *reinterpret_cast<const float*>(scales + kTokenScaleBytes + 128 + 4 * (kb & 3));
        } else {
          sc = __ldg(sa + kb) * __ldg(sb + kb);
          if constexpr (kGated) sc_u = __ldg(sa + kb) * __ldg(su + kb);
        }
        const uint64_t scale = pw::pack_f32x2(__float_as_uint(sc), __float_as_uint(sc));
        const uint64_t scale_u = kGated ? pw::pack_f32x2(__float_as_uint(sc_u), __float_as_uint(sc_u)) : 0;
        if (!(ok = wait(sh.done[buf], acc.parity, sh, p))) break;
        pw::tc_fence_after();
        const uint32_t src = tmem + lanes + buf * C::kN + C::kHalf * side;
        uint32_t v[2][16];
#pragma unroll
        for (int c = 0; c < C::kCols / 32; ++c) {
          const bool other = kGated && 32 * c >= C::kHalf;           // gated: kHalf columns of each weight
          const int col = other ? C::kOutN - C::kHalf + 32 * c : 32 * c;
          pw::tmem_ld_x16(src + col, v[0]);
          pw::tmem_ld_x16(src + col + 16, v[1]);
          pw::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sum[16 * c + i] = pw::fma_f32x2(pw::pack_f32x2(v[i / 8][2 * (i % 8)], v[i / 8][2 * (i % 8) + 1]),
                                            other ? scale_u : scale, sum[16 * c + i]);
        }
        pw::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            pw::mbar_arrive_cluster(read0 + 8 * buf);
          else
            pw::mbar_arrive(read0 + 8 * buf);
        }
        acc.next();
      }
      if (!ok) break;
      if (!kPair && p.splits > 1) {
        // rows of sums for the cluster; the copies' memory is free (every MMA
        // of the CTA has completed)
        float* part = reinterpret_cast<float*>(smem) + (32 * quarter + lane) * C::kPartRow + C::kHalf * side;
#pragma unroll
        for (int i = 0; i < C::kCols / 4; ++i) {
          float4 f;
          pw::unpack_f32x2(sum[2 * i], f.x, f.y);
          pw::unpack_f32x2(sum[2 * i + 1], f.z, f.w);
          *reinterpret_cast<float4*>(part + 4 * i + (4 * i >= C::kHalf ? C::kOutN - C::kHalf : 0)) = f;
        }
        break;   // one tile per cluster
      }
      if constexpr (kGated) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < C::kHalf / 2; ++i) {
          float h0, h1;
          sum[i] = gated2(sum[i], sum[C::kHalf / 2 + i], p.act);
          pw::unpack_f32x2(sum[i], h0, h1);
          top = pw::max3_nan(top, fabsf(h0), fabsf(h1));
        }
        if (C::kCodes && p.q) {
          gsh.top[turn][side][32 * quarter + lane] = top;
          __syncwarp();
          if (lane == 0) pw::mbar_arrive(pw::smem_u32(&gsh.met[quarter]));
          if (!(ok = wait(gsh.met[quarter], turn_parity, sh, p))) break;
          top = pw::max_nan(top, gsh.top[turn][side ^ 1][32 * quarter + lane]);
          turn ^= 1;
          turn_parity ^= 1;
          const float s = pw::max_nan(top / pw::kE4m3Max, pw::kMinScale);
          const pw::PairDivisor by{pw::Divisor(s)};
          if (m < p.M) {
            if (side == 0) p.scale[static_cast<int64_t>(m) * p.scale_stride + nt] = s;
            uint8_t* q = p.q + static_cast<int64_t>(m) * p.ldq + n0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = pw::e4m3_pairs(by(sum[8 * i + 2 * j]), by(sum[8 * i + 2 * j + 1]));
              if (p.wide_q && n0 + 16 * i + 16 <= p.N) {
                *reinterpret_cast<uint4*>(q + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (n0 + 16 * i + j < p.N) q[16 * i + j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
              }
            }
          }
        }
        if (!p.y) continue;
      }
      if constexpr (kRagged) {
        constexpr int kW = C::kHalf < 64 ? C::kHalf : 64;
#pragma unroll
        for (int box = 0; box < C::kHalf / kW; ++box) {
          const int n = n0 + kW * box;
          store_rows<T, kW>(sum + kW / 2 * box, static_cast<T*>(p.y) + static_cast<int64_t>(m0) * p.ldy + n, p.ldy, p.M - m0,
                            p.N - n, out);
        }
      } else if constexpr (kGated && !C::kCodes) {   // 32 columns a row: 64 bytes
        if (m < p.M) {
          T* y = static_cast<T*>(p.y) + static_cast<int64_t>(m) * p.ldy + n0;
#pragma unroll
          for (int i = 0; i < C::kHalf / 8; ++i) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) pw::unpack_f32x2(sum[4 * i + j], f[2 * j], f[2 * j + 1]);
            if (n0 + 8 * i + 8 <= p.N) {
              *reinterpret_cast<uint4*>(y + 8 * i) = make_uint4(pw::pack2<T>(f[0], f[1]), pw::pack2<T>(f[2], f[3]),
                                                                pw::pack2<T>(f[4], f[5]), pw::pack2<T>(f[6], f[7]));
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (n0 + 8 * i + j < p.N) y[8 * i + j] = pw::from_float<T>(f[j]);
            }
          }
        }
      } else {
        // 16-bit rows through shared memory, 32 rows x 64 columns at a time.  A
        // tiled store drops what lies past the matrix in whole units of 16 bytes
        // only: where N ends inside one, the last box goes value by value.
#pragma unroll
        for (int box = 0; box < C::kHalf / 64; ++box) {
          const int n = n0 + 64 * box;
          if (p.N % 8 == 0 || n + 64 <= p.N) {
            pw::bulk_wait_read();   // the box before has left
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float lo, hi;
                pw::unpack_f32x2(sum[32 * box + 4 * i + j], lo, hi);
                w[j] = pw::pack2<T>(lo, hi);
              }
              *reinterpret_cast<uint4*>(out + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            pw::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && m0 < p.M && n < p.N) {
              pw::tma_store_2d(&maps.y, n, m0, pw::smem_u32(out));
              pw::bulk_commit();
            }
          } else if (m < p.M) {
            T* y = static_cast<T*>(p.y) + static_cast<int64_t>(m) * p.ldy + n;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float lo, hi;
              pw::unpack_f32x2(sum[32 * box + i], lo, hi);
              if (n + 2 * i < p.N) y[2 * i] = pw::from_float<T>(lo);
              if (n + 2 * i + 1 < p.N) y[2 * i + 1] = pw::from_float<T>(hi);
            }
          }
        }
      }
    }
    if (lane == 0) pw::bulk_wait();
  }
  __syncwarp();
  pw::tc_fence_before();
  __syncthreads();
  if (group_size > 1) pw::cluster_sync();   // sums are in place; nobody still signals or feeds a CTA that leaves
  pw::tc_fence_after();
  if (warp == kMmaWarp) {
    if constexpr (kPair)
      pw::tmem_dealloc_pair(tmem, 512);
    else
      pw::tmem_dealloc(tmem, 512);
  }
  if constexpr (!kPair) {
    if (p.splits > 1) {
      // each CTA of the cluster finishes its share of the tile's rows
      int mt, nt;
      tile_at<C::kM>(first_tile, tiles_m, tiles_n, mt, nt);
      const int rows = min(C::kM, p.M - mt * C::kM), col = 4 * lane, n = nt * C::kOutN + col;
      auto sum_at = [&](uint32_t at) {   // all loads, then the sum in the order of the ranks
        float4 part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < p.splits) part[i] = pw::ld_cluster_f4(pw::map_shared(at, i));
        float4 v = part[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          if (i >= p.splits) break;
          v.x += part[i].x;
          v.y += part[i].y;
          v.z += part[i].z;
          v.w += part[i].w;
        }
        return v;
      };
      for (int row = rank + p.splits * warp; row < rows; row += p.splits * (C::kThreads / 32)) {
        if (col >= C::kOutN) continue;
        const uint32_t at = stages + 4u * static_cast<uint32_t>(row * C::kPartRow + col);
        float4 v = sum_at(at);
        if constexpr (kGated) {
          const float4 u = sum_at(at + 4 * C::kOutN);
          v = make_float4(gated(v.x, u.x, p.act), gated(v.y, u.y, p.act), gated(v.z, u.z, p.act), gated(v.w, u.w, p.act));
        }
        if (sh.dead) continue;
        if constexpr (kGated) {
          if (C::kCodes && p.q) {   // the warp has the 128 columns of a scale
            float top = pw::max_nan(pw::max_nan(fabsf(v.x), fabsf(v.y)), pw::max_nan(fabsf(v.z), fabsf(v.w)));
#pragma unroll
            for (int o = 16; o; o >>= 1) top = pw::max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            const float s = pw::max_nan(top / pw::kE4m3Max, pw::kMinScale);
            const pw::Divisor by(s);
            const int64_t m = mt * C::kM + row;
            if (lane == 0) p.scale[m * p.scale_stride + nt] = s;
            const uint32_t w = pw::e4m3x4(by(v.x), by(v.y), by(v.z), by(v.w));
            uint8_t* q = p.q + m * p.ldq + n;
            if (p.wide_q && n + 4 <= p.N) {
              *reinterpret_cast<uint32_t*>(q) = w;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n + i < p.N) q[i] = static_cast<uint8_t>(w >> (8 * i));
            }
          }
          if (!p.y) continue;
        }
        T* y = static_cast<T*>(p.y) + static_cast<int64_t>(mt * C::kM + row) * p.ldy + n;
        if (p.wide_y && n + 4 <= p.N) {
          *reinterpret_cast<uint2*>(y) = make_uint2(pw::pack2<T>(v.x, v.y), pw::pack2<T>(v.z, v.w));
        } else {
          const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < p.N) y[i] = pw::from_float<T>(f[i]);
        }
      }
      pw::cluster_sync();   // the sums have been read
    }
  }
}

// The kernel's shared memory, set once per device.
template <typename T, int kTokens, int kWide, bool kGated, bool kRagged>
int allow_smem(int dev) {
  constexpr int kDevs = 64;
  static bool done[kDevs] = {};
  if (dev < kDevs && done[dev]) return PW_OK;
  PW_CUDA_TRY(cudaFuncSetAttribute(linear_tile_kernel<T, kTokens, kWide, kGated, kRagged>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   Tile<kTokens, kWide, kGated>::kSmem));
  if (dev < kDevs) done[dev] = true;
  return PW_OK;
}

// How many clusters of n CTAs the device runs at once (asked once per device).
template <typename T, int kTokens, int kWide, bool kGated, bool kRagged>
int clusters_at_once(int dev, int n, int& fit) {
  using C = Tile<kTokens, kWide, kGated>;
  constexpr int kDevs = 64;
  static int known[kDevs][8] = {};
  if (dev < kDevs && known[dev][n]) {
    fit = known[dev][n] - 1;
    return PW_OK;
  }
  if (int e = allow_smem<T, kTokens, kWide, kGated, kRagged>(dev)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(n));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(n);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  PW_CUDA_TRY(cudaOccupancyMaxActiveClusters(&fit, linear_tile_kernel<T, kTokens, kWide, kGated, kRagged>, &cfg));
  if (dev < kDevs) known[dev][n] = fit + 1;
  return PW_OK;
}

// How many CTAs share the groups of each of `tiles` tiles of single CTAs.  Few
// tiles: 2 or 4, as long as all clusters run at once (4 do not fit everywhere).  A
// group less of the loop takes 0.28 us, a cluster and its addition 1.5 with 64 tokens
// and 3 with 128: 32 x 2048 x 4096 takes 13.0, 10.2 and 8.0 us with 1, 2 and 4, 32 x
// 2048 x 1024 5.7, 6.0 and 5.4, 100 x 4096 x 1024 6.1, 7.3 and 7.4.
template <typename T, int kTokens, int kWide, bool kGated, bool kRagged>
int splits_of(long long tiles, int groups, int& splits) {
  int dev = 0;
  PW_CUDA_TRY(cudaGetDevice(&dev));
  splits = 1;
  for (int n = 2; n <= 4; n *= 2) {
    int fit = 0;
    if (int e = clusters_at_once<T, kTokens, kWide, kGated, kRagged>(dev, n, fit)) return e;
    if (tiles <= fit && groups - groups / n >= (kTokens == 64 ? 6 : 12)) splits = n;
  }
  return PW_OK;
}

template <typename T, int kTokens, int kWide, bool kGated, bool kRagged>
int launch_tile_as(Params<kGated> p, int sms, cudaStream_t s) {
  using C = Tile<kTokens, kWide, kGated>;
  constexpr bool kPair = C::kPair;
  int dev = 0;
  PW_CUDA_TRY(cudaGetDevice(&dev));
  if (int e = allow_smem<T, kTokens, kWide, kGated, kRagged>(dev)) return e;
  Maps<kGated> maps;
  const uint64_t da[2] = {static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.M)};
  const uint64_t db[2] = {static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.N)};
  const uint64_t dy[2] = {static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.M)};
  const uint64_t sta[1] = {static_cast<uint64_t>(p.lda)}, stb[1] = {static_cast<uint64_t>(p.ldb)};
  const uint64_t sty[1] = {2 * static_cast<uint64_t>(p.ldy)};
  const uint32_t box[2] = {kBoxBytes, C::kRowsA}, boxw[2] = {kBoxBytes, static_cast<uint32_t>(kGated ? C::kOutN : C::kRowsB)}, boxy[2] = {64, 32};
  if (int e = pw::encode_tensor_map(&maps.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.a, da, sta, box)) return e;
  if (int e = pw::encode_tensor_map(&maps.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.b, db, stb, boxw)) return e;
  maps.y = maps.sa = maps.sb = maps.a;
  const uint64_t dsb[2] = {static_cast<uint64_t>(p.KB), static_cast<uint64_t>((p.N + pw::kGroup - 1) / pw::kGroup)};
  const uint32_t boxb[2] = {4, kGated ? 1u : C::kN / 128u};
  if (p.wide_scales) {
    const uint64_t dsa[2] = {static_cast<uint64_t>(p.KB), static_cast<uint64_t>(p.M)};
    const uint64_t stsa[1] = {4 * static_cast<uint64_t>(p.sa_stride)}, stsb[1] = {4 * static_cast<uint64_t>(p.sb_stride)};
    const uint32_t boxa[2] = {4, C::kRowsA};
    if (int e = pw::encode_tensor_map(&maps.sa, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.sa, dsa, stsa, boxa, false)) return e;
    if (int e = pw::encode_tensor_map(&maps.sb, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.sb, dsb, stsb, boxb, false)) return e;
  }
  if constexpr (kGated) {
    const uint64_t stu[1] = {static_cast<uint64_t>(p.ldu)}, stsu[1] = {4 * static_cast<uint64_t>(p.su_stride)};
    if (int e = pw::encode_tensor_map(&maps.u, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.u, db, stu, boxw)) return e;
    maps.su = maps.sb;
    if (p.wide_scales)
      if (int e = pw::encode_tensor_map(&maps.su, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.su, dsb, stsu, boxb, false)) return e;
  }
  if (p.wide_y)
    if (int e = pw::encode_tensor_map(&maps.y, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, p.y, dy, sty, boxy)) return e;
  const long long tiles = static_cast<long long>((p.M + C::kM - 1) / C::kM) * ((p.N + C::kOutN - 1) / C::kOutN);
  int cluster = 1;
  long long ctas;
  if (kPair) {
    cluster = 2;
    ctas = 2 * (tiles < sms / 2 ? tiles : sms / 2);
  } else {
    if (int e = splits_of<T, kTokens, kWide, kGated, kRagged>(tiles, p.KB, p.splits)) return e;
    cluster = p.splits;
    ctas = p.splits > 1 ? tiles * p.splits : (tiles < sms ? tiles : sms);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  PW_CUDA_TRY(cudaLaunchKernelEx(&cfg, linear_tile_kernel<T, kTokens, kWide, kGated, kRagged>, p, maps));
  return PW_OK;
}

template <typename T, int kTokens, int kWide, bool kGated>
int launch_tile(const Params<kGated>& p, int sms, cudaStream_t s) {
  return p.y && !p.wide_y ? launch_tile_as<T, kTokens, kWide, kGated, true>(p, sms, s)
                          : launch_tile_as<T, kTokens, kWide, kGated, false>(p, sms, s);
}

}  // namespace pw_fp8
