// Product of two e4m3 matrices with a scale per row and 128 columns of the
// activations and per 128 x 128 block of the weights:
//
//   y[m][n] = sum_kb sa[m][kb] * sb[n / 128][kb] * sum_{k in kb} a[m][k] * b[n][k]
//
// The inner sum of a 128-column group runs on the tensor cores, the outer one
// in 32-bit registers.
#include "ops_common.cuh"
#include "umma.cuh"

namespace {

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

constexpr int kRows = 16;    // weight rows of a CTA: the m16 side of the warp MMA

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

// Few tokens: the weights stream from memory into registers.  A CTA owns 16
// weight rows and kGroups x 8 tokens; its warps take every kWarps-th group of
// 128 columns.  A lane loads 32 contiguous bytes of a row and feeds them to four
// MMAs as if they were the columns that each of those wants: the same reordering
// of k on both operands leaves the sum as it is.  Memory bounds it, and what
// counts is that it sees whole 128-byte lines (halves of a line, in two loads of
// 16 bytes, take a tenth longer) and many warps with one group under way (two
// groups a warp at once, or L2 prefetches of the rows, scatter the accesses and
// take a tenth to a third longer).  8 x 6144 x 4096: 7.5 us, 3.4 TB/s of weights
// with the launch included; 2 x 28672 x 8192: 38 us, 6.2 TB/s.
template <typename T, int kGroups, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) linear_stream_kernel(const __grid_constant__ LinearParams p) {
  constexpr int kTokens = 8 * kGroups;
  __shared__ float red[kWarps][kRows][kTokens + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRows;
  const uint8_t* b_lo = p.b + static_cast<int64_t>(n0 + g) * p.ldb;
  const uint8_t* b_hi = b_lo + 8 * p.ldb;
  const bool v_lo = n0 + g < p.N, v_hi = n0 + g + 8 < p.N;
  const float* sb = p.sb + (n0 / pw::kGroup) * p.sb_stride;
  const uint8_t* a[kGroups];
  const float* sa[kGroups][2];   // of the lane's two tokens of the result
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int c = 8 * i + 2 * t;
    a[i] = p.a + static_cast<int64_t>(8 * i + g) * p.lda;
    sa[i][0] = p.sa + static_cast<int64_t>(c < p.M ? c : 0) * p.sa_stride;
    sa[i][1] = p.sa + static_cast<int64_t>(c + 1 < p.M ? c + 1 : 0) * p.sa_stride;
  }
  float sum[kGroups][4] = {};
  for (int kb = warp; kb < p.KB; kb += kWarps) {
    const int k = kb * pw::kGroup + 32 * t;
    uint32_t lo[8], hi[8];
    load32(b_lo, k, p.K, v_lo, p.wide_b, lo);
    load32(b_hi, k, p.K, v_hi, p.wide_b, hi);
    const float s = __ldg(sb + kb);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      uint32_t x[8];
      load32(a[i], k, p.K, 8 * i + g < p.M, false, x);
      const float s0 = s * __ldg(sa[i][0] + kb), s1 = s * __ldg(sa[i][1] + kb);
      float acc[4] = {};
#pragma unroll
      for (int j = 0; j < 8; j += 2) pw::mma_16832_e4m3(acc, lo[j], hi[j], lo[j + 1], hi[j + 1], x[j], x[j + 1]);
      sum[i][0] += s0 * acc[0];
      sum[i][1] += s1 * acc[1];
      sum[i][2] += s0 * acc[2];
      sum[i][3] += s1 * acc[3];
    }
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    red[warp][g][8 * i + 2 * t] = sum[i][0];
    red[warp][g][8 * i + 2 * t + 1] = sum[i][1];
    red[warp][g + 8][8 * i + 2 * t] = sum[i][2];
    red[warp][g + 8][8 * i + 2 * t + 1] = sum[i][3];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kRows * kTokens; e += 32 * kWarps) {
    const int row = e % kRows, col = e / kRows;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += red[i][row][col];
    if (n0 + row < p.N && col < p.M)
      static_cast<T*>(p.y)[static_cast<int64_t>(col) * p.ldy + n0 + row] = pw::from_float<T>(v);
  }
}

template <typename T, int kGroups, int kWarps>
int launch_stream(const LinearParams& p, cudaStream_t s) {
  linear_stream_kernel<T, kGroups, kWarps><<<static_cast<unsigned>((p.N + kRows - 1) / kRows), 32 * kWarps, 0, s>>>(p);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
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

template <int kTokens, int kWide>
struct Tile {
  static constexpr bool kPair = kTokens == 256;
  static constexpr int kM = kTokens;                  // tokens
  static constexpr int kN = kWide;                    // weight rows
  static constexpr int kRowsA = kPair ? 128 : kM;     // of both, in one CTA's shared memory
  static constexpr int kRowsB = kPair ? kN / 2 : kN;
  static constexpr int kCols = kN / 2;                // of one warpgroup's sums
  static constexpr int kQuarters = kRowsA / 32;       // warps of a warpgroup with tokens
  static constexpr int kStages = kRowsA == 128 ? 5 : 7;
  static constexpr int kAccs = 512 / kN;              // accumulators in Tensor Memory
  static constexpr bool kMove = kN == 256;            // registers move to the sums
  static constexpr int kThreads = kMove ? 384 : 320;  // whole warpgroups for that
  static constexpr int kStageBytes = (kRowsA + kRowsB) * kBoxBytes;
  static constexpr int kSmem = kStages * kStageBytes + kSumWarps * kOutBytes + kScaleSlots * kScaleBytes + 1024;
};
constexpr int kPartRow = 132;       // floats of a row of sums in shared memory: 16-byte lanes on distinct banks

struct alignas(8) TileShared {
  uint64_t full[7], empty[7], done[4], read[4], scales[kScaleSlots], drained;
  uint32_t tmem;
  int dead;   // a wait ran out: everybody leaves
};

__device__ __forceinline__ bool wait(const uint64_t& bar, uint32_t parity, TileShared& sh, const LinearParams& p) {
  return pw::warp_wait(&bar, parity, &sh.dead, p.status);
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

template <typename T, int kTokens, int kWide>
__global__ void __launch_bounds__(Tile<kTokens, kWide>::kThreads, 1)
    linear_tile_kernel(const __grid_constant__ LinearParams p, const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_y,
                       const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb) {
  using C = Tile<kTokens, kWide>;
  constexpr bool kPair = C::kPair;
  extern __shared__ unsigned char smem_raw[];
  __shared__ TileShared sh;
  unsigned char* smem = smem_raw + ((1024u - (pw::smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t stages = pw::smem_u32(smem);
  const int warp = pw::uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int tiles_m = (p.M + C::kM - 1) / C::kM, tiles_n = (p.N + C::kN - 1) / C::kN, tiles = tiles_m * tiles_n;
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
    const int row_a = mt * C::kM + (kPair ? 128 * rank : 0), row_b = nt * C::kN + (kPair ? C::kRowsB * rank : 0);
    const uint32_t bar = pw::smem_u32(&sh.full[stage.at]), dst = stages + stage.at * C::kStageBytes;
    if (p.wide_scales && (kb == kb0 || (kb & 3) == 0)) {
      // The slot is free: the MMAs of group x - kStages are done, they were
      // issued after every warp had read the accumulator of group x - kStages -
      // kAccs (at most 11 back), and the slot's last user is at least 14 back
      // (seven fours of a tile of two groups or more).
      const uint32_t sbar = pw::smem_u32(&sh.scales[slot.at]), sdst = scale_smem + slot.at * kScaleBytes;
      if (pw::elect_one()) {
        pw::mbar_arrive_expect_tx(sbar, 16 * (C::kRowsA + C::kN / 128));
        pw::tma_load_2d(sdst, &map_sa, kb & ~3, row_a, sbar);
        pw::tma_load_2d(sdst + kTokenScaleBytes, &map_sb, kb & ~3, nt * (C::kN / 128), sbar);
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
        pw::tma_load_2d_pair(dst, &map_a, kb * pw::kGroup, row_a, lead);
        pw::tma_load_2d_pair(dst + C::kRowsA * kBoxBytes, &map_b, kb * pw::kGroup, row_b, lead);
      } else {
        pw::mbar_arrive_expect_tx(bar, C::kStageBytes);
        pw::tma_load_2d(dst, &map_a, kb * pw::kGroup, row_a, bar);
        pw::tma_load_2d(dst + C::kRowsA * kBoxBytes, &map_b, kb * pw::kGroup, row_b, bar);
      }
    }
    stage.next();
    ++x;
    __syncwarp();
  };
  int kb_early = kb0;   // groups of the first tile that are under way before the set-up is done
  if (warp == kCopyWarp) {
    if (pw::elect_one()) {
      pw::prefetch_tmap(&map_a);
      pw::prefetch_tmap(&map_b);
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
  } else if (warp > kMmaWarp || (warp & 3) >= C::kQuarters) {
    if constexpr (C::kMove) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");   // a warpgroup gives as a whole
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
    for (int tile = first_tile; ok && tile < tiles; tile += tile_step) {
      int mt, nt;
      tile_at<C::kM>(tile, tiles_m, tiles_n, mt, nt);
      const int m0 = mt * C::kM + (kPair ? 128 * rank : 0) + 32 * quarter, m = m0 + lane;
      const int n0 = nt * C::kN + C::kCols * side;
      const float* sa = p.sa + static_cast<int64_t>(m < p.M ? m : 0) * p.sa_stride;
      const float* sb = p.sb + static_cast<int64_t>(min(n0, p.N - 1) / pw::kGroup) * p.sb_stride;
      uint64_t sum[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) sum[i] = 0;
      // Scales, four groups at a time, through shared memory where their layout
      // allows: a load from here would queue behind the ring's copies, 160 KB
      // of them, and hold up the sums for 450 cycles at every fourth group.
      const unsigned char* scales = smem + (scale_smem - stages);
      for (int kb = kb0; kb < kb1; ++kb) {
        const uint32_t buf = acc.at;
        float sc;
        if (p.wide_scales) {
          if (kb == kb0 || (kb & 3) == 0) {
            if (!(ok = wait(sh.scales[slot.at], slot.parity, sh, p))) break;
            scales = smem + (scale_smem - stages) + slot.at * kScaleBytes;
            slot.next();
          }
          sc = *reinterpret_cast<const float*>(scales + (32 * quarter + lane) * 16 + 4 * (kb & 3)) *
               *reinterpret_cast<const float*>(scales + kTokenScaleBytes + (C::kN == 256 ? 16 * side : 0) + 4 * (kb & 3));
        } else {
          sc = __ldg(sa + kb) * __ldg(sb + kb);
        }
        const uint64_t scale = pw::pack_f32x2(__float_as_uint(sc), __float_as_uint(sc));
        if (!(ok = wait(sh.done[buf], acc.parity, sh, p))) break;
        pw::tc_fence_after();
        const uint32_t src = tmem + lanes + buf * C::kN + C::kCols * side;
        uint32_t v[2][16];
#pragma unroll
        for (int c = 0; c < C::kCols / 32; ++c) {
          pw::tmem_ld_x16(src + 32 * c, v[0]);
          pw::tmem_ld_x16(src + 32 * c + 16, v[1]);
          pw::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sum[16 * c + i] = pw::fma_f32x2(pw::pack_f32x2(v[i / 8][2 * (i % 8)], v[i / 8][2 * (i % 8) + 1]), scale, sum[16 * c + i]);
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
        float* part = reinterpret_cast<float*>(smem) + (32 * quarter + lane) * kPartRow + C::kCols * side;
#pragma unroll
        for (int i = 0; i < C::kCols / 4; ++i) {
          float4 f;
          pw::unpack_f32x2(sum[2 * i], f.x, f.y);
          pw::unpack_f32x2(sum[2 * i + 1], f.z, f.w);
          *reinterpret_cast<float4*>(part + 4 * i) = f;
        }
        break;   // one tile per cluster
      }
      // 16-bit rows through shared memory, 32 rows x 64 columns at a time.  A
      // tiled store drops what lies past the matrix in whole units of 16 bytes
      // only: where N ends inside one, the last box goes value by value.
#pragma unroll
      for (int box = 0; box < C::kCols / 64; ++box) {
        const int n = n0 + 64 * box;
        if (p.wide_y && (p.N % 8 == 0 || n + 64 <= p.N)) {
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
            pw::tma_store_2d(&map_y, n, m0, pw::smem_u32(out));
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
      const int rows = min(C::kM, p.M - mt * C::kM), col = 4 * lane, n = nt * 128 + col;
      for (int row = rank + p.splits * warp; row < rows; row += p.splits * (C::kThreads / 32)) {
        const uint32_t at = stages + 4u * static_cast<uint32_t>(row * kPartRow + col);
        float4 part[4];   // all loads, then the sum in the order of the ranks
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
        if (sh.dead) continue;
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

// How many clusters of n CTAs the device runs at once (asked once per device).
template <typename T, int kTokens, int kWide>
int clusters_at_once(int dev, int n, int& fit) {
  using C = Tile<kTokens, kWide>;
  constexpr int kDevs = 64;
  static int known[kDevs][8] = {};
  if (dev < kDevs && known[dev][n]) {
    fit = known[dev][n] - 1;
    return PW_OK;
  }
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
  PW_CUDA_TRY(cudaOccupancyMaxActiveClusters(&fit, linear_tile_kernel<T, kTokens, kWide>, &cfg));
  if (dev < kDevs) known[dev][n] = fit + 1;
  return PW_OK;
}

template <typename T, int kTokens, int kWide>
int launch_tile(LinearParams p, int sms, cudaStream_t s) {
  using C = Tile<kTokens, kWide>;
  constexpr bool kPair = C::kPair;
  constexpr int kDevs = 64;
  static bool attr_done[kDevs] = {};
  int dev = 0;
  PW_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= kDevs || !attr_done[dev]) {
    PW_CUDA_TRY(cudaFuncSetAttribute(linear_tile_kernel<T, kTokens, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
    if (dev < kDevs) attr_done[dev] = true;
  }
  CUtensorMap ma, mb, my, msa, msb;
  const uint64_t da[2] = {static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.M)};
  const uint64_t db[2] = {static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.N)};
  const uint64_t dy[2] = {static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.M)};
  const uint64_t sta[1] = {static_cast<uint64_t>(p.lda)}, stb[1] = {static_cast<uint64_t>(p.ldb)};
  const uint64_t sty[1] = {2 * static_cast<uint64_t>(p.ldy)};
  const uint32_t box[2] = {kBoxBytes, C::kRowsA}, boxw[2] = {kBoxBytes, C::kRowsB}, boxy[2] = {64, 32};
  if (int e = pw::encode_tensor_map(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.a, da, sta, box)) return e;
  if (int e = pw::encode_tensor_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.b, db, stb, boxw)) return e;
  my = msa = msb = ma;
  if (p.wide_scales) {
    const uint64_t dsa[2] = {static_cast<uint64_t>(p.KB), static_cast<uint64_t>(p.M)};
    const uint64_t dsb[2] = {static_cast<uint64_t>(p.KB), static_cast<uint64_t>((p.N + pw::kGroup - 1) / pw::kGroup)};
    const uint64_t stsa[1] = {4 * static_cast<uint64_t>(p.sa_stride)}, stsb[1] = {4 * static_cast<uint64_t>(p.sb_stride)};
    const uint32_t boxa[2] = {4, C::kRowsA}, boxb[2] = {4, C::kN / 128};
    if (int e = pw::encode_tensor_map(&msa, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.sa, dsa, stsa, boxa, false)) return e;
    if (int e = pw::encode_tensor_map(&msb, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.sb, dsb, stsb, boxb, false)) return e;
  }
  if (p.wide_y)
    if (int e = pw::encode_tensor_map(&my, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, p.y, dy, sty, boxy)) return e;
  const long long tiles = static_cast<long long>((p.M + C::kM - 1) / C::kM) * ((p.N + C::kN - 1) / C::kN);
  int cluster = 1;
  long long ctas;
  if (kPair) {
    cluster = 2;
    ctas = 2 * (tiles < sms / 2 ? tiles : sms / 2);
  } else {
    // Few tiles: 2 or 4 CTAs share one's groups, as long as all clusters run at
    // once (4 do not fit everywhere).  A group less of the loop takes 0.28 us, a
    // cluster and its addition 1.5 with 64 tokens and 3 with 128: 32 x 2048 x
    // 4096 takes 13.0, 10.2 and 8.0 us with 1, 2 and 4, 32 x 2048 x 1024 5.7, 6.0
    // and 5.4, 100 x 4096 x 1024 6.1, 7.3 and 7.4.
    p.splits = 1;
    for (int n = 2; n <= 4; n *= 2) {
      int fit = 0;
      if (int e = clusters_at_once<T, kTokens, kWide>(dev, n, fit)) return e;
      if (tiles <= fit && p.KB - p.KB / n >= (kTokens == 64 ? 6 : 12)) p.splits = n;
    }
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
  PW_CUDA_TRY(cudaLaunchKernelEx(&cfg, linear_tile_kernel<T, kTokens, kWide>, p, ma, mb, my, msa, msb));
  return PW_OK;
}

template <typename T>
int launch(const LinearParams& p, cudaStream_t s) {
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  // Up to 8 tokens, the weights stream through the warps' registers (8 x 6144 x
  // 4096: 7.5 us, 10.4 by tiles); with 16 warps a CTA where all of them are on
  // the SMs at once (8 x 4096 x 4096: 5.7 us, 7.0 with 8 warps; 8 x 16384 x 4096,
  // in more than one wave: 15.1 and 14.7).
  const int ctas = (p.N + kRows - 1) / kRows;
  if (p.M <= 8) return ctas <= 2 * sms && p.KB > 8 ? launch_stream<T, 1, 16>(p, s) : launch_stream<T, 1, 8>(p, s);
  // Up to 32 they do where a warp has one or two groups of columns and the CTAs
  // are on the SMs at once: there the tiles' 4 us of set-up weigh more.  One CTA
  // of 16 warps an SM: 16 x 2048 x 4096 takes 6.0 us, 7.7 by tiles, 32 x 2048 x
  // 2048 4.5 (6.1), but 32 x 2048 x 4096 9.1 (8.0 by tiles).  Two or three of 8
  // warps: 16 x 4096 x 2048 5.0 us, 6.7 by tiles, 16 x 6144 x 2048 6.9 (8.5), 32 x
  // 4096 x 2048 7.0 (7.2), but 16 x 4096 x 4096 9.4 (9.0 by tiles).
  const bool few = p.M <= 16;
  if (p.M <= 32 && ctas <= sms && p.KB > 8 && p.KB <= (few ? 32 : 16))
    return few ? launch_stream<T, 2, 16>(p, s) : launch_stream<T, 4, 16>(p, s);
  if (p.M <= 32 && ctas <= (few ? 3 : 2) * sms && p.KB <= 16)
    return few ? launch_stream<T, 2, 8>(p, s) : launch_stream<T, 4, 8>(p, s);
  if (p.M <= 64) return launch_tile<T, 64, 128>(p, sms, s);
  // Above, whichever needs less time in whole rounds over the SMs: a round of
  // pairs takes 1.5 times one of single CTAs (14.0 and 9.7 us at K = 4096) and
  // does twice the work.  1024 x 6144 x 4096: 32.0 and 34.1 us, 300 x 8192 x 6144:
  // 24.7 and 33.5; 509 x 4096 x 4096: 17.7 and 13.7.
  const long long pairs = static_cast<long long>((p.M + 255) / 256) * ((p.N + 255) / 256);
  const long long singles = static_cast<long long>((p.M + 127) / 128) * ((p.N + 127) / 128);
  const long long pair_rounds = (pairs + sms / 2 - 1) / (sms / 2), single_rounds = (singles + sms - 1) / sms;
  return 3 * pair_rounds <= 2 * single_rounds ? launch_tile<T, 256, 256>(p, sms, s) : launch_tile<T, 128, 128>(p, sms, s);
}

}  // namespace

extern "C" int pw_fp8_linear(const pw_linear_args* args, void* stream) {
  if (!args) return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: NULL argument");
  const pw_linear_args& a = *args;
  if (!pw::is_16bit(a.dtype)) return pw::set_error(PW_ERR_UNSUPPORTED, "fp8_linear: dtype %d", a.dtype);
  if (a.m < 0 || a.n < 1 || a.k < 1)
    return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: bad sizes m=%d n=%d k=%d", a.m, a.n, a.k);
  if (a.m > (1 << 20) || a.n > (1 << 24) || a.k > (1 << 24))
    return pw::set_error(PW_ERR_UNSUPPORTED, "fp8_linear: m=%d (at most 2^20), n=%d, k=%d (at most 2^24)", a.m, a.n, a.k);
  const int kb = (a.k + pw::kGroup - 1) / pw::kGroup;
  if (a.lda < a.k || a.ldb < a.k || a.ldy < a.n || a.a_scale_stride < kb || a.b_scale_stride < kb)
    return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: a row stride is below its columns");
  if (a.m == 0) return PW_OK;
  if (!a.a || !a.a_scale || !a.b || !a.b_scale || !a.y || !a.status)
    return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: NULL argument");
  if (!pw::aligned(a.a, 16) || !pw::aligned(a.b, 16) || a.lda % 16 || a.ldb % 16)
    return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: the rows of a and b must be 16-byte aligned");
  // what a tensor map can hold
  if (a.lda >= (1ll << 39) || a.ldb >= (1ll << 39) || a.ldy >= (1ll << 38) || a.a_scale_stride >= (1ll << 37) ||
      a.b_scale_stride >= (1ll << 37))
    return pw::set_error(PW_ERR_UNSUPPORTED, "fp8_linear: a row stride is too large");
  if (!pw::aligned(a.a_scale, 4) || !pw::aligned(a.b_scale, 4) || !pw::aligned(a.y, 2) || !pw::aligned(a.status, 4))
    return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: a pointer is not aligned to its values");
  LinearParams p{};
  p.a = a.a;
  p.b = a.b;
  p.sa = a.a_scale;
  p.sb = a.b_scale;
  p.y = a.y;
  p.lda = a.lda;
  p.ldb = a.ldb;
  p.ldy = a.ldy;
  p.sa_stride = a.a_scale_stride;
  p.sb_stride = a.b_scale_stride;
  p.M = a.m;
  p.N = a.n;
  p.K = a.k;
  p.KB = kb;
  p.splits = 1;
  p.status = a.status;
  p.wide_b = pw::aligned(a.b, 32) && a.ldb % 32 == 0;
  // (8192 x 8192 x 6144 at the shape's own strides 281 us; with rows of y at odd
  // addresses 842, with rows of scales at 4-byte ones 379)
  p.wide_y = pw::aligned(a.y, 16) && a.ldy % 8 == 0;
  // with one group a tile the slots of the scales would be reused too early
  p.wide_scales = kb >= 2 && pw::aligned(a.a_scale, 16) && pw::aligned(a.b_scale, 16) && a.a_scale_stride % 4 == 0 &&
                  a.b_scale_stride % 4 == 0;
  cudaStream_t s = pw::as_stream(stream);
  return a.dtype == PW_DTYPE_F16 ? launch<__half>(p, s) : launch<__nv_bfloat16>(p, s);
}
