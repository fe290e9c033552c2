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
  int32_t* status;
  uint64_t wait_ns;
  bool wide_y;      // rows of y take 16-byte stores
};

constexpr int kRows = 16;    // weight rows of a CTA: the m16 side of the warp MMA
constexpr int kWarps = 8;

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

// Few tokens: the weights stream from memory into registers.  A CTA owns 16
// weight rows and 8 * kTiles tokens; its warps take every eighth group of 128
// columns.  A lane loads 16 contiguous bytes of a row and feeds them to two
// MMAs as if they were the four columns each of those wants: the same
// reordering of k on both operands leaves the sum as it is.
template <typename T, int kTiles>
__global__ void __launch_bounds__(32 * kWarps) linear_stream_kernel(const __grid_constant__ LinearParams p) {
  __shared__ float red[kWarps][kRows][8 * kTiles + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRows, m0 = blockIdx.y * 8 * kTiles;
  const uint8_t* b_lo = p.b + static_cast<int64_t>(n0 + g) * p.ldb;
  const uint8_t* b_hi = b_lo + 8 * p.ldb;
  const bool v_lo = n0 + g < p.N, v_hi = n0 + g + 8 < p.N;
  const float* sb = p.sb + (n0 / pw::kGroup) * p.sb_stride;
  float sum[kTiles][4] = {};
  for (int kb = warp; kb < p.KB; kb += kWarps) {
    const int k = kb * pw::kGroup + 16 * t;
    const uint4 w0 = load16(b_lo, k, p.K, v_lo), w1 = load16(b_hi, k, p.K, v_hi);
    const uint4 w2 = load16(b_lo, k + 64, p.K, v_lo), w3 = load16(b_hi, k + 64, p.K, v_hi);
    const float s = sb[kb];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      const int m = m0 + 8 * j + g;
      const uint8_t* a = p.a + static_cast<int64_t>(m) * p.lda;
      const uint4 x0 = load16(a, k, p.K, m < p.M), x1 = load16(a, k + 64, p.K, m < p.M);
      float acc[4] = {};
      pw::mma_16832_e4m3(acc, w0.x, w1.x, w0.y, w1.y, x0.x, x0.y);
      pw::mma_16832_e4m3(acc, w0.z, w1.z, w0.w, w1.w, x0.z, x0.w);
      pw::mma_16832_e4m3(acc, w2.x, w3.x, w2.y, w3.y, x1.x, x1.y);
      pw::mma_16832_e4m3(acc, w2.z, w3.z, w2.w, w3.w, x1.z, x1.w);
      const int c = m0 + 8 * j + 2 * t;   // the lane's two tokens of the result
      const float s0 = c < p.M ? s * p.sa[c * p.sa_stride + kb] : 0.0f;
      const float s1 = c + 1 < p.M ? s * p.sa[(c + 1) * p.sa_stride + kb] : 0.0f;
      sum[j][0] += s0 * acc[0];
      sum[j][1] += s1 * acc[1];
      sum[j][2] += s0 * acc[2];
      sum[j][3] += s1 * acc[3];
    }
  }
#pragma unroll
  for (int j = 0; j < kTiles; ++j) {
    red[warp][g][8 * j + 2 * t] = sum[j][0];
    red[warp][g][8 * j + 2 * t + 1] = sum[j][1];
    red[warp][g + 8][8 * j + 2 * t] = sum[j][2];
    red[warp][g + 8][8 * j + 2 * t + 1] = sum[j][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * 8 * kTiles; i += 32 * kWarps) {
    const int row = i % kRows, col = i / kRows;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][row][col];
    if (n0 + row < p.N && m0 + col < p.M)
      static_cast<T*>(p.y)[static_cast<int64_t>(m0 + col) * p.ldy + n0 + row] = pw::from_float<T>(v);
  }
}

template <typename T, int kTiles>
int launch_stream(const LinearParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.N + kRows - 1) / kRows),
                  static_cast<unsigned>((p.M + 8 * kTiles - 1) / (8 * kTiles)));
  linear_stream_kernel<T, kTiles><<<grid, 32 * kWarps, 0, s>>>(p);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

// ---------------------------------------------------------------------------
// Many tokens: 128 tokens x kN weight rows a tile on the tcgen05 tensor cores.
// The MMAs of one 128-column group write a fresh accumulator in Tensor Memory;
// eight warps (four for kN 128) read it, multiply by the group's scales and add
// to sums in registers, while the next group's MMAs fill the other
// accumulator.  A thread owns one token and 128 weight rows, that is one scale
// product per group.  Persistent: one CTA per SM walks the tiles.
// ---------------------------------------------------------------------------
constexpr int kTileM = 128;
constexpr int kTmaBoxBytes = 128;   // one group of columns: a swizzled row

template <int kN>
struct Tile {
  static constexpr int kStages = kN == 256 ? 4 : 6;
  static constexpr int kSumWarps = 4 * (kN / 128);
  static constexpr int kThreads = kN == 256 ? 384 : 192;   // whole warpgroups where registers are moved
  static constexpr int kStageBytes = (kTileM + kN) * kTmaBoxBytes;
  static constexpr int kSmem = kStages * kStageBytes + 1024;
};

template <int kN>
struct alignas(8) TileShared {
  uint64_t full[Tile<kN>::kStages], empty[Tile<kN>::kStages], done[2], read[2];
  uint32_t tmem;
  int dead;   // a wait ran out: everybody leaves
};

__device__ __forceinline__ bool wait(const uint64_t* bar, uint32_t parity, int* dead, const LinearParams& p) {
  return pw::warp_wait_or_dead(bar, parity, dead, p.status, p.wait_ns);
}

// Tiles in strips of 16 token tiles, so that the CTAs that run at the same
// time share both operands through L2.
__device__ __forceinline__ void tile_at(int tile, int tiles_m, int tiles_n, int& mt, int& nt) {
  const int per_strip = 16 * tiles_n, strip = tile / per_strip, r = tile - strip * per_strip;
  const int height = min(16, tiles_m - strip * 16);
  nt = r / height;
  mt = strip * 16 + r - nt * height;
}

// Wide tiles: registers move to the sums.  256 threads x 208 and 128 x 88 are
// the launch's 384 x 168.
template <int kN>
__device__ __forceinline__ void give_registers() {
  if constexpr (kN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
}

template <typename T, int kN>
__global__ void __launch_bounds__(Tile<kN>::kThreads, 1)
    linear_tile_kernel(const __grid_constant__ LinearParams p, const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b) {
  using C = Tile<kN>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ TileShared<kN> sh;
  const uint32_t stages = (pw::smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = pw::uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int tiles_m = (p.M + kTileM - 1) / kTileM, tiles_n = (p.N + kN - 1) / kN, tiles = tiles_m * tiles_n;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      pw::mbar_init(pw::smem_u32(&sh.full[i]), 1);
      pw::mbar_init(pw::smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      pw::mbar_init(pw::smem_u32(&sh.done[i]), 1);
      pw::mbar_init(pw::smem_u32(&sh.read[i]), C::kSumWarps);
    }
    sh.dead = 0;
    pw::mbar_init_fence();
  }
  if (warp == C::kSumWarps) {
    pw::tmem_alloc(pw::smem_u32(&sh.tmem), 2 * kN);
    pw::tmem_relinquish();
  }
  pw::tc_fence_before();
  __syncthreads();
  pw::tc_fence_after();
  const uint32_t tmem = pw::uniform(sh.tmem);

  if (warp == C::kSumWarps) {
    give_registers<kN>();
    // copies
    if (pw::elect_one()) {
      pw::prefetch_tmap(&map_a);
      pw::prefetch_tmap(&map_b);
    }
    uint32_t x = 0;   // groups started
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      int mt, nt;
      tile_at(tile, tiles_m, tiles_n, mt, nt);
      for (int kb = 0; kb < p.KB; ++kb, ++x) {
        const uint32_t s = x % C::kStages;
        if (x >= C::kStages && !(ok = wait(&sh.empty[s], (x / C::kStages + 1) & 1u, &sh.dead, p))) break;
        const uint32_t bar = pw::smem_u32(&sh.full[s]), dst = stages + s * C::kStageBytes;
        if (pw::elect_one()) {
          pw::mbar_arrive_expect_tx(bar, C::kStageBytes);
          pw::tma_load_2d(dst, &map_a, kb * pw::kGroup, mt * kTileM, bar);
          pw::tma_load_2d(dst + kTileM * kTmaBoxBytes, &map_b, kb * pw::kGroup, nt * kN, bar);
        }
        __syncwarp();
      }
    }
    // no copy may be in flight when the CTA leaves
    if (!ok)
      for (uint32_t i = x > C::kStages ? x - C::kStages : 0; i < x; ++i)
        pw::mbar_wait(pw::smem_u32(&sh.full[i % C::kStages]), (i / C::kStages) & 1u, p.wait_ns);
  } else if (warp == C::kSumWarps + 1) {
    give_registers<kN>();
    // matrix instructions
    constexpr uint32_t kIdesc = pw::idesc_f32(kTileM, kN, false, false);
    uint32_t x = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      for (int kb = 0; kb < p.KB; ++kb, ++x) {
        const uint32_t s = x % C::kStages, buf = x & 1u;
        if (x >= 2) ok = wait(&sh.read[buf], ((x >> 1) + 1) & 1u, &sh.dead, p);
        if (!ok || !(ok = wait(&sh.full[s], (x / C::kStages) & 1u, &sh.dead, p))) break;
        pw::tc_fence_after();
        const uint64_t a = pw::sdesc_kmajor_sw128(stages + s * C::kStageBytes);
        const uint64_t b = pw::sdesc_kmajor_sw128(stages + s * C::kStageBytes + kTileM * kTmaBoxBytes);
        if (pw::elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i)   // 32 columns a step: 2 units of 16 bytes
            pw::tc_mma_f8(tmem + buf * kN, a + 2 * i, b + 2 * i, kIdesc, i);
          pw::tc_commit(pw::smem_u32(&sh.empty[s]));
          pw::tc_commit(pw::smem_u32(&sh.done[buf]));
        }
        __syncwarp();
      }
    }
    if (!ok)   // the accumulators go back only when nothing writes them
      for (uint32_t i = x > 2 ? x - 2 : 0; i < x; ++i)
        pw::mbar_wait(pw::smem_u32(&sh.done[i & 1u]), (i >> 1) & 1u, p.wait_ns);
  } else if (warp > C::kSumWarps) {
    give_registers<kN>();   // a warpgroup gives and takes as a whole
  } else {   // sums
    if constexpr (kN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    uint32_t x = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      int mt, nt;
      tile_at(tile, tiles_m, tiles_n, mt, nt);
      const int m = mt * kTileM + 32 * quarter + lane, n0 = nt * kN + 128 * half;
      const bool live = m < p.M;
      const float* sa = p.sa + static_cast<int64_t>(live ? m : 0) * p.sa_stride;
      const float* sb = p.sb + static_cast<int64_t>(min(n0, p.N - 1) / pw::kGroup) * p.sb_stride;
      uint64_t sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      float next = __ldg(sa) * __ldg(sb);
      for (int kb = 0; kb < p.KB; ++kb, ++x) {
        const uint32_t buf = x & 1u;
        const float scale = next;
        if (kb + 1 < p.KB) next = __ldg(sa + kb + 1) * __ldg(sb + kb + 1);
        const uint64_t s2 = pw::pack_f32x2(__float_as_uint(scale), __float_as_uint(scale));
        if (!(ok = wait(&sh.done[buf], (x >> 1) & 1u, &sh.dead, p))) break;
        pw::tc_fence_after();
        const uint32_t src = tmem + lanes + buf * kN + 128u * half;
        uint32_t v[2][16];
        pw::tmem_ld_x16(src, v[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          pw::tmem_ld_wait();
          if (c < 7) pw::tmem_ld_x16(src + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            sum[8 * c + i] = pw::fma_f32x2(pw::pack_f32x2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), s2, sum[8 * c + i]);
        }
        pw::tc_fence_before();
        __syncwarp();
        if (lane == 0) pw::mbar_arrive(pw::smem_u32(&sh.read[buf]));
      }
      if (!ok || !live) continue;
      T* y = static_cast<T*>(p.y) + static_cast<int64_t>(m) * p.ldy + n0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) pw::unpack_f32x2(sum[4 * i + j], f[2 * j], f[2 * j + 1]);
        if (p.wide_y && n0 + 8 * i + 8 <= p.N) {
          *reinterpret_cast<uint4*>(y + 8 * i) = make_uint4(pw::pack2<T>(f[0], f[1]), pw::pack2<T>(f[2], f[3]),
                                                            pw::pack2<T>(f[4], f[5]), pw::pack2<T>(f[6], f[7]));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (n0 + 8 * i + j < p.N) y[8 * i + j] = pw::from_float<T>(f[j]);
        }
      }
    }
  }
  __syncwarp();
  pw::tc_fence_before();
  __syncthreads();
  pw::tc_fence_after();
  if (warp == C::kSumWarps) pw::tmem_dealloc(tmem, 2 * kN);
}

template <typename T, int kN>
int launch_tile(const LinearParams& p, cudaStream_t s) {
  using C = Tile<kN>;
  constexpr int kDevs = 64;
  static bool attr_done[kDevs] = {};
  int dev = 0;
  PW_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= kDevs || !attr_done[dev]) {
    PW_CUDA_TRY(cudaFuncSetAttribute(linear_tile_kernel<T, kN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
    if (dev < kDevs) attr_done[dev] = true;
  }
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  CUtensorMap ma, mb;
  const uint64_t da[2] = {static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.M)};
  const uint64_t db[2] = {static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.N)};
  const uint64_t sta[1] = {static_cast<uint64_t>(p.lda)}, stb[1] = {static_cast<uint64_t>(p.ldb)};
  const uint32_t ba[2] = {kTmaBoxBytes, kTileM}, bb[2] = {kTmaBoxBytes, kN};
  if (int e = pw::encode_tensor_map(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.a, da, sta, ba)) return e;
  if (int e = pw::encode_tensor_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.b, db, stb, bb)) return e;
  const long long tiles = static_cast<long long>((p.M + kTileM - 1) / kTileM) * ((p.N + kN - 1) / kN);
  linear_tile_kernel<T, kN><<<static_cast<unsigned>(tiles < sms ? tiles : sms), C::kThreads, C::kSmem, s>>>(p, ma, mb);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

template <typename T>
int launch(const LinearParams& p, cudaStream_t s) {
  if (p.M <= 8) return launch_stream<T, 1>(p, s);
  if (p.M <= 16) return launch_stream<T, 2>(p, s);
  if (p.M <= 64) return launch_stream<T, 4>(p, s);
  // wide tiles once they fill the SMs: half the weight reads per product
  const long long wide = static_cast<long long>((p.M + kTileM - 1) / kTileM) * ((p.N + 255) / 256);
  return wide >= pw::sm_count() ? launch_tile<T, 256>(p, s) : launch_tile<T, 128>(p, s);
}

}  // namespace

extern "C" int pw_fp8_linear(const uint8_t* d_a, int64_t lda, const float* d_a_scale, int64_t a_scale_stride,
                             const uint8_t* d_b, int64_t ldb, const float* d_b_scale, int64_t b_scale_stride, int M,
                             int N, int K, int dtype, void* d_y, int64_t ldy, int32_t* d_status, void* stream) {
  if (!pw::is_16bit(dtype)) return pw::set_error(PW_ERR_UNSUPPORTED, "fp8_linear: dtype %d", dtype);
  if (M < 0 || N < 1 || K < 1) return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: bad sizes M=%d N=%d K=%d", M, N, K);
  if (M > (1 << 20) || N > (1 << 24) || K > (1 << 24))
    return pw::set_error(PW_ERR_UNSUPPORTED, "fp8_linear: M=%d (at most 2^20), N=%d, K=%d (at most 2^24)", M, N, K);
  const int kb = (K + pw::kGroup - 1) / pw::kGroup;
  if (lda < K || ldb < K || ldy < N || a_scale_stride < kb || b_scale_stride < kb)
    return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: a row stride is below its columns");
  if (M == 0) return PW_OK;
  if (!d_a || !d_a_scale || !d_b || !d_b_scale || !d_y || !d_status)
    return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: NULL argument");
  if (!pw::aligned(d_a, 16) || !pw::aligned(d_b, 16) || lda % 16 || ldb % 16)
    return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: the rows of a and b must be 16-byte aligned");
  if (!pw::aligned(d_a_scale, 4) || !pw::aligned(d_b_scale, 4) || !pw::aligned(d_y, 2))
    return pw::set_error(PW_ERR_INVALID_ARG, "fp8_linear: a pointer is not aligned to its values");
  LinearParams p{};
  p.a = d_a;
  p.b = d_b;
  p.sa = d_a_scale;
  p.sb = d_b_scale;
  p.y = d_y;
  p.lda = lda;
  p.ldb = ldb;
  p.ldy = ldy;
  p.sa_stride = a_scale_stride;
  p.sb_stride = b_scale_stride;
  p.M = M;
  p.N = N;
  p.K = K;
  p.KB = kb;
  p.status = d_status;
  p.wait_ns = 2000000000ull;
  p.wide_y = pw::aligned(d_y, 16) && ldy % 8 == 0;
  cudaStream_t s = pw::as_stream(stream);
  return dtype == PW_DTYPE_F16 ? launch<__half>(p, s) : launch<__nv_bfloat16>(p, s);
}
