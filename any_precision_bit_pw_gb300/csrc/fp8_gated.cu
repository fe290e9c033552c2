// Gated feed-forward block up to its down projection, of e4m3 matrices with a
// scale per row and 128 columns of the activations and per 128 x 128 block of the
// weights:
//
//   g[m][n] = sum_k a[m][k] gate[n][k],   u[m][n] = sum_k a[m][k] up[n][k]
//   h[m][n] = act(g[m][n]) * u[m][n]
//
// in 16 bits, or in e4m3 with a scale per row and 128 columns: what the down
// projection reads.  Neither g nor u is stored.
//
// Few tokens: the weights' bytes bound it (7 x 14336 x 4096 in 8 bits 24 us, 4.8 TB/s; by
// a line through K of 2048 to 8192, 4.9 us and then 6.0 TB/s, with a 16-bit result, whose
// CTAs need no cluster, 5.4 us and 6.7 TB/s).
// Many: the accumulators, which are read and scaled once a group of 128, and the power
// limit (8192 x 16384 x 6144 in 8 bits 1257 to 1285 us, 2.6 PFLOP/s; cool, in 16 bits,
// 1160, the product of one weight as large as both 1077).  Between them, the rounds of the
// tiles over the SMs and their beginning and end (509 x 1408 x 2048 in 16 bits 9.4 us).
#include "fp8_tile.cuh"

namespace {

using pw_fp8::gated;
using pw_fp8::GatedParams;
using pw_fp8::launch_tile;
using pw_fp8::load32;

// Few tokens: the weights stream from memory into registers, as in the product of
// one weight.  A warp takes 8 columns of h and every kSplits-th group of 128 columns
// of K: one MMA tile is 8 rows of the gate's weight and the same 8 of the other's,
// so that a thread's results hold g and u of the same column.  A CTA has kWide such
// strips of 8 columns.  A scale of the 8-bit result belongs to 128 columns: a
// cluster of CTAs, which tell each other their largest magnitudes.
template <typename T, int kGroups, int kWide, int kSplits>
__global__ void __launch_bounds__(32 * kWide * kSplits) gated_stream_kernel(const __grid_constant__ GatedParams p) {
  constexpr int kTokens = 8 * kGroups, kCols = 8 * kWide, kThreads = 32 * kWide * kSplits;
  constexpr int kCluster = pw::kGroup / kCols;
  __shared__ float red[kSplits][2][kCols][kTokens + 1];   // of g and of u
  __shared__ float h[kTokens][kCols + 1];
  __shared__ float top[kTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int strip = warp % kWide, split = warp / kWide;
  const int n0 = blockIdx.x * kCols, n = n0 + 8 * strip + g;
  const bool valid = n < p.N;
  const uint8_t* gate = p.b + static_cast<int64_t>(n) * p.ldb;
  const uint8_t* up = p.u + static_cast<int64_t>(n) * p.ldu;
  const int block = min(n0, p.N - 1) / pw::kGroup;   // (a cluster's last CTAs may have no columns)
  const float* sg = p.sb + block * p.sb_stride;
  const float* su = p.su + block * p.su_stride;
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
  for (int kb = split; kb < p.KB; kb += kSplits) {
    const int k = kb * pw::kGroup + 32 * t;
    uint32_t wg[8], wu[8];
    load32(gate, k, p.K, valid, p.wide_b, wg);
    load32(up, k, p.K, valid, p.wide_b, wu);
    const float scale_g = __ldg(sg + kb), scale_u = __ldg(su + kb);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      uint32_t x[8];
      load32(a[i], k, p.K, 8 * i + g < p.M, false, x);
      const float s0 = __ldg(sa[i][0] + kb), s1 = __ldg(sa[i][1] + kb);
      float acc[4] = {};
#pragma unroll
      for (int e = 0; e < 8; e += 2) pw::mma_16832_e4m3(acc, wg[e], wu[e], wg[e + 1], wu[e + 1], x[e], x[e + 1]);
      sum[i][0] += scale_g * s0 * acc[0];
      sum[i][1] += scale_g * s1 * acc[1];
      sum[i][2] += scale_u * s0 * acc[2];
      sum[i][3] += scale_u * s1 * acc[3];
    }
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[split][j >> 1][8 * strip + g][8 * i + 2 * t + (j & 1)] = sum[i][j];
  __syncthreads();
  for (int e = threadIdx.x; e < kCols * kTokens; e += kThreads) {
    const int col = e % kCols, token = e / kCols;
    float vg = 0.0f, vu = 0.0f;
#pragma unroll
    for (int i = 0; i < kSplits; ++i) {
      vg += red[i][0][col][token];
      vu += red[i][1][col][token];
    }
    const float v = gated(vg, vu, p.act);   // 0 for columns past the end
    if (p.q) h[token][col] = v;
    if (p.y && n0 + col < p.N && token < p.M)
      static_cast<T*>(p.y)[static_cast<int64_t>(token) * p.ldy + n0 + col] = pw::from_float<T>(v);
  }
  if (!p.q) return;
  __syncthreads();
  for (int token = warp; token < kTokens; token += kWide * kSplits) {
    float most = 0.0f;
    for (int i = lane; i < kCols; i += 32) most = pw::max_nan(most, fabsf(h[token][i]));
#pragma unroll
    for (int o = 16; o; o >>= 1) most = pw::max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    if (lane == 0) top[token] = most;
  }
  pw::cluster_sync();
  const uint32_t rank = pw::cluster_rank();
  for (int token = warp; token < min(kTokens, p.M); token += kWide * kSplits) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < kCluster; ++i) most = pw::max_nan(most, pw::ld_cluster_f32(pw::map_shared(pw::smem_u32(&top[token]), i)));
    const float s = pw::max_nan(most / pw::kE4m3Max, pw::kMinScale);
    const pw::Divisor by(s);
    if (rank == 0 && lane == 0) p.scale[static_cast<int64_t>(token) * p.scale_stride + block] = s;
    for (int i = lane; i < kCols; i += 32)
      if (n0 + i < p.N) p.q[static_cast<int64_t>(token) * p.ldq + n0 + i] = static_cast<uint8_t>(pw::e4m3x2(by(h[token][i]), 0.0f));
  }
  pw::cluster_sync();   // nobody leaves while its magnitudes are read
}

template <typename T, int kGroups, int kWide, int kSplits>
int launch_stream(const GatedParams& p, cudaStream_t s) {
  constexpr unsigned kCols = 8 * kWide, kCluster = pw::kGroup / kCols;
  const unsigned ctas = (static_cast<unsigned>(p.N) + kCols - 1) / kCols;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.q ? (ctas + kCluster - 1) / kCluster * kCluster : ctas);
  cfg.blockDim = dim3(32 * kWide * kSplits);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.q ? 1 : 0;
  PW_CUDA_TRY(cudaLaunchKernelEx(&cfg, gated_stream_kernel<T, kGroups, kWide, kSplits>, p));
  return PW_OK;
}

template <typename T>
int launch(const GatedParams& p, cudaStream_t s) {
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  // Up to 8 tokens, the weights stream through the warps' registers.  Where all
  // CTAs of 16 columns and 8 splits of K are on the SMs at once (two an SM), they
  // have most loads under way (4096 x 4096: 10.7 us, 17.8 with 32 columns and two
  // splits, 11.9 by tiles); beyond, a cluster of 8 waits for 8 free places, and
  // clusters of 4 larger CTAs are faster (14336 x 4096: 23.9 us, 33.6; 24.3 by
  // tiles).  A 16-bit result needs no cluster (22.3 and 22.5 us).
  const int ctas = (p.N + 15) / 16;
  if (p.M <= 8) return ctas <= 2 * sms || !p.q ? launch_stream<T, 1, 2, 8>(p, s) : launch_stream<T, 1, 4, 2>(p, s);
  // Up to 16, and up to 32 for a 16-bit result, where one CTA an SM and one or two
  // groups of K a warp are all: 16 x 1408 x 2048 in 8 bits 5.7 us, 7.4 by tiles, in 16 bits 4.1
  // and 7.2; 32 tokens in 16 bits 5.5 and 7.7, in 8 bits 8.0 and 8.0; but 16 x
  // 4096 x 2048 18.8 and 9.7.
  if (ctas <= sms && p.KB <= 16) {
    if (p.M <= 16) return launch_stream<T, 2, 2, 8>(p, s);
    if (p.M <= 32 && !p.q) return launch_stream<T, 4, 2, 8>(p, s);
  }
  // Above, whichever tiles need least time, in groups of K (0.42 us each): those of
  // a CTA times the rounds over the SMs, and the addition of a cluster that shares a
  // tile's groups (4 with 64 tokens, 9 with 128).  In us by pairs of CTAs, 128 and 64 tokens:
  // 128 x 1408 x 2048 12.7, 10.4 and 9.1; 256 x 1408 x 4096 19.8, 13.4 and 15.0;
  // 300 x 2048 x 6144 26.1, 20.7 and 26.7; 1024 x 1408 x 2048 14.0, 13.6 and
  // 22.6; 128 x 14336 x 4096 37.3, 26.2 and 37.6.
  const long long wide = (p.N + 127) / 128, strips = (p.M + 127) / 128;
  auto groups = [&](long long tiles, int splits, double added) {
    return splits > 1 ? p.KB / splits + added : static_cast<double>((tiles + sms - 1) / sms) * p.KB;
  };
  int split = 1;
  if (int e = pw_fp8::splits_of<T, 64, 256, true, false>((p.M + 63) / 64 * wide, p.KB, split)) return e;
  const double by_64 = groups((p.M + 63) / 64 * wide, split, 4);
  if (int e = pw_fp8::splits_of<T, 128, 256, true, false>(strips * wide, p.KB, split)) return e;
  const double by_128 = p.M <= 64 ? INFINITY : groups(strips * wide, split, 9);
  const long long pairs = (p.M + 255) / 256 * wide;
  const double by_pairs = p.M <= 64 ? INFINITY : static_cast<double>((pairs + sms / 2 - 1) / (sms / 2)) * p.KB;
  const double least = fmin(fmin(by_64, by_128), by_pairs);
  // For 16-bit results also 128 tokens by 64 columns: three quarters of a group's
  // time for half of the work, but 4 groups less to begin and end with (509 x 1408 x
  // 2048 9.3 us, 12.3 by pairs; 64 x 1408 x 2048 7.8 and 8.7; but 1024 x 1408 x
  // 2048 15.5 and 12.9, 128 x 14336 x 4096 29.0 and 26.3).
  if (!p.q) {
    const long long tiles = strips * ((p.N + 63) / 64);
    if (int e = pw_fp8::splits_of<T, 128, 128, true, false>(tiles, p.KB, split)) return e;
    if (0.76 * groups(tiles, split, 7) - 4 < least) return launch_tile<T, 128, 128, true>(p, sms, s);
  }
  if (least == by_pairs) return launch_tile<T, 256, 256, true>(p, sms, s);
  return least == by_128 ? launch_tile<T, 128, 256, true>(p, sms, s) : launch_tile<T, 64, 256, true>(p, sms, s);
}

}  // namespace

extern "C" int pw_fp8_gated_linear(const pw_gated_args* args, void* stream) {
  const char* op = "fp8_gated_linear";
  if (!args) return pw::set_error(PW_ERR_INVALID_ARG, "%s: NULL argument", op);
  const pw_gated_args& a = *args;
  if (!pw::is_16bit(a.dtype)) return pw::set_error(PW_ERR_UNSUPPORTED, "%s: dtype %d", op, a.dtype);
  if (a.activation != PW_ACT_SILU && a.activation != PW_ACT_GELU_TANH)
    return pw::set_error(PW_ERR_UNSUPPORTED, "%s: activation %d", op, a.activation);
  if (a.m < 0 || a.n < 1 || a.k < 1)
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: bad sizes m=%d n=%d k=%d", op, a.m, a.n, a.k);
  if (a.m > (1 << 20) || a.n > (1 << 23) || a.k > (1 << 24))
    return pw::set_error(PW_ERR_UNSUPPORTED, "%s: m=%d (at most 2^20), n=%d (2^23), k=%d (2^24)", op, a.m, a.n, a.k);
  const int kb = (a.k + pw::kGroup - 1) / pw::kGroup, nb = (a.n + pw::kGroup - 1) / pw::kGroup;
  if (a.lda < a.k || a.ld_gate < a.k || a.ld_up < a.k || a.a_scale_stride < kb || a.gate_scale_stride < kb ||
      a.up_scale_stride < kb || (a.y && a.ldy < a.n) || (a.q && (a.ldq < a.n || a.scale_stride < nb)))
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: a row stride is below its columns", op);
  if (a.m == 0) return PW_OK;
  if (!a.a || !a.a_scale || !a.gate || !a.gate_scale || !a.up || !a.up_scale || !a.status)
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: NULL argument", op);
  if (!a.y && !a.q) return pw::set_error(PW_ERR_INVALID_ARG, "%s: neither a 16-bit nor an 8-bit output", op);
  if (!a.q != !a.scale) return pw::set_error(PW_ERR_INVALID_ARG, "%s: 8-bit codes and scales come together", op);
  if (!pw::aligned(a.a, 16) || !pw::aligned(a.gate, 16) || !pw::aligned(a.up, 16) || a.lda % 16 || a.ld_gate % 16 || a.ld_up % 16)
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: the rows of a, gate and up must be 16-byte aligned", op);
  // what a tensor map can hold
  for (int64_t bytes : {a.lda, a.ld_gate, a.ld_up, 2 * (a.y ? a.ldy : 0), 4 * a.a_scale_stride, 4 * a.gate_scale_stride,
                        4 * a.up_scale_stride})
    if (bytes < 0 || bytes >= (1ll << 39)) return pw::set_error(PW_ERR_UNSUPPORTED, "%s: a row stride is too large", op);
  if (!pw::aligned(a.a_scale, 4) || !pw::aligned(a.gate_scale, 4) || !pw::aligned(a.up_scale, 4) || !pw::aligned(a.scale, 4) ||
      !pw::aligned(a.y, 2) || !pw::aligned(a.status, 4))
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: a pointer is not aligned to its values", op);
  GatedParams p{};
  p.a = a.a;
  p.b = a.gate;
  p.u = a.up;
  p.sa = a.a_scale;
  p.sb = a.gate_scale;
  p.su = a.up_scale;
  p.y = a.y;
  p.q = a.q;
  p.scale = a.scale;
  p.lda = a.lda;
  p.ldb = a.ld_gate;
  p.ldu = a.ld_up;
  p.ldy = a.ldy;
  p.ldq = a.ldq;
  p.sa_stride = a.a_scale_stride;
  p.sb_stride = a.gate_scale_stride;
  p.su_stride = a.up_scale_stride;
  p.scale_stride = a.scale_stride;
  p.M = a.m;
  p.N = a.n;
  p.K = a.k;
  p.KB = kb;
  p.splits = 1;
  p.act = a.activation;
  p.status = a.status;
  p.wide_b = pw::aligned(a.gate, 32) && a.ld_gate % 32 == 0 && pw::aligned(a.up, 32) && a.ld_up % 32 == 0;
  p.wide_y = a.y && pw::aligned(a.y, 16) && a.ldy % 8 == 0;
  p.wide_q = pw::aligned(a.q, 16) && a.ldq % 16 == 0;
  // with one group a tile the slots of the scales would be reused too early
  p.wide_scales = kb >= 2 && pw::aligned(a.a_scale, 16) && pw::aligned(a.gate_scale, 16) && pw::aligned(a.up_scale, 16) &&
                  a.a_scale_stride % 4 == 0 && a.gate_scale_stride % 4 == 0 && a.up_scale_stride % 4 == 0;
  cudaStream_t s = pw::as_stream(stream);
  return a.dtype == PW_DTYPE_F16 ? launch<__half>(p, s) : launch<__nv_bfloat16>(p, s);
}
