// Gated feed-forward block up to its down projection, of e4m3 matrices with a
// scale per row and 128 columns of the activations and per 128 x 128 block of the
// weights:
//
//   g[m][n] = sum_k a[m][k] gate[n][k],   u[m][n] = sum_k a[m][k] up[n][k]
//   h[m][n] = act(g[m][n]) * u[m][n]
//
// in 16 bits, or in e4m3 with a scale per row and 128 columns: what the down
// projection reads.  Neither g nor u is stored.
#include "fp8_tile.cuh"

namespace {

using pw_fp8::gated;
using pw_fp8::GatedParams;
using pw_fp8::launch_tile;
using pw_fp8::load32;

// Few tokens: the weights stream from memory into registers, as in the product of
// one weight.  A CTA owns 16 columns of h: two MMA tiles of 8 rows of the gate's
// weight and the same 8 of the other's, so that a thread's results hold g and u of
// the same column.  A scale of the 8-bit result belongs to 128 columns: a cluster of
// 8 CTAs, which tell each other their largest magnitudes.
constexpr int kCols = 16, kSets = 2, kCluster = 8;

template <typename T, int kGroups, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) gated_stream_kernel(const __grid_constant__ GatedParams p) {
  constexpr int kTokens = 8 * kGroups;
  __shared__ float red[kWarps][kSets][16][kTokens + 1];
  __shared__ float h[kTokens][kCols];
  __shared__ float top[kTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kCols;
  const uint8_t* gate[kSets];
  const uint8_t* up[kSets];
  bool valid[kSets];
#pragma unroll
  for (int j = 0; j < kSets; ++j) {
    valid[j] = n0 + 8 * j + g < p.N;
    gate[j] = p.b + static_cast<int64_t>(n0 + 8 * j + g) * p.ldb;
    up[j] = p.u + static_cast<int64_t>(n0 + 8 * j + g) * p.ldu;
  }
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
  float sum[kSets][kGroups][4] = {};
  for (int kb = warp; kb < p.KB; kb += kWarps) {
    const int k = kb * pw::kGroup + 32 * t;
    uint32_t wg[kSets][8], wu[kSets][8];
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      load32(gate[j], k, p.K, valid[j], p.wide_b, wg[j]);
      load32(up[j], k, p.K, valid[j], p.wide_b, wu[j]);
    }
    const float scale_g = __ldg(sg + kb), scale_u = __ldg(su + kb);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      uint32_t x[8];
      load32(a[i], k, p.K, 8 * i + g < p.M, false, x);
      const float s0 = __ldg(sa[i][0] + kb), s1 = __ldg(sa[i][1] + kb);
#pragma unroll
      for (int j = 0; j < kSets; ++j) {
        float acc[4] = {};
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          pw::mma_16832_e4m3(acc, wg[j][e], wu[j][e], wg[j][e + 1], wu[j][e + 1], x[e], x[e + 1]);
        sum[j][i][0] += scale_g * s0 * acc[0];
        sum[j][i][1] += scale_g * s1 * acc[1];
        sum[j][i][2] += scale_u * s0 * acc[2];
        sum[j][i][3] += scale_u * s1 * acc[3];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kSets; ++j)
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      red[warp][j][g][8 * i + 2 * t] = sum[j][i][0];
      red[warp][j][g][8 * i + 2 * t + 1] = sum[j][i][1];
      red[warp][j][g + 8][8 * i + 2 * t] = sum[j][i][2];
      red[warp][j][g + 8][8 * i + 2 * t + 1] = sum[j][i][3];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < kCols * kTokens; e += 32 * kWarps) {
    const int col = e % kCols, token = e / kCols;
    float vg = 0.0f, vu = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      vg += red[i][col >> 3][col & 7][token];
      vu += red[i][col >> 3][8 + (col & 7)][token];
    }
    const float v = gated(vg, vu, p.act);   // 0 for columns past the end
    if (p.q) h[token][col] = v;
    if (p.y && n0 + col < p.N && token < p.M)
      static_cast<T*>(p.y)[static_cast<int64_t>(token) * p.ldy + n0 + col] = pw::from_float<T>(v);
  }
  if (!p.q) return;
  __syncthreads();
  if (threadIdx.x < kTokens) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) most = pw::max_nan(most, fabsf(h[threadIdx.x][i]));
    top[threadIdx.x] = most;
  }
  pw::cluster_sync();
  const uint32_t rank = pw::cluster_rank();
  for (int token = warp; token < min(kTokens, p.M); token += kWarps) {
    float most = pw::ld_cluster_f32(pw::map_shared(pw::smem_u32(&top[token]), lane % kCluster));
#pragma unroll
    for (int o = kCluster / 2; o; o >>= 1) most = pw::max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    const float s = pw::max_nan(most / pw::kE4m3Max, pw::kMinScale);
    if (rank == 0 && lane == 0) p.scale[static_cast<int64_t>(token) * p.scale_stride + block] = s;
    if (lane < kCols && n0 + lane < p.N)
      p.q[static_cast<int64_t>(token) * p.ldq + n0 + lane] = static_cast<uint8_t>(pw::e4m3x2(pw::Divisor(s)(h[token][lane]), 0.0f));
  }
  pw::cluster_sync();   // nobody leaves while its magnitudes are read
}

template <typename T, int kGroups, int kWarps>
int launch_stream(const GatedParams& p, cudaStream_t s) {
  const unsigned ctas = static_cast<unsigned>((p.N + kCols - 1) / kCols);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.q ? (ctas + kCluster - 1) / kCluster * kCluster : ctas);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.q ? 1 : 0;
  PW_CUDA_TRY(cudaLaunchKernelEx(&cfg, gated_stream_kernel<T, kGroups, kWarps>, p));
  return PW_OK;
}

template <typename T>
int launch(const GatedParams& p, cudaStream_t s) {
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  if (p.M <= 8) return launch_stream<T, 1, 8>(p, s);
  if (p.M <= 64) return launch_tile<T, 64, 256, true>(p, sms, s);
  const long long wide = (p.N + 127) / 128;
  const long long pairs = (p.M + 255) / 256 * wide, singles = (p.M + 127) / 128 * wide;
  const long long pair_rounds = (pairs + sms / 2 - 1) / (sms / 2), single_rounds = (singles + sms - 1) / sms;
  return pair_rounds <= single_rounds ? launch_tile<T, 256, 256, true>(p, sms, s) : launch_tile<T, 128, 256, true>(p, sms, s);
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
