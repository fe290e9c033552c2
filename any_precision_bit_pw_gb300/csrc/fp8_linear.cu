// Product of two e4m3 matrices with a scale per row and 128 columns of the
// activations and per 128 x 128 block of the weights:
//
//   y[m][n] = sum_kb sa[m][kb] * sb[n / 128][kb] * sum_{k in kb} a[m][k] * b[n][k]
//
// The inner sum of a 128-column group runs on the tensor cores, the outer one
// in 32-bit registers.
#include "fp8_tile.cuh"

namespace {

using pw_fp8::launch_tile;
using pw_fp8::LinearParams;
using pw_fp8::load32;

constexpr int kRows = 16;    // weight rows of a CTA: the m16 side of the warp MMA

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
  if (p.M <= 64) return launch_tile<T, 64, 128, false>(p, sms, s);
  // Above, whichever needs less time in whole rounds over the SMs: a round of
  // pairs takes 1.5 times one of single CTAs (14.0 and 9.7 us at K = 4096) and
  // does twice the work.  1024 x 6144 x 4096: 32.0 and 34.1 us, 300 x 8192 x 6144:
  // 24.7 and 33.5; 509 x 4096 x 4096: 17.7 and 13.7.
  const long long pairs = static_cast<long long>((p.M + 255) / 256) * ((p.N + 255) / 256);
  const long long singles = static_cast<long long>((p.M + 127) / 128) * ((p.N + 127) / 128);
  const long long pair_rounds = (pairs + sms / 2 - 1) / (sms / 2), single_rounds = (singles + sms - 1) / sms;
  return 3 * pair_rounds <= 2 * single_rounds ? launch_tile<T, 256, 256, false>(p, sms, s) : launch_tile<T, 128, 128, false>(p, sms, s);
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
  // (8192 x 8192 x 6144 at the shape's own strides 281 us; with rows of scales at
  // 4-byte addresses 379; with rows of y at odd ones, 8191 columns, 324)
  p.wide_y = pw::aligned(a.y, 16) && a.ldy % 8 == 0;
  // with one group a tile the slots of the scales would be reused too early
  p.wide_scales = kb >= 2 && pw::aligned(a.a_scale, 16) && pw::aligned(a.b_scale, 16) && a.a_scale_stride % 4 == 0 &&
                  a.b_scale_stride % 4 == 0;
  cudaStream_t s = pw::as_stream(stream);
  return a.dtype == PW_DTYPE_F16 ? launch<__half>(p, s) : launch<__nv_bfloat16>(p, s);
}
