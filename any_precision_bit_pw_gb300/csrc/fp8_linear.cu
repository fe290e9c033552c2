// Product of two e4m3 matrices with a scale per row and 128 columns of the
// activations and per 128 x 128 block of the weights:
//
//   y[m][n] = sum_kb sa[m][kb] * sb[n / 128][kb] * sum_{k in kb} a[m][k] * b[n][k]
//
// The inner sum of a 128-column group runs on the tensor cores, the outer one
// in 32-bit registers.
#include "ops_common.cuh"

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

template <typename T>
int launch(const LinearParams& p, cudaStream_t s) {
  if (p.M <= 8) return launch_stream<T, 1>(p, s);
  if (p.M <= 16) return launch_stream<T, 2>(p, s);
  return launch_stream<T, 4>(p, s);
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
  cudaStream_t s = pw::as_stream(stream);
  return dtype == PW_DTYPE_F16 ? launch<__half>(p, s) : launch<__nv_bfloat16>(p, s);
}
