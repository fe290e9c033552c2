// Residual addition with root-mean-square norm, and 16-bit to e4m3 conversion
// with a scale per 128 columns of a row or per 128 x 128 block.
//
//   r = x + residual,  y = r * rsqrt(mean(r^2) + eps) * w
//   s = max(max|y over the group| / 448, 2^-100),  q = e4m3(y / s)
//
// Both read and write every value once; memory bandwidth bounds them (8192 x
// 6144 with residual to e4m3: 55 us, 6.4 TB/s; weights of 8192 x 6144: 26 us,
// 5.9 TB/s), and for a few rows the latency of one load, one reduction and one
// store (one row of 4096: 2.0 us with the launch).
#include "ops_common.cuh"

namespace {

constexpr int kVec = 8;               // values a thread holds of one chunk: 16 bytes
constexpr int kMaxCols = 32768;       // 512 threads x 8 chunks

struct RowParams {
  const void* x;
  const void* res;
  const void* w;
  void* res_out;
  void* y;
  uint8_t* q;
  float* scale;
  int64_t x_stride, res_stride, res_out_stride, y_stride, q_stride, scale_stride;
  int64_t rows;
  int cols;
  float eps;
};

// Eight values at columns c .. c+7 of a row, packed; columns past the end are 0.
template <typename T, bool kAligned>
__device__ __forceinline__ uint4 load8(const T* row, int c, int cols) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (kAligned) {
    if (c < cols) u = *reinterpret_cast<const uint4*>(row + c);
  } else {
    const uint16_t* v = reinterpret_cast<const uint16_t*>(row) + c;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (c + 2 * i < cols ? v[2 * i] : 0u) | (c + 2 * i + 1 < cols ? static_cast<uint32_t>(v[2 * i + 1]) << 16 : 0u);
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return u;
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[kVec]) {
  pw::unpack2<T>(u.x, v[0], v[1]);
  pw::unpack2<T>(u.y, v[2], v[3]);
  pw::unpack2<T>(u.z, v[4], v[5]);
  pw::unpack2<T>(u.w, v[6], v[7]);
}
template <typename T, bool kAligned>
__device__ __forceinline__ void store8(T* row, int c, int cols, const float (&v)[kVec]) {
  if (kAligned) {
    if (c < cols)
      *reinterpret_cast<uint4*>(row + c) = make_uint4(pw::pack2<T>(v[0], v[1]), pw::pack2<T>(v[2], v[3]),
                                                      pw::pack2<T>(v[4], v[5]), pw::pack2<T>(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (c + i < cols) row[c + i] = pw::from_float<T>(v[i]);
  }
}
template <bool kAligned>
__device__ __forceinline__ void store8_e4m3(uint8_t* row, int c, int cols, const float (&v)[kVec], const pw::Divisor& by) {
  const uint32_t lo = pw::e4m3x4(by(v[0]), by(v[1]), by(v[2]), by(v[3]));
  const uint32_t hi = pw::e4m3x4(by(v[4]), by(v[5]), by(v[6]), by(v[7]));
  if (kAligned) {
    if (c < cols) *reinterpret_cast<uint2*>(row + c) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (c + i < cols) row[c + i] = static_cast<uint8_t>((i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) & 0xFFu);
  }
}

// A CTA takes every gridDim-th row.  A thread holds 8 values of each of kChunks
// chunks in registers, so a row is read once, and loads the next row before the
// reduction of this one, so that copies are always under way.  16 neighbouring
// threads hold a group of 128 columns: a group's largest value is four
// shuffles away.  (Conversion alone of 32 values a thread: two CTAs an SM, which
// takes 64 registers a thread; left to itself the compiler took 120, and 4096 x
// 9001 83 us instead of 45.)
template <typename T, int kChunks, bool kAligned, bool kNorm>
__global__ void __launch_bounds__(kChunks > 2 ? 512 : 1024, kChunks == 4 && !kNorm ? 2 : 1) row_kernel(const __grid_constant__ RowParams p) {
  __shared__ float sums[2][32];
  const int tid = threadIdx.x, nthr = blockDim.x;
  uint4 w[kChunks], x[kChunks], res[kChunks];
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int col = (c * nthr + tid) * kVec;
      x[c] = load8<T, kAligned>(static_cast<const T*>(p.x) + row * p.x_stride, col, p.cols);
      if (kNorm && p.res) res[c] = load8<T, kAligned>(static_cast<const T*>(p.res) + row * p.res_stride, col, p.cols);
    }
  };
  load_row(blockIdx.x);
  if (kNorm) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) w[c] = load8<T, kAligned>(static_cast<const T*>(p.w), (c * nthr + tid) * kVec, p.cols);
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    float v[kChunks][kVec];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      unpack8<T>(x[c], v[c]);
      if (kNorm && p.res) {
        float r[kVec];
        unpack8<T>(res[c], r);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[c][i] += r[i];
      }
    }
    if (row + gridDim.x < p.rows) load_row(row + gridDim.x);
    if (kNorm) {
      if (p.res_out) {
        T* res_out = static_cast<T*>(p.res_out) + row * p.res_out_stride;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) store8<T, kAligned>(res_out, (c * nthr + tid) * kVec, p.cols, v[c]);
      }
      // the sum of squares in 32 bits: 8 x kChunks terms a thread, then a tree
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < kVec; ++i) sum += v[c][i] * v[c][i];
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if ((tid & 31) == 0) sums[turn][tid >> 5] = sum;
      __syncthreads();   // the two buffers take turns: one barrier a row
      sum = (tid & 31) < (nthr >> 5) ? sums[turn][tid & 31] : 0.0f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      const float rs = rsqrtf(sum / static_cast<float>(p.cols) + p.eps);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        float wv[kVec];
        unpack8<T>(w[c], wv);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[c][i] = v[c][i] * rs * wv[i];
      }
      if (p.y) {
        T* y = static_cast<T*>(p.y) + row * p.y_stride;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) store8<T, kAligned>(y, (c * nthr + tid) * kVec, p.cols, v[c]);
      }
    }
    if (p.q) {
      uint8_t* q = p.q + row * p.q_stride;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int col = (c * nthr + tid) * kVec;
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) top = pw::max_nan(top, fabsf(v[c][i]));
#pragma unroll
        for (int o = 8; o; o >>= 1) top = pw::max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float s = pw::max_nan(top / pw::kE4m3Max, pw::kMinScale);
        if (col < p.cols && (tid & 15) == 0) p.scale[row * p.scale_stride + col / pw::kGroup] = s;
        store8_e4m3<kAligned>(q, col, p.cols, v[c], pw::Divisor(s));
      }
    }
  }
}

// One CTA per 128 x 128 block: 256 threads hold 64 values each, packed: of 8
// rows, or of 4 rows by accesses of 32 bytes (kWide), where they can be (8192 x
// 6144: 25.7 us, 27.0 by 16 bytes).
template <typename T, bool kAligned, bool kWide>
__global__ void __launch_bounds__(256) block_kernel(const __grid_constant__ RowParams p) {
  constexpr int kParts = kWide ? 2 : 1, kTurns = 8 / kParts, kLanes = 16 / kParts, kStep = 256 / kLanes;
  __shared__ float tops[8];
  const int tid = threadIdx.x;
  const int kb = blockIdx.x;
  const int col = kb * pw::kGroup + (tid % kLanes) * kParts * kVec;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * pw::kGroup + tid / kLanes;
  uint4 x[kTurns][kParts];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t row = row0 + kStep * i;
    const bool valid = row < p.rows && col < p.cols;
    const T* src = static_cast<const T*>(p.x) + (row < p.rows ? row : 0) * p.x_stride;
    if constexpr (kWide) {
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (valid)
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x[i][0].x), "=r"(x[i][0].y), "=r"(x[i][0].z), "=r"(x[i][0].w), "=r"(x[i][1].x), "=r"(x[i][1].y),
                       "=r"(x[i][1].z), "=r"(x[i][1].w)
                     : "l"(src + col));
    } else {
      x[i][0] = load8<T, kAligned>(src, valid ? col : p.cols, p.cols);
    }
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kTurns; ++i)
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
      float v[kVec];
      unpack8<T>(x[i][h], v);
#pragma unroll
      for (int j = 0; j < kVec; ++j) top = pw::max_nan(top, fabsf(v[j]));
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = pw::max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if ((tid & 31) == 0) tops[tid >> 5] = top;
  __syncthreads();
  top = tops[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) top = pw::max_nan(top, tops[i]);
  const float s = pw::max_nan(top / pw::kE4m3Max, pw::kMinScale);
  if (tid == 0) p.scale[blockIdx.y * p.scale_stride + kb] = s;
  const pw::Divisor by(s);
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t row = row0 + kStep * i;
    if (row >= p.rows) break;
    uint8_t* dst = p.q + row * p.q_stride;
    if constexpr (kWide) {
      uint32_t c[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[kVec];
        unpack8<T>(x[i][h], v);
        c[2 * h] = pw::e4m3x4(by(v[0]), by(v[1]), by(v[2]), by(v[3]));
        c[2 * h + 1] = pw::e4m3x4(by(v[4]), by(v[5]), by(v[6]), by(v[7]));
      }
      if (col < p.cols) *reinterpret_cast<uint4*>(dst + col) = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
      float v[kVec];
      unpack8<T>(x[i][0], v);
      store8_e4m3<kAligned>(dst, col, p.cols, v, by);
    }
  }
}

template <typename T, int kChunks, bool kAligned, bool kNorm>
int launch_chunks(const RowParams& p, int threads, int sms, cudaStream_t s) {
  // as many CTAs as run at once
  static int regs = 0;
  if (!regs) {
    cudaFuncAttributes at{};
    PW_CUDA_TRY(cudaFuncGetAttributes(&at, row_kernel<T, kChunks, kAligned, kNorm>));
    regs = (at.numRegs + 7) & ~7;
  }
  const int by_regs = 65536 / (regs * threads), by_threads = 2048 / threads;
  const int at_once = by_regs < by_threads ? (by_regs < 1 ? 1 : by_regs) : by_threads;
  const int64_t ctas = p.rows < static_cast<int64_t>(sms) * at_once ? p.rows : static_cast<int64_t>(sms) * at_once;
  row_kernel<T, kChunks, kAligned, kNorm><<<static_cast<unsigned>(ctas), threads, 0, s>>>(p);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

template <typename T, bool kAligned, bool kNorm>
int launch_rows(const RowParams& p, cudaStream_t s) {
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  // Few rows: one chunk a thread where 1024 threads suffice, for the shortest
  // way through a row.  Many: up to 512 threads, so that several CTAs an SM are
  // at different stages (8192 x 6144 with residual to e4m3: 55 us, 66 with 768
  // threads a row and 107 with 192).
  const int units = (p.cols + kVec - 1) / kVec, most = p.rows <= sms ? 1024 : 512;
  int chunks = 1;
  while ((units + chunks - 1) / chunks > (chunks > 2 ? 512 : most)) chunks *= 2;
  const int threads = ((units + chunks - 1) / chunks + 31) & ~31;
  switch (chunks) {
    case 1: return launch_chunks<T, 1, kAligned, kNorm>(p, threads, sms, s);
    case 2: return launch_chunks<T, 2, kAligned, kNorm>(p, threads, sms, s);
    case 4: return launch_chunks<T, 4, kAligned, kNorm>(p, threads, sms, s);
    default: return launch_chunks<T, 8, kAligned, kNorm>(p, threads, sms, s);
  }
}

template <typename T, bool kAligned>
int launch_blocks(const RowParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.cols + pw::kGroup - 1) / pw::kGroup),
                  static_cast<unsigned>((p.rows + pw::kGroup - 1) / pw::kGroup));
  if constexpr (kAligned) {
    if (pw::aligned(p.x, 32) && pw::aligned(p.q, 16) && p.x_stride % 16 == 0 && p.q_stride % 16 == 0 && p.cols % 16 == 0) {
      block_kernel<T, true, true><<<grid, 256, 0, s>>>(p);
      PW_CUDA_TRY(cudaGetLastError());
      return PW_OK;
    }
  }
  block_kernel<T, kAligned, false><<<grid, 256, 0, s>>>(p);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

// 16-byte accesses of 16-bit rows need the address, the stride and the width
// in multiples of 8 values.  Otherwise a thread's 8 values are accesses of 2
// bytes (8192 x 6143: norm to e4m3 256 us, rows to e4m3 53 us, blocks 100 us, where
// 6144 columns take 55, 29 and 26).
bool rows_aligned(const void* ptr, int64_t stride, int cols) {
  return !ptr || (pw::aligned(ptr, 16) && stride % kVec == 0 && cols % kVec == 0);
}
bool codes_aligned(const void* ptr, int64_t stride) { return !ptr || (pw::aligned(ptr, 8) && stride % 8 == 0); }

int check_matrix(const char* op, const char* name, int64_t stride, int cols) {
  if (stride < cols)
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: row stride %lld of %s is below the %d columns", op,
                         static_cast<long long>(stride), name, cols);
  return PW_OK;
}

}  // namespace

extern "C" {

int pw_add_rmsnorm(const pw_norm_args* args, void* stream) {
  if (!args) return pw::set_error(PW_ERR_INVALID_ARG, "add_rmsnorm: NULL argument");
  const pw_norm_args& a = *args;
  if (!pw::is_16bit(a.dtype)) return pw::set_error(PW_ERR_UNSUPPORTED, "add_rmsnorm: dtype %d", a.dtype);
  if (a.rows < 0 || a.cols < 1)
    return pw::set_error(PW_ERR_INVALID_ARG, "add_rmsnorm: %lld rows of %d columns", static_cast<long long>(a.rows), a.cols);
  if (a.cols > kMaxCols || a.rows > 0x7FFFFFFF)
    return pw::set_error(PW_ERR_UNSUPPORTED, "add_rmsnorm: at most %d columns (got %d) and 2^31 - 1 rows", kMaxCols, a.cols);
  if (!(a.eps >= 0.0f)) return pw::set_error(PW_ERR_INVALID_ARG, "add_rmsnorm: eps %g", static_cast<double>(a.eps));
  if (!a.y && !a.q) return pw::set_error(PW_ERR_INVALID_ARG, "add_rmsnorm: neither a 16-bit nor an 8-bit output");
  if (!a.q != !a.scale) return pw::set_error(PW_ERR_INVALID_ARG, "add_rmsnorm: 8-bit codes and scales come together");
  if (int e = check_matrix("add_rmsnorm", "x", a.x_stride, a.cols)) return e;
  if (a.residual)
    if (int e = check_matrix("add_rmsnorm", "residual", a.residual_stride, a.cols)) return e;
  if (a.residual_out)
    if (int e = check_matrix("add_rmsnorm", "residual_out", a.residual_out_stride, a.cols)) return e;
  if (a.y)
    if (int e = check_matrix("add_rmsnorm", "y", a.y_stride, a.cols)) return e;
  if (a.q) {
    if (int e = check_matrix("add_rmsnorm", "q", a.q_stride, a.cols)) return e;
    if (int e = check_matrix("add_rmsnorm", "scale", a.scale_stride, (a.cols + pw::kGroup - 1) / pw::kGroup)) return e;
  }
  if (a.rows == 0) return PW_OK;
  if (!a.x || !a.weight) return pw::set_error(PW_ERR_INVALID_ARG, "add_rmsnorm: NULL argument");
  if (!pw::aligned(a.x, 2) || !pw::aligned(a.weight, 2) || !pw::aligned(a.residual, 2) ||
      !pw::aligned(a.residual_out, 2) || !pw::aligned(a.y, 2) || !pw::aligned(a.scale, 4))
    return pw::set_error(PW_ERR_INVALID_ARG, "add_rmsnorm: a pointer is not aligned to its values");
  RowParams p{};
  p.x = a.x;
  p.res = a.residual;
  p.w = a.weight;
  p.res_out = a.residual_out;
  p.y = a.y;
  p.q = a.q;
  p.scale = a.scale;
  p.x_stride = a.x_stride;
  p.res_stride = a.residual_stride;
  p.res_out_stride = a.residual_out_stride;
  p.y_stride = a.y_stride;
  p.q_stride = a.q_stride;
  p.scale_stride = a.scale_stride;
  p.rows = a.rows;
  p.cols = a.cols;
  p.eps = a.eps;
  const bool al = rows_aligned(a.x, a.x_stride, a.cols) && rows_aligned(a.residual, a.residual_stride, a.cols) &&
                  rows_aligned(a.weight, kVec, a.cols) && rows_aligned(a.residual_out, a.residual_out_stride, a.cols) &&
                  rows_aligned(a.y, a.y_stride, a.cols) && codes_aligned(a.q, a.q_stride);
  cudaStream_t s = pw::as_stream(stream);
  if (a.dtype == PW_DTYPE_F16) return al ? launch_rows<__half, true, true>(p, s) : launch_rows<__half, false, true>(p, s);
  return al ? launch_rows<__nv_bfloat16, true, true>(p, s) : launch_rows<__nv_bfloat16, false, true>(p, s);
}

int pw_quantize_fp8(const pw_quant_args* args, void* stream) {
  if (!args) return pw::set_error(PW_ERR_INVALID_ARG, "quantize_fp8: NULL argument");
  const pw_quant_args& a = *args;
  if (!pw::is_16bit(a.dtype)) return pw::set_error(PW_ERR_UNSUPPORTED, "quantize_fp8: dtype %d", a.dtype);
  if (a.block_rows != 1 && a.block_rows != pw::kGroup)
    return pw::set_error(PW_ERR_UNSUPPORTED, "quantize_fp8: block_rows %d (1 or 128)", a.block_rows);
  if (a.rows < 0 || a.cols < 1)
    return pw::set_error(PW_ERR_INVALID_ARG, "quantize_fp8: %lld rows of %d columns", static_cast<long long>(a.rows), a.cols);
  // blocks: the grid's second axis counts 128-row strips
  if (a.block_rows == 1 ? (a.cols > kMaxCols || a.rows > 0x7FFFFFFF)
                        : (a.rows > 65535ll * pw::kGroup || a.cols > 0x7FFFFFFF - pw::kGroup))
    return pw::set_error(PW_ERR_UNSUPPORTED, "quantize_fp8: %lld rows of %d columns are too large",
                         static_cast<long long>(a.rows), a.cols);
  if (int e = check_matrix("quantize_fp8", "x", a.x_stride, a.cols)) return e;
  if (int e = check_matrix("quantize_fp8", "q", a.q_stride, a.cols)) return e;
  if (int e = check_matrix("quantize_fp8", "scale", a.scale_stride, (a.cols + pw::kGroup - 1) / pw::kGroup)) return e;
  if (a.rows == 0) return PW_OK;
  if (!a.x || !a.q || !a.scale) return pw::set_error(PW_ERR_INVALID_ARG, "quantize_fp8: NULL argument");
  if (!pw::aligned(a.x, 2) || !pw::aligned(a.scale, 4))
    return pw::set_error(PW_ERR_INVALID_ARG, "quantize_fp8: a pointer is not aligned to its values");
  RowParams p{};
  p.x = a.x;
  p.q = a.q;
  p.scale = a.scale;
  p.x_stride = a.x_stride;
  p.q_stride = a.q_stride;
  p.scale_stride = a.scale_stride;
  p.rows = a.rows;
  p.cols = a.cols;
  const bool al = rows_aligned(a.x, a.x_stride, a.cols) && codes_aligned(a.q, a.q_stride);
  cudaStream_t s = pw::as_stream(stream);
  if (a.block_rows == 1) {
    if (a.dtype == PW_DTYPE_F16)
      return al ? launch_rows<__half, true, false>(p, s) : launch_rows<__half, false, false>(p, s);
    return al ? launch_rows<__nv_bfloat16, true, false>(p, s) : launch_rows<__nv_bfloat16, false, false>(p, s);
  }
  if (a.dtype == PW_DTYPE_F16) return al ? launch_blocks<__half, true>(p, s) : launch_blocks<__half, false>(p, s);
  return al ? launch_blocks<__nv_bfloat16, true>(p, s) : launch_blocks<__nv_bfloat16, false>(p, s);
}

}  // extern "C"
