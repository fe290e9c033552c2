// The norms on both sides of a block, with what is between them:
//
//   u = x * rsqrt(mean(x^2) + eps) * post_weight      (x: the block's output)
//   r = residual_scale * residual + block_scale * gate * u
//   y = r * rsqrt(mean(r^2) + eps) * weight           (in 16 bits and/or in e4m3)
//
// Every value is read and written once: memory bandwidth bounds it, and for a
// few rows the latency of one load, two reductions and one store.
#include "rows.cuh"

namespace {

using pw::kVec;

constexpr int kMaxCols = 32768;       // 512 threads x 8 chunks

struct NormsParams {
  const void* x;
  const void* res;
  const void* post;
  const void* gate;
  const void* w;
  void* res_out;
  void* y;
  uint8_t* q;
  float* scale;
  int64_t x_stride, res_stride, gate_stride, res_out_stride, y_stride, q_stride, scale_stride;
  int64_t rows;
  int cols;
  float eps, res_scale, block_scale;
  bool wide_q;      // rows of q start at 8-byte addresses
};

// The sum over a CTA's threads, for all of them; `part` is not written again
// before another barrier of the CTA.
__device__ __forceinline__ float block_sum(float sum, float* part) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  return sum;
}

// A CTA takes every gridDim-th row.  A thread holds a unit of 8 values of each
// of kChunks chunks in registers, so a row is read once, and loads the next row
// before the reductions of this one, so that copies are always under way.  The
// row vectors (weights, gate) stay in registers where a row has few chunks, and
// come from the L1 cache again for every row otherwise.  Rows of 8 chunks (more
// than 16384 columns) fill the registers: their loads are not ahead.
constexpr int most_threads(int chunks) { return chunks == 1 ? 1024 : chunks == 2 ? 384 : 512; }
template <typename T, int kChunks, bool kAligned, bool kMatrix>
__global__ void __launch_bounds__(most_threads(kChunks), kChunks == 2 ? 2 : 1) norms_kernel(const __grid_constant__ NormsParams p) {
  constexpr bool kKeep = kChunks <= 2, kAhead = kChunks < 8;
  __shared__ float sums[2][2][32];   // two rows in turn, two sums: one barrier a sum
  const int tid = threadIdx.x, nthr = blockDim.x;
  uint4 x[kChunks], res[kChunks], gate[kChunks], post[kChunks], w[kChunks];
  auto col = [&](int c) { return (c * nthr + tid) * kVec; };
  auto load = [&](const void* base, int64_t row, int64_t stride, int c) {
    const T* at = static_cast<const T*>(base) + row * stride;
    return kAligned ? pw::load8<T, true>(at, col(c), p.cols) : pw::load_granule(at, col(c) - pw::row_shift(at), p.cols);
  };
  auto unit = [&](const uint4& v, const void* base, int64_t row, int64_t stride, int c, float (&t)[kVec]) {
    const T* at = static_cast<const T*>(base) + row * stride;
    pw::unpack8<T>(kAligned ? v : pw::unit_of(v, at, col(c), p.cols), t);
  };
  auto store = [&](void* base, int64_t row, int64_t stride, int c, const float (&t)[kVec]) {
    T* at = static_cast<T*>(base) + row * stride;
    if (kAligned)
      pw::store8<T, true>(at, col(c), p.cols, t);
    else
      pw::store_unit(at, col(c), p.cols, t);
  };
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      x[c] = load(p.x, row, p.x_stride, c);
      res[c] = load(p.res, row, p.res_stride, c);
      if (kMatrix) gate[c] = load(p.gate, row, p.gate_stride, c);
    }
  };
  auto vector = [&](const void* base, int c) {
    const T* v = static_cast<const T*>(base);
    if (kAligned || ((reinterpret_cast<uintptr_t>(v) & 15) == 0 && col(c) + kVec <= p.cols)) return pw::load8<T, true>(v, col(c), p.cols);
    return pw::load8<T, false>(v, col(c), p.cols);
  };
  if (kAhead) load_row(blockIdx.x);
  if (kKeep) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (p.post) post[c] = vector(p.post, c);
      if (!kMatrix && p.gate) gate[c] = vector(p.gate, c);
      if (p.w) w[c] = vector(p.w, c);
    }
  }
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    if (!kAhead) load_row(row);
    float v[kChunks][kVec];
    uint4 r_in[kChunks], g_in[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      unit(x[c], p.x, row, p.x_stride, c, v[c]);
      r_in[c] = res[c];
      if (kMatrix) g_in[c] = gate[c];
    }
    if (kAhead && row + gridDim.x < p.rows) load_row(row + gridDim.x);
    float factor = p.block_scale;
    if (p.post) {
      // the sums of squares in 32 bits: 8 x kChunks terms a thread, then a tree
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < kVec; ++i) sum += v[c][i] * v[c][i];
      factor *= rsqrtf(block_sum(sum, sums[turn][0]) * inv_cols + p.eps);
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float t[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[c][i] *= factor;
      if (p.post) {
        pw::unpack8<T>(kKeep ? post[c] : vector(p.post, c), t);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[c][i] *= t[i];
      }
      if (p.gate) {
        if (kMatrix)
          unit(g_in[c], p.gate, row, p.gate_stride, c, t);
        else
          pw::unpack8<T>(kKeep ? gate[c] : vector(p.gate, c), t);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[c][i] *= t[i];
      }
      unit(r_in[c], p.res, row, p.res_stride, c, t);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        v[c][i] = fmaf(p.res_scale, t[i], v[c][i]);
        sum += v[c][i] * v[c][i];
      }
    }
    // (after every read of this row: residual_out may be the residual)
    if (p.res_out) {
      if (!kAligned) __syncthreads();
#pragma unroll
      for (int c = 0; c < kChunks; ++c) store(p.res_out, row, p.res_out_stride, c, v[c]);
    }
    if (!p.y && !p.q) continue;
    const float rs = rsqrtf(block_sum(sum, sums[turn][1]) * inv_cols + p.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float t[kVec];
      pw::unpack8<T>(kKeep ? w[c] : vector(p.w, c), t);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[c][i] = v[c][i] * rs * t[i];
      if (p.y) store(p.y, row, p.y_stride, c, v[c]);
      if (p.q) {
        const float s = pw::group_scale(v[c]);
        if (col(c) < p.cols && (tid & 15) == 0) p.scale[row * p.scale_stride + col(c) / pw::kGroup] = s;
        uint8_t* q = p.q + row * p.q_stride;
        if (kAligned || (p.wide_q && col(c) + kVec <= p.cols))
          pw::store8_e4m3<true>(q, col(c), p.cols, v[c], pw::Divisor(s));
        else
          pw::store8_e4m3<false>(q, col(c), p.cols, v[c], pw::Divisor(s));
      }
    }
  }
}

template <typename T, int kChunks, bool kAligned, bool kMatrix>
int launch_chunks(const NormsParams& p, int threads, int sms, cudaStream_t s) {
  // as many CTAs as run at once
  static int regs = 0;
  if (!regs) {
    cudaFuncAttributes at{};
    PW_CUDA_TRY(cudaFuncGetAttributes(&at, norms_kernel<T, kChunks, kAligned, kMatrix>));
    regs = (at.numRegs + 7) & ~7;
  }
  const int by_regs = 65536 / (regs * threads), by_threads = 2048 / threads;
  const int at_once = by_regs < by_threads ? (by_regs < 1 ? 1 : by_regs) : by_threads;
  const int64_t most = static_cast<int64_t>(sms) * at_once;
  norms_kernel<T, kChunks, kAligned, kMatrix><<<static_cast<unsigned>(p.rows < most ? p.rows : most), threads, 0, s>>>(p);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

template <typename T, bool kAligned, bool kMatrix>
int launch_rows(const NormsParams& p, cudaStream_t s) {
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  // Few rows: one chunk a thread where 1024 threads suffice, for the shortest
  // way through a row.  Many: up to 512 threads, so that several CTAs an SM are
  // at different stages.
  const int units = (p.cols + kVec - 1) / kVec, most = p.rows <= sms ? 1024 : 512;
  int chunks = 1;
  while ((units + chunks - 1) / chunks > (chunks > 1 ? most_threads(chunks) : most)) chunks *= 2;
  const int threads = ((units + chunks - 1) / chunks + 31) & ~31;
  switch (chunks) {
    case 1: return launch_chunks<T, 1, kAligned, kMatrix>(p, threads, sms, s);
    case 2: return launch_chunks<T, 2, kAligned, kMatrix>(p, threads, sms, s);
    case 4: return launch_chunks<T, 4, kAligned, kMatrix>(p, threads, sms, s);
    default: return launch_chunks<T, 8, kAligned, kMatrix>(p, threads, sms, s);
  }
}

template <typename T>
int launch(const NormsParams& p, bool aligned, cudaStream_t s) {
  const bool matrix = p.gate && p.gate_stride != 0 && p.rows > 1;
  if (aligned) return matrix ? launch_rows<T, true, true>(p, s) : launch_rows<T, true, false>(p, s);
  return matrix ? launch_rows<T, false, true>(p, s) : launch_rows<T, false, false>(p, s);
}

}  // namespace

extern "C" int pw_norm_add_norm(const pw_norms_args* args, void* stream) {
  if (!args) return pw::set_error(PW_ERR_INVALID_ARG, "norm_add_norm: NULL argument");
  const pw_norms_args& a = *args;
  const char* op = "norm_add_norm";
  if (!pw::is_16bit(a.dtype)) return pw::set_error(PW_ERR_UNSUPPORTED, "%s: dtype %d", op, a.dtype);
  if (a.rows < 0 || a.cols < 1)
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: %lld rows of %d columns", op, static_cast<long long>(a.rows), a.cols);
  if (a.cols > kMaxCols || a.rows > 0x7FFFFFFF)
    return pw::set_error(PW_ERR_UNSUPPORTED, "%s: at most %d columns (got %d) and 2^31 - 1 rows", op, kMaxCols, a.cols);
  if (!(a.eps >= 0.0f)) return pw::set_error(PW_ERR_INVALID_ARG, "%s: eps %g", op, static_cast<double>(a.eps));
  if (!std::isfinite(a.residual_scale) || !std::isfinite(a.block_scale))
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: a scale is not finite", op);
  if (a.rows == 0) return PW_OK;
  if (!a.residual_out && !a.y && !a.q) return pw::set_error(PW_ERR_INVALID_ARG, "%s: no output", op);
  if (!a.q != !a.scale) return pw::set_error(PW_ERR_INVALID_ARG, "%s: 8-bit codes and scales come together", op);
  if (!a.weight != (!a.y && !a.q)) return pw::set_error(PW_ERR_INVALID_ARG, "%s: weight and y or q come together", op);
  if (int e = pw::check_matrix(op, "x", a.x_stride, a.cols)) return e;
  if (int e = pw::check_matrix(op, "residual", a.residual_stride, a.cols)) return e;
  if (a.gate && a.gate_stride != 0)
    if (int e = pw::check_matrix(op, "gate", a.gate_stride, a.cols)) return e;
  if (a.residual_out)
    if (int e = pw::check_matrix(op, "residual_out", a.residual_out_stride, a.cols)) return e;
  if (a.y)
    if (int e = pw::check_matrix(op, "y", a.y_stride, a.cols)) return e;
  if (a.q) {
    if (int e = pw::check_matrix(op, "q", a.q_stride, a.cols)) return e;
    if (int e = pw::check_matrix(op, "scale", a.scale_stride, (a.cols + pw::kGroup - 1) / pw::kGroup)) return e;
  }
  if (!a.x || !a.residual) return pw::set_error(PW_ERR_INVALID_ARG, "%s: NULL argument", op);
  for (const void* ptr : {a.x, a.residual, a.post_weight, a.gate, a.weight, static_cast<const void*>(a.residual_out),
                          static_cast<const void*>(a.y)})
    if (!pw::aligned(ptr, 2)) return pw::set_error(PW_ERR_INVALID_ARG, "%s: a pointer is not aligned to its values", op);
  if (!pw::aligned(a.scale, 4)) return pw::set_error(PW_ERR_INVALID_ARG, "%s: a pointer is not aligned to its values", op);
  NormsParams p{};
  p.x = a.x;
  p.res = a.residual;
  p.post = a.post_weight;
  p.gate = a.gate;
  p.w = a.weight;
  p.res_out = a.residual_out;
  p.y = a.y;
  p.q = a.q;
  p.scale = a.scale;
  p.x_stride = a.x_stride;
  p.res_stride = a.residual_stride;
  p.gate_stride = a.gate_stride;
  p.res_out_stride = a.residual_out_stride;
  p.y_stride = a.y_stride;
  p.q_stride = a.q_stride;
  p.scale_stride = a.scale_stride;
  p.rows = a.rows;
  p.cols = a.cols;
  p.eps = a.eps;
  p.res_scale = a.residual_scale;
  p.block_scale = a.block_scale;
  p.wide_q = pw::codes_aligned(a.q, a.q_stride);
  const bool aligned = pw::rows_aligned(a.x, a.x_stride, a.cols) && pw::rows_aligned(a.residual, a.residual_stride, a.cols) &&
                       pw::rows_aligned(a.post_weight, 0, a.cols) && pw::rows_aligned(a.gate, a.gate_stride, a.cols) &&
                       pw::rows_aligned(a.weight, 0, a.cols) && pw::rows_aligned(a.residual_out, a.residual_out_stride, a.cols) &&
                       pw::rows_aligned(a.y, a.y_stride, a.cols) && p.wide_q;
  cudaStream_t s = pw::as_stream(stream);
  return a.dtype == PW_DTYPE_F16 ? launch<__half>(p, aligned, s) : launch<__nv_bfloat16>(p, aligned, s);
}
