// The norms on both sides of a block, with what is between them:
//
//   u = x * rsqrt(mean(x^2) + eps) * post_weight      (x: the block's output)
//   r = residual_scale * residual + block_scale * gate * u
//   y = r * rsqrt(mean(r^2) + eps) * weight           (in 16 bits and/or in e4m3)
//
// Every value is read and written once: memory bandwidth bounds it (8192 x 6144
// bf16 to e4m3 60.5 us, 5.8 TB/s; 8192 x 5120 in 16 bits 52.5 us, 6.4 TB/s; with a gate for
// every row 75 us at 6144 columns, 6.7 TB/s), for a few rows the latency of one load, two
// reductions and one store (one row of 4096: 2.6 us).  Odd widths: 2.5 us for a row of
// every CTA, 1.8 at 5120 columns, and 2.7 us more to begin (1531 x 5121 20 us, 13.4 at
// 5120); issue is at 49 % and 33 % of the warps are there, so it is neither memory nor the
// 46 instructions a value alone.
#include "rows.cuh"

namespace {

using pw::Access;

constexpr int kMaxCols = 32768;       // 512 threads x 64 columns

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
  int q_align;      // 16 or 8: rows of q start at such addresses; 1 otherwise
};

constexpr int kMaxWarps = 16;
// Rows of one part: two CTAs an SM, whose 64 registers a thread set the threads; 80
// with a gate for every row, and where cells move (8192 x 5121: 73 us, 94 with 64).
constexpr int most_threads(int parts, bool more) { return parts == 1 && more ? 384 : 32 * kMaxWarps; }
constexpr int line_floats(int parts) { return parts * 32 * kMaxWarps + 1; }

// The sum over a CTA's threads, for all of them.  `part` (of the warps, zeros
// behind them) is not written again before another barrier of the CTA.
__device__ __forceinline__ float block_sum(uint64_t two, float* part) {
  float lo, hi;
  pw::unpack_f32x2(two, lo, hi);
  float sum = lo + hi;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxWarps / 4; ++i) {
    if (128 * i >= static_cast<int>(blockDim.x)) break;
    const float4 v = reinterpret_cast<const float4*>(part)[i];
    sum += (v.x + v.y) + (v.z + v.w);
  }
  return sum;
}

// A CTA takes every gridDim-th row.  A thread holds 16 neighbouring columns of each
// of kParts parts of the row in registers, so a row is read once, and starts the
// loads of the next row as soon as a register is free, so that copies are always
// under way.  The vectors of a row's columns (block_scale * post_weight * gate,
// and weight) wait as 32-bit numbers in shared memory, where each thread finds its
// own (kSame, whose columns move with the row: [column % 16][column / 16], so that
// neighbouring threads find neighbouring words).  Rows of more than 16384 columns
// fill the registers and more: they read the vectors from the L1 cache and load
// nothing ahead (2048 rows of 16384: 47 us, of 20000 104, at 6.8 TB/s 40 and 48); shifted
// ones of that length also spill up to 200 bytes a thread (2048 x 20001: 240 us).
// Arithmetic in packed pairs: with single instructions the kernel was bound by
// their number (39 a value; 8192 x 6144 to e4m3 102 us, now 60.5).
template <typename T, int kParts, Access kAccess, bool kMatrix>
__global__ void __launch_bounds__(most_threads(kParts, kMatrix || kAccess == Access::kSame), kParts == 1 ? 2 : 1) norms_kernel(const __grid_constant__ NormsParams p) {
  constexpr bool kKeep = kParts <= 2, kAhead = kParts <= 2, kSame = kAccess == Access::kSame;
  static_assert(!kSame || kKeep, "moving columns find the vectors in shared memory");
  __shared__ __align__(16) float sums[2][2][kMaxWarps];   // two rows in turn, two sums: one barrier a sum
  extern __shared__ __align__(16) uint64_t vectors[];     // [kParts][2][4][threads] of two pairs
  __shared__ uint32_t tops[kSame ? 2 : 1][kSame ? kParts * 32 * kMaxWarps * 16 / pw::kGroup + 1 : 1];   // of the groups, two rows in turn
  const int tid = threadIdx.x, nthr = blockDim.x;
  constexpr int kPitch = line_floats(kParts);   // kSame: of a line of the vectors, [which][16 lines][cells, from -1]
  float* const lines = reinterpret_cast<float*>(vectors);
  if constexpr (kSame) {
    for (int i = tid; i < static_cast<int>(sizeof(tops) / 4); i += nthr) (&tops[0][0])[i] = 0u;
    if (tid < 32) lines[tid * kPitch] = 0.0f;
  }
  for (int i = tid; i < 4 * kMaxWarps; i += nthr) (&sums[0][0][0])[i] = 0.0f;
  int shift = 0;   // kSame: of the row
  auto shift_of = [&](int64_t row) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const T*>(p.x) + row * p.x_stride) >> 1 & 15);
  };
  auto col = [&](int c) { return (c * nthr + tid) * 16 - (kSame ? shift : 0); };
  auto at = [&](const void* base, int64_t row, int64_t stride) { return static_cast<const T*>(base) + row * stride; };
  auto load = [&](const void* base, int64_t row, int64_t stride, int c) {
    if constexpr (kSame) {
      // (of a row ahead: its own shift.)  The matrix may end before the first row's first cell does, and with
      // the last row.
      const int first = (c * nthr + tid) * 16 - shift_of(row);
      const bool inside = row > 0 && row + 1 < p.rows && stride >= 16;
      return pw::load_cell(at(base, row, stride), first, p.cols, inside || (first >= 0 && first + 16 <= p.cols));
    } else {
      return pw::load16<T, kAccess>(at(base, row, stride), col(c), p.cols);
    }
  };
  auto values = [&](pw::Sixteen v, const void* base, int64_t row, int64_t stride, int c, uint64_t (&t)[8]) {
    if constexpr (kSame) {
      pw::clip_cell(v, col(c), p.cols);
      pw::unpack16<T>(v, t);
    } else {
      pw::unpack16<T>(pw::columns16<T, kAccess>(v, at(base, row, stride), col(c), p.cols), t);
    }
  };
  auto store = [&](void* base, int64_t row, int64_t stride, int c, const uint64_t (&t)[8]) {
    pw::store16<T, kAccess>(static_cast<T*>(base) + row * stride, col(c), p.cols, pw::pack16<T>(t));
  };
  // block_scale * post * gate (which = 0) or the weight (1) at the thread's columns, from memory
  auto vector = [&](int which, int c, uint64_t (&t)[8]) {
    const uint64_t scale = pw::twice(which ? 1.0f : p.block_scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = scale;
    const void* of[2] = {which ? p.w : p.post, which || kMatrix ? nullptr : p.gate};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!of[k]) continue;
      const T* v = static_cast<const T*>(of[k]);
      pw::Sixteen u;
      if (kAccess == Access::kWide || kAccess == Access::kHalves) {
        u = pw::load16<T, Access::kHalves>(v, col(c), p.cols);
      } else {
        u.lo = pw::load8<T, false>(v, col(c), p.cols);
        u.hi = pw::load8<T, false>(v, col(c) + pw::kVec, p.cols);
      }
      uint64_t f[8];
      pw::unpack16<T>(u, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = pw::mul_f32x2(t[i], f[i]);
    }
  };
  auto kept = [&](int which, int c, uint64_t (&t)[8]) {
    if constexpr (!kKeep) {
      vector(which, c, t);
    } else if constexpr (kSame) {
      // columns below 16 cell belong to the cell before
      const float* const here = lines + which * 16 * kPitch + c * nthr + tid + 1 - shift * kPitch;
      const float* const before = here + 16 * kPitch - 1;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        t[i] = pw::pack_f32x2(__float_as_uint((2 * i < shift ? before : here)[2 * i * kPitch]),
                              __float_as_uint((2 * i + 1 < shift ? before : here)[(2 * i + 1) * kPitch]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const ulonglong2 v = reinterpret_cast<const ulonglong2*>(vectors)[((c * 2 + which) * 4 + i) * nthr + tid];
        t[2 * i] = v.x;
        t[2 * i + 1] = v.y;
      }
    }
  };
  pw::Sixteen x[kParts], res[kParts], gate[kParts];
  int64_t row = blockIdx.x;
#pragma unroll
  for (int c = 0; c < kParts; ++c) {
    if (!kAhead) break;
    x[c] = load(p.x, row, p.x_stride, c);
    res[c] = load(p.res, row, p.res_stride, c);
    if (kMatrix) gate[c] = load(p.gate, row, p.gate_stride, c);
  }
  if (kKeep) {
#pragma unroll
    for (int c = 0; c < kParts; ++c)
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint64_t t[8];
        vector(which, c, t);
        if constexpr (kSame) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float two[2];
            pw::unpack_f32x2(t[i], two[0], two[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) lines[(which * 16 + 2 * i + j) * kPitch + c * nthr + tid + 1] = two[j];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<ulonglong2*>(vectors)[((c * 2 + which) * 4 + i) * nthr + tid] = make_ulonglong2(t[2 * i], t[2 * i + 1]);
        }
      }
  }
  __syncthreads();
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  const uint64_t res_scale = pw::twice(p.res_scale);
  for (int turn = 0; row < p.rows; row += gridDim.x, turn ^= 1) {
    const bool more = kAhead && row + gridDim.x < p.rows;
    if (kSame) shift = shift_of(row);
    uint64_t v[kParts][8];
#pragma unroll
    for (int c = 0; c < kParts; ++c) {
      if (!kAhead) x[c] = load(p.x, row, p.x_stride, c);
      values(x[c], p.x, row, p.x_stride, c, v[c]);
      if (more) x[c] = load(p.x, row + gridDim.x, p.x_stride, c);
    }
    uint64_t factor = pw::twice(1.0f);
    if (p.post) {
      // the sums of squares in 32 bits: 8 x kParts terms in two sums a thread, then a tree
      uint64_t sum = 0;
#pragma unroll
      for (int c = 0; c < kParts; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = pw::fma_f32x2(v[c][i], v[c][i], sum);
      factor = pw::twice(rsqrtf(block_sum(sum, sums[turn][0]) * inv_cols + p.eps));
    }
    uint64_t sum = 0;
#pragma unroll
    for (int c = 0; c < kParts; ++c) {
      uint64_t t[8];
      kept(0, c, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = pw::mul_f32x2(pw::mul_f32x2(v[c][i], factor), t[i]);
      if (kMatrix) {
        if (!kAhead) gate[c] = load(p.gate, row, p.gate_stride, c);
        values(gate[c], p.gate, row, p.gate_stride, c, t);
        if (more) gate[c] = load(p.gate, row + gridDim.x, p.gate_stride, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = pw::mul_f32x2(v[c][i], t[i]);
      }
      if (!kAhead) res[c] = load(p.res, row, p.res_stride, c);
      values(res[c], p.res, row, p.res_stride, c, t);
      if (more) res[c] = load(p.res, row + gridDim.x, p.res_stride, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = pw::fma_f32x2(res_scale, t[i], v[c][i]);
        sum = pw::fma_f32x2(v[c][i], v[c][i], sum);
      }
    }
    if (p.res_out) {
      // the results may lie over x or the residual, whose granules neighbouring warps share
      if (kAccess == Access::kShifted) __syncthreads();
#pragma unroll
      for (int c = 0; c < kParts; ++c) store(p.res_out, row, p.res_out_stride, c, v[c]);
    }
    if (!p.y && !p.q) continue;
    factor = pw::twice(rsqrtf(block_sum(sum, sums[turn][1]) * inv_cols + p.eps));
#pragma unroll
    for (int c = 0; c < kParts; ++c) {
      uint64_t t[8];
      kept(1, c, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = pw::mul_f32x2(pw::mul_f32x2(v[c][i], factor), t[i]);
      if (p.y) store(p.y, row, p.y_stride, c, v[c]);
      if (kSame && p.q) continue;   // below
      if (p.q) {
        // 8 neighbouring threads hold a group
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float lo, hi;
          pw::unpack_f32x2(v[c][i], lo, hi);
          top = pw::max3_nan(top, fabsf(lo), fabsf(hi));
        }
#pragma unroll
        for (int o = 4; o; o >>= 1) top = pw::max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float s = pw::max_nan(top / pw::kE4m3Max, pw::kMinScale);
        if (col(c) < p.cols && (tid & 7) == 0) p.scale[row * p.scale_stride + col(c) / pw::kGroup] = s;
        const pw::PairDivisor by{pw::Divisor(s)};
        uint32_t code[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) code[i] = pw::e4m3_pairs(by(v[c][2 * i]), by(v[c][2 * i + 1]));
        pw::store_codes16(p.q + row * p.q_stride, col(c), p.cols, code, p.q_align);
      }
    }
    if constexpr (kSame) {
      if (!p.q) continue;
      // A thread's columns belong to one group or two; each group's largest
      // magnitude by way of shared memory (as whole numbers, which rank the same
      // way, NaN above infinity).
      auto split_of = [&](int c) { return (col(c) + 15) / pw::kGroup * pw::kGroup - col(c); };   // columns before the second one
#pragma unroll
      for (int c = 0; c < kParts; ++c) {
        if (col(c) >= p.cols) continue;
        const int split = split_of(c), group = (col(c) + 15) / pw::kGroup;
        float before = 0.0f, top = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float two[2];
          pw::unpack_f32x2(v[c][i / 2], two[0], two[1]);
          const float f = fabsf(two[i & 1]);
          before = pw::max_nan(before, i < split ? f : 0.0f);
          top = pw::max_nan(top, i < split ? 0.0f : f);
        }
        if (col(c) + max(split, 0) < p.cols) atomicMax(&tops[turn][group], __float_as_uint(top));
        if (split > 0 && col(c) >= 0) atomicMax(&tops[turn][group - 1], __float_as_uint(before));
      }
      __syncthreads();
      for (int i = tid; i < static_cast<int>(sizeof(tops[0]) / 4); i += nthr) tops[turn ^ 1][i] = 0u;   // read to the end a row ago
#pragma unroll
      for (int c = 0; c < kParts; ++c) {
        if (col(c) >= p.cols) continue;
        const int split = split_of(c), group = (col(c) + 15) / pw::kGroup;
        auto scale_of = [&](int g) { return pw::max_nan(__uint_as_float(tops[turn][g]) / pw::kE4m3Max, pw::kMinScale); };
        const float s = scale_of(group);
        const pw::Divisor by(s), by_before(split > 0 && group > 0 ? scale_of(group - 1) : s);
        if (split >= 0 && split < 16 && col(c) + split < p.cols) p.scale[row * p.scale_stride + group] = s;   // it begins here
        uint32_t code[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[4];
          pw::unpack_f32x2(v[c][2 * i], f[0], f[1]);
          pw::unpack_f32x2(v[c][2 * i + 1], f[2], f[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = 4 * i + j < split ? by_before(f[j]) : by(f[j]);
          code[i] = pw::e4m3x4(f[0], f[1], f[2], f[3]);
        }
        pw::store_codes16(p.q + row * p.q_stride, col(c), p.cols, code, 16);
      }
    }
  }
}

template <typename T, int kParts, Access kAccess, bool kMatrix>
int launch_parts(const NormsParams& p, int threads, int sms, cudaStream_t s) {
  constexpr size_t kMost = kParts <= 2 ? 2 * 64 * static_cast<size_t>(line_floats(kParts)) : 0;
  const size_t smem = kAccess == Access::kSame ? kMost : kParts <= 2 ? 2 * 64 * static_cast<size_t>(kParts) * threads : 0;
  constexpr int kDevs = 64;
  static int known[kDevs][kMaxWarps + 1] = {};   // CTAs that an SM runs at once, by the number of warps
  int dev = 0;
  PW_CUDA_TRY(cudaGetDevice(&dev));
  int at_once = dev < kDevs ? known[dev][threads / 32] : 0;
  if (!at_once) {
    if (kParts <= 2)
      PW_CUDA_TRY(cudaFuncSetAttribute(norms_kernel<T, kParts, kAccess, kMatrix>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kMost)));
    PW_CUDA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&at_once, norms_kernel<T, kParts, kAccess, kMatrix>, threads, smem));
    if (at_once < 1) return pw::set_error(PW_ERR_CUDA, "norm_add_norm: the kernel does not fit an SM");
    if (dev < kDevs) known[dev][threads / 32] = at_once;
  }
  const int64_t most = static_cast<int64_t>(sms) * at_once;
  norms_kernel<T, kParts, kAccess, kMatrix><<<static_cast<unsigned>(p.rows < most ? p.rows : most), threads, smem, s>>>(p);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

template <typename T, Access kAccess, bool kMatrix>
int launch_rows(const NormsParams& p, cudaStream_t s) {
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  const int units = (p.cols + (kAccess == Access::kSame ? 30 : 15)) / 16;   // 16 columns each, or up to 15 before them
  int parts = 1;
  while ((units + parts - 1) / parts > most_threads(parts, kMatrix || kAccess == Access::kSame)) parts *= 2;
  const int threads = ((units + parts - 1) / parts + 31) & ~31;
  switch (parts) {
    case 1: return launch_parts<T, 1, kAccess, kMatrix>(p, threads, sms, s);
    case 2: return launch_parts<T, 2, kAccess, kMatrix>(p, threads, sms, s);
    default:
      if constexpr (kAccess == Access::kSame)
        return pw::set_error(PW_ERR_UNSUPPORTED, "norm_add_norm: moving columns in four parts");   // not chosen
      else
        return launch_parts<T, 4, kAccess, kMatrix>(p, threads, sms, s);
  }
}

template <typename T, Access kAccess>
int launch_access(const NormsParams& p, cudaStream_t s) {
  const bool matrix = p.gate && p.gate_stride != 0 && p.rows > 1;
  return matrix ? launch_rows<T, kAccess, true>(p, s) : launch_rows<T, kAccess, false>(p, s);
}

template <typename T>
int launch(const NormsParams& p, Access access, cudaStream_t s) {
  switch (access) {
    case Access::kWide: return launch_access<T, Access::kWide>(p, s);
    case Access::kHalves: return launch_access<T, Access::kHalves>(p, s);
    case Access::kSame: return launch_access<T, Access::kSame>(p, s);
    default: return launch_access<T, Access::kShifted>(p, s);
  }
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
  const struct { const void* ptr; int64_t stride; } matrices[] = {
      {a.x, a.x_stride}, {a.residual, a.residual_stride}, {a.gate, a.gate_stride}, {a.residual_out, a.residual_out_stride},
      {a.y, a.y_stride}};
  const auto whole = [&](size_t bytes) {   // every row of every matrix in pieces of `bytes`, the vectors in halves
    const int64_t values = static_cast<int64_t>(bytes) / 2;
    if (a.cols % values) return false;
    for (const auto& m : matrices)
      if (m.ptr && (!pw::aligned(m.ptr, bytes) || m.stride % values)) return false;
    return pw::aligned(a.post_weight, 16) && pw::aligned(a.weight, 16);
  };
  // Widths or strides of odd numbers of values, as in matrices of an odd width one
  // beside the other in memory: every row starts at its own place of a 32-byte cell, the same in all
  // matrices.  (A gate of one row is a vector.  Where a row takes four parts, the
  // vectors do not wait in shared memory.)
  const auto same = [&] {
    const auto place = [](const void* ptr) { return reinterpret_cast<uintptr_t>(ptr) / 2 % 16; };
    for (const auto& m : matrices)
      if (m.ptr && !(m.ptr == a.gate && (a.gate_stride == 0 || a.rows == 1)) &&
          (place(m.ptr) != place(a.x) || (a.rows > 1 && (m.stride - a.x_stride) % 16)))
        return false;
    if (a.q && (reinterpret_cast<uintptr_t>(a.q) % 16 != place(a.x) || (a.rows > 1 && (a.q_stride - a.x_stride) % 16))) return false;
    return (a.cols + 30) / 16 <= 2 * 32 * kMaxWarps;
  };
  const Access access = whole(32) ? Access::kWide : whole(16) ? Access::kHalves : same() ? Access::kSame : Access::kShifted;
  p.q_align = pw::aligned(a.q, 16) && a.q_stride % 16 == 0 ? 16 : pw::aligned(a.q, 8) && a.q_stride % 8 == 0 ? 8 : 1;
  cudaStream_t s = pw::as_stream(stream);
  return a.dtype == PW_DTYPE_F16 ? launch<__half>(p, access, s) : launch<__nv_bfloat16>(p, access, s);
}
