// Log probabilities of a model's next tokens from its logits, by rows:
//
//   z = scale * logit,  m = max z,  S = sum e^(z - m),  T = sum e^(z - m) (z - m)
//   log p(t) = z_t - m - ln S,   lse = m + ln S,   entropy = ln S - T / S
//
// in one pass with the running maximum: m' > m turns S into e^(m - m') S and T
// into e^(m - m') (T + (m - m') S).  Both terms of the entropy are positive and do
// not cancel where one token has nearly all of the probability.
//
// The most probable tokens come from the same pass.  Every thread remembers the
// largest logit of each of its segments, 8 vectors of 32 bytes and more.  The k-th largest
// of the threads' maxima is no larger than the k-th largest value, so the k largest
// lie in the segments whose maxima are not below it, at most 4 k of them: those are read again,
// from L2, and their values go through a sorted list in the registers of each warp.
//
// Memory bandwidth bounds it (4096 rows of 131072 bf16 logits: 178 us with one
// alternative, 6.0 TB/s, and 161 without), with the instructions close behind: 9 a
// value, one of them an exponential (ex2.approx: within 2^-22 of its value).  For few
// rows it is the chain of a load, reductions and the second look at a few segments
// (one row of 32000: 8.2 us), and so it is for many short ones, a row a CTA: 4096 rows of 1000 bf16 logits 15.7 us without alternatives,
// 25.4 with one, 42 with twenty, of 8000 20.3, 30 and 46.  Few rows: a cluster of up to 8
// CTAs shares one and joins its results through distributed shared memory.
#include <type_traits>

#include "ops_common.cuh"
#include "umma.cuh"

namespace {

constexpr int kSegments = 4;          // of a thread
constexpr int kAhead = 4;             // vectors that a thread has under way
constexpr int kLeast = 8;             // vectors of a segment at the least, where there are several
constexpr int kFold = 64;             // vectors of a thread whose terms one sum takes: 512 in each of two parts
constexpr int kMaxTop = 32;           // a list is one value a lane
constexpr int kMaxCluster = 8;        // CTAs of a row
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNothing = -200.0f;   // 2^-200 is 0, and a finite factor leaves it 0 in T

struct LogprobParams {
  pw_logprob_args a;
  float scale_log2;   // scale * log2(e): sums run in powers of two
};

// The element types of the logits; a vector is 32 bytes of them.
template <typename T>
struct Vec;
template <typename T>
__device__ __forceinline__ float largest16(const uint32_t (&w)[8]) {
  using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
  const T2* v = reinterpret_cast<const T2*>(w);
  const T2 m = __hmax2(__hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3])), __hmax2(__hmax2(v[4], v[5]), __hmax2(v[6], v[7])));
  return fmaxf(pw::to_float(m.x), pw::to_float(m.y));
}
template <>
struct Vec<__half> {
  static constexpr int kSize = 16;
  static constexpr uint32_t kLowest = 0xFC00FC00u;   // -inf
  static __device__ __forceinline__ float largest(const uint32_t (&w)[8]) { return largest16<__half>(w); }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kSize = 16;
  static constexpr uint32_t kLowest = 0xFF80FF80u;
  static __device__ __forceinline__ float largest(const uint32_t (&w)[8]) { return largest16<__nv_bfloat16>(w); }
};
template <>
struct Vec<float> {
  static constexpr int kSize = 8;
  static constexpr uint32_t kLowest = 0xFF800000u;
  static __device__ __forceinline__ float largest(const uint32_t (&w)[8]) {
    const float* v = reinterpret_cast<const float*>(w);
    return fmaxf(pw::max3(pw::max3(v[0], v[1], v[2]), v[3], v[4]), pw::max3(v[5], v[6], v[7]));
  }
};

// Values 2i and 2i + 1 of a vector.
template <typename T>
__device__ __forceinline__ void two_values(const uint32_t (&w)[8], int i, float& lo, float& hi) {
  if constexpr (Vec<T>::kSize == 8) {
    lo = __uint_as_float(w[2 * i]);
    hi = __uint_as_float(w[2 * i + 1]);
  } else {
    pw::unpack2<T>(w[i], lo, hi);
  }
}

// A row as vectors at 32-byte addresses: the first and the last may hold values
// of its neighbours, which are not read.
template <typename T>
struct Row {
  const T* data;      // value `lead` of vector 0
  int lead, size, vectors;
  __device__ __forceinline__ Row(const void* base, int64_t stride, int64_t row, int n) {
    data = static_cast<const T*>(base) + row * stride;
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(data) & 31) / sizeof(T));
    size = n;
    vectors = (lead + n + Vec<T>::kSize - 1) / Vec<T>::kSize;
  }
  __device__ __forceinline__ int first_of(int v) const { return v * Vec<T>::kSize - lead; }
  // Vector v, or nothing but -inf from vector `end` on.
  __device__ __forceinline__ void load(int v, int end, uint32_t (&w)[8]) const {
    const int first = first_of(v);
    if (first >= 0 && first + Vec<T>::kSize <= size && v < end) {
      asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(data + first));
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = Vec<T>::kLowest;
    if (v >= end) return;
#pragma unroll
    for (int i = 0; i < Vec<T>::kSize; ++i) {
      if (first + i < 0 || first + i >= size) continue;
      if constexpr (Vec<T>::kSize == 8) {
        w[i] = reinterpret_cast<const uint32_t*>(data)[first + i];
      } else {
        const uint32_t x = reinterpret_cast<const uint16_t*>(data)[first + i];
        w[i >> 1] = i & 1 ? (w[i >> 1] & 0xFFFFu) | x << 16 : (w[i >> 1] & 0xFFFF0000u) | x;
      }
    }
  }
};

// ---------------------------------------------------------------- sums
// S and T of the logits so far, in powers of two, relative to the largest of them,
// m (to 0 while there is none but -inf).  Differences x - m are formed first: they
// are exact near the maximum whatever its size.
struct alignas(16) Sums {
  float m, s, t;
};
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }
// Moves the sums to a larger maximum.  (A maximum that was -inf has sums of 0.)
__device__ __forceinline__ void raise(Sums& a, float m, float scale_log2) {
  const float by = a.m == -INFINITY ? kNothing : fmaxf((a.m - m) * scale_log2, kNothing), keep = pw::exp2_fast(by);
  a.t = keep * (a.t + by * a.s);
  a.s *= keep;
  a.m = m;
}
__device__ __forceinline__ Sums joined(Sums a, Sums b, float scale_log2) {
  const float m = fmaxf(a.m, b.m);
  if (a.m != m) raise(a, m, scale_log2);
  if (b.m != m) raise(b, m, scale_log2);
  return {m, a.s + b.s, a.t + b.t};
}

// The sums of `n` lanes (a power of two) together, in all of them.
__device__ __forceinline__ Sums joined_lanes(Sums a, int n, float scale_log2) {
  for (int o = n / 2; o; o >>= 1)
    a = joined(a, Sums{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o),
                       __shfl_xor_sync(0xFFFFFFFFu, a.t, o)}, scale_log2);
  return a;
}

// ---------------------------------------------------------------- ranked keys
// A value and its index as one number: larger is more probable, equal values
// rank by the lower index.  NaN ranks as -inf; 0 is no key.
__device__ __forceinline__ uint32_t rank_of(float v) {
  v = v != v ? -INFINITY : v + 0.0f;   // -0 ranks as 0
  const uint32_t u = __float_as_uint(v);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ranked(uint32_t r) { return __uint_as_float(r & 0x80000000u ? r ^ 0x80000000u : ~r); }
__device__ __forceinline__ uint64_t key_of(float v, int index) {
  return static_cast<uint64_t>(rank_of(v)) << 32 | ~static_cast<uint32_t>(index);
}
__device__ __forceinline__ int index_of(uint64_t key) { return static_cast<int>(~static_cast<uint32_t>(key)); }

// A list is one key a lane, in falling order.
__device__ __forceinline__ uint64_t other(uint64_t key, int mask) { return __shfl_xor_sync(0xFFFFFFFFu, key, mask); }
__device__ __forceinline__ uint64_t sorted(uint64_t key) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k *= 2)
#pragma unroll
    for (int j = k / 2; j; j /= 2) {
      const uint64_t o = other(key, j);
      const bool larger = ((lane & j) == 0) == ((lane & k) == 0);
      key = larger == (o > key) ? o : key;
    }
  return key;
}
// The 32 largest of two lists; `b_reversed` is the second one from its end.
__device__ __forceinline__ uint64_t merged(uint64_t a, uint64_t b_reversed) {
  const int lane = threadIdx.x & 31;
  uint64_t key = a > b_reversed ? a : b_reversed;
#pragma unroll
  for (int j = 16; j; j /= 2) {
    const uint64_t o = other(key, j);
    key = ((lane & j) == 0) == (o > key) ? o : key;
  }
  return key;
}
template <int kThreads, bool kLong>
struct Shared {
  static constexpr int kWarps = kThreads / 32;
  Sums sums[kWarps], total, folded[kLong ? kThreads : 1];
  uint64_t lists[kWarps][kMaxTop];
  uint64_t segments[kSegments][kThreads];   // their maxima; 0: no values
  uint64_t bound, best[kWarps], result[kMaxTop];
  int chosen[kSegments * kMaxTop], count;   // segments to look at, by the vector of their maximum
};

__device__ __forceinline__ uint64_t largest_key(uint64_t key) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t k = other(key, o);
    key = k > key ? k : key;
  }
  return key;
}
// The list of the first `warps` warps' lists together, in warp 0 (for one value only
// its first key).  All threads of the CTA come here.
template <int kThreads, bool kLong>
__device__ __forceinline__ uint64_t join_lists(uint64_t list, int warps, int top, Shared<kThreads, kLong>& sh) {
  constexpr int kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (top == 1) {
    if (lane == 0) sh.best[warp] = list;
    __syncthreads();
    return warp == 0 ? largest_key(lane < warps ? sh.best[lane] : 0) : 0;
  }
#pragma unroll
  for (int half = kWarps / 2; half; half /= 2) {
    if (half >= warps) continue;
    if (warp >= half && warp < 2 * half) sh.lists[warp][lane] = list;
    __syncthreads();
    if (warp < half) list = merged(list, sh.lists[warp + half][31 - lane]);
    __syncthreads();
  }
  return list;
}

// ---------------------------------------------------------------- the kernel
// CTA `rank` of the cluster takes its share of the row's vectors; a thread takes
// every kThreads-th of them.
//
// kLong: more than kFold vectors a thread.  Of n equal terms, one running sum may lose 2^-25 n
// of its size (2^28 tokens in a row: 9e-4), so these threads start afresh after kFold
// vectors and add up their sums in shared memory (1e-5).  Apart, because it costs the
// others 1 to 3 % (4096 x 131072 175.5 and 177.6 us).
template <typename T, int kThreads, bool kLong>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logprobs_kernel(const __grid_constant__ LogprobParams p, int cluster) {
  constexpr int kSize = Vec<T>::kSize, kWarps = kThreads / 32;
  __shared__ Shared<kThreads, kLong> sh;
  const pw_logprob_args& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cluster > 1 ? static_cast<int>(pw::cluster_rank()) : 0;
  const int64_t row_index = blockIdx.x / cluster;
  const Row<T> row(a.logits, a.stride, row_index, a.vocab);
  const int begin = static_cast<int>(static_cast<int64_t>(row.vectors) * rank / cluster);
  const int end = static_cast<int>(static_cast<int64_t>(row.vectors) * (rank + 1) / cluster);
  const int steps = (end - begin + kThreads - 1) / kThreads;
  const int length = max(kLeast, ((steps + kSegments - 1) / kSegments + kAhead - 1) / kAhead * kAhead);   // steps of a segment

  if (kLong) sh.folded[tid] = {-INFINITY, 0.0f, 0.0f};
  Sums sum{-INFINITY, 0.0f, 0.0f};
  uint64_t s2 = 0, t2 = 0;              // two parts of S and T
  auto fold_sums = [&] {
    float s0, s1, t0, t1;
    pw::unpack_f32x2(s2, s0, s1);
    pw::unpack_f32x2(t2, t0, t1);
    sh.folded[tid] = joined(sh.folded[tid], Sums{sum.m, s0 + s1, t0 + t1}, p.scale_log2);
    s2 = t2 = 0;
  };
  uint64_t best = 0;                    // the thread's largest value
  const uint64_t scale2 = pw::twice(p.scale_log2);
  for (int seg = 0; seg < kSegments && seg * length < steps; ++seg) {
    const int v0 = begin + seg * length * kThreads + tid, v1 = min(end, begin + (seg + 1) * length * kThreads);
    float top = -INFINITY;              // of the segment, and the vector that has it
    int at = v0;
    int until = v0;                     // the next fold
    for (int v = v0; v < v1; v += kAhead * kThreads) {
      if (kLong && v >= until) {
        fold_sums();                    // of what came before
        until = v + kFold * kThreads;
      }
      uint32_t w[kAhead][8];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) row.load(v + i * kThreads, v1, w[i]);
      float most = -INFINITY;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float x = Vec<T>::largest(w[i]);
        most = fmaxf(most, x);
        if (x > top) {
          top = x;
          at = v + i * kThreads;
        }
      }
      if (most > sum.m) {   // once for all the vectors: it takes as long as six values of one
        float lo, hi;
        pw::unpack_f32x2(s2, lo, hi);
        sum.s = lo + hi;
        pw::unpack_f32x2(t2, lo, hi);
        sum.t = lo + hi;
        raise(sum, most, p.scale_log2);
        s2 = pw::pack_f32x2(__float_as_uint(sum.s), 0u);
        t2 = pw::pack_f32x2(__float_as_uint(sum.t), 0u);
      }
      const uint64_t off2 = pw::twice(-base_of(sum.m));
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int j = 0; j < kSize / 2; ++j) {
          float lo, hi;
          two_values<T>(w[i], j, lo, hi);
          float d0, d1;
          pw::unpack_f32x2(pw::mul_f32x2(pw::add_f32x2(pw::pack_f32x2(__float_as_uint(lo), __float_as_uint(hi)), off2), scale2),
                           d0, d1);
          d0 = pw::max_nan(d0, kNothing);
          d1 = pw::max_nan(d1, kNothing);
          const uint64_t e = pw::pack_f32x2(__float_as_uint(pw::exp2_fast(d0)), __float_as_uint(pw::exp2_fast(d1)));
          s2 = pw::add_f32x2(s2, e);
          t2 = pw::fma_f32x2(e, pw::pack_f32x2(__float_as_uint(d0), __float_as_uint(d1)), t2);
        }
    }
    if (a.top) {
      const uint64_t key = v0 < v1 ? key_of(top, at) : 0;
      sh.segments[seg][tid] = key;
      best = key > best ? key : best;
    }
  }
  {
    float s0, s1, t0, t1;
    pw::unpack_f32x2(s2, s0, s1);
    pw::unpack_f32x2(t2, t0, t1);
    sum.s = s0 + s1;
    sum.t = t0 + t1;
  }
  if (kLong) sum = joined(sh.folded[tid], sum, p.scale_log2);
  sum = joined_lanes(sum, 32, p.scale_log2);
  if (lane == 0) sh.sums[warp] = sum;

  uint64_t list = 0;
  if (a.top) {
    if (tid == 0) sh.count = 0;
    list = join_lists(a.top == 1 ? largest_key(best) : sorted(best), kWarps, a.top, sh);
    if (warp == 0 && lane == a.top - 1) sh.bound = list;
    __syncthreads();
    const uint64_t last = sh.bound;     // 0: fewer threads than wanted values have any
    for (int i = 0; i < kSegments && i * length < steps; ++i) {
      const uint64_t key = sh.segments[i][tid];
      if (key && key >= last) sh.chosen[atomicAdd(&sh.count, 1)] = index_of(key);
    }
    __syncthreads();
    const int items = sh.count * length;
    // What ranks behind the last value of the bound's vector is not wanted.
    const uint64_t least = last ? (last & 0xFFFFFFFF00000000ull) | ~static_cast<uint32_t>(row.first_of(index_of(last)) + kSize - 1) : 1;
    list = 0;
    uint64_t want = least;              // a key below this one changes nothing
    for (int e0 = warp * 32; e0 < items; e0 += kThreads) {
      const int e = e0 + lane;
      uint32_t w[8];
      int first = 0;
      bool live = false;
      if (e < items) {
        const int place = sh.chosen[e / length] - begin, step = place / kThreads / length * length + e % length;
        const int v = begin + step * kThreads + place % kThreads;
        row.load(v, end, w);
        first = row.first_of(v);
        live = v < end && rank_of(Vec<T>::largest(w)) >= static_cast<uint32_t>(want >> 32);
      }
      if (!__any_sync(0xFFFFFFFFu, live)) continue;
#pragma unroll
      for (int i = 0; i < kSize; ++i) {
        float two[2];
        two_values<T>(w, i / 2, two[0], two[1]);
        const float x = two[i & 1];
        const int index = first + i;
        const uint64_t key = live && index >= 0 && index < row.size ? key_of(x, index) : 0;
        uint32_t found = __ballot_sync(0xFFFFFFFFu, key >= want);
        while (found) {
          const uint64_t next = __shfl_sync(0xFFFFFFFFu, key, __ffs(found) - 1);
          found &= found - 1;
          if (next < want) continue;
          const uint64_t up = __shfl_up_sync(0xFFFFFFFFu, list, 1);
          list = list > next ? list : lane == 0 || up > next ? next : up;
          const uint64_t kth = __shfl_sync(0xFFFFFFFFu, list, a.top - 1);
          want = kth >= least ? kth + 1 : least;
        }
      }
    }
    list = join_lists(list, kWarps, a.top, sh);
  } else {
    __syncthreads();
  }

  // the CTA's sums, then the cluster's
  sum = joined_lanes(sh.sums[lane % kWarps], kWarps, p.scale_log2);
  if (cluster > 1) {
    if (warp == 0) {
      sh.result[lane] = list;
      if (lane == 0) sh.total = sum;
    }
    pw::cluster_sync();
    if (rank == 0) {
      const uint64_t theirs = warp < cluster ? pw::ld_cluster_u64(pw::map_shared(pw::smem_u32(&sh.result[lane]), warp)) : 0;
      const float4 t = pw::ld_cluster_f4(pw::map_shared(pw::smem_u32(&sh.total), lane % cluster));
      sum = joined_lanes(Sums{t.x, t.y, t.z}, cluster, p.scale_log2);
      if (a.top) list = join_lists(theirs, cluster, a.top, sh);
    }
    pw::cluster_sync();                 // nobody leaves while its results are read
    if (rank != 0) return;
  }

  const float log_s = log2f(sum.s), base = base_of(sum.m);
  const bool empty = sum.m == -INFINITY && sum.s == 0.0f;   // nothing but -inf: no token has a probability
  // (not in powers of two: 1.44 times a masked logit, the lowest of its type, is infinite)
  auto logprob = [&](float x) { return empty ? -INFINITY : fmaf(x - base, a.scale, -log_s * kLn2); };
  if (tid == 0) {
    if (a.lse) a.lse[row_index] = empty ? -INFINITY : fmaf(base, a.scale, log_s * kLn2);
    if (a.entropy) a.entropy[row_index] = empty ? 0.0f : (log_s - sum.t / sum.s) * kLn2;
  }
  for (int i = tid; i < a.given; i += kThreads) {
    const int token = a.targets[row_index * a.targets_stride + i];
    float lp = token < 0 ? 0.0f : NAN;
    if (token >= 0 && token < row.size) {
      if constexpr (kSize == 8)
        lp = logprob(row.data[token]);
      else
        lp = logprob(pw::to_float(row.data[token]));
    }
    a.logprobs[row_index * a.logprobs_stride + i] = lp;
  }
  if (warp == 0 && lane < a.top) {
    a.top_ids[row_index * a.top_ids_stride + lane] = index_of(list);
    a.top_logprobs[row_index * a.top_logprobs_stride + lane] = logprob(ranked(static_cast<uint32_t>(list >> 32)));
  }
}

template <typename T, int kThreads, bool kLong>
int launch_threads(const LogprobParams& p, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.a.rows * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  PW_CUDA_TRY(cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kThreads, kLong>, p, cluster));
  return PW_OK;
}

template <typename T>
int launch(const LogprobParams& p, cudaStream_t s) {
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  const int vectors = (p.a.vocab + Vec<T>::kSize - 1) / Vec<T>::kSize;
  // Few rows: as many CTAs of a cluster as two an SM allow, with 4 vectors a thread
  // and more each.  One row of 131072 16-bit logits, 20 alternatives: 14.3, 11.6, 9.7 and 9.1 us
  // by 1, 2, 4 and 8 CTAs; of 32000: 8.2 and 8.7 by 1 and 2; 61 rows of 151937
  // 32-bit ones 25.9, 19.1, 16.2 and 17.5; 128 rows of 131072 18.4, 16.7 and 18.0.
  int cluster = 1;
  while (cluster < kMaxCluster && p.a.rows * 2 * cluster <= 2 * sms && vectors >= 2 * cluster * 1024) cluster *= 2;
  // Many short rows: CTAs of 128 threads, so that an SM has twice as many rows at
  // different stages (4096 rows of 32000: 59 us, 72 with 256 threads; of 8000: 30
  // and 53; but 4096 rows of 131072 with 20 alternatives 199 and 194; 512 rows of 32000
  // 16.8 and 16.2).
  if (p.a.rows > 4 * sms && vectors <= 4096) return launch_threads<T, 128, false>(p, cluster, s);
  // (a row may begin inside its first vector)
  if ((vectors + cluster) / cluster > kFold * 256) return launch_threads<T, 256, true>(p, cluster, s);
  return launch_threads<T, 256, false>(p, cluster, s);
}

}  // namespace

extern "C" int pw_token_logprobs(const pw_logprob_args* args, void* stream) {
  const char* op = "token_logprobs";
  if (!args) return pw::set_error(PW_ERR_INVALID_ARG, "%s: NULL argument", op);
  const pw_logprob_args& a = *args;
  if (!pw::is_16bit(a.dtype) && a.dtype != PW_DTYPE_F32) return pw::set_error(PW_ERR_UNSUPPORTED, "%s: dtype %d", op, a.dtype);
  if (a.rows < 0 || a.vocab < 1 || a.given < 0 || a.top < 0 || a.top > a.vocab)
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: bad sizes rows=%lld vocab=%d given=%d top=%d", op,
                         static_cast<long long>(a.rows), a.vocab, a.given, a.top);
  if (a.rows > (1 << 24) || a.vocab > (1 << 28) || a.top > kMaxTop)
    return pw::set_error(PW_ERR_UNSUPPORTED, "%s: rows=%lld (at most 2^24), vocab=%d (2^28), top=%d (%d)", op,
                         static_cast<long long>(a.rows), a.vocab, a.top, kMaxTop);
  if (!(a.scale > 0.0f) || !std::isfinite(a.scale * 1.4426950408889634f))   // in powers of two
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: scale %g", op, static_cast<double>(a.scale));
  if (a.stride < a.vocab || (a.given && (a.targets_stride < a.given || a.logprobs_stride < a.given)) ||
      (a.top && (a.top_ids_stride < a.top || a.top_logprobs_stride < a.top)))
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: a row stride is below its columns", op);
  if (a.rows == 0) return PW_OK;
  if (!a.logits || (a.given && (!a.targets || !a.logprobs)) || (a.top && (!a.top_ids || !a.top_logprobs)))
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: NULL argument", op);
  if (!a.given && !a.top && !a.lse && !a.entropy) return pw::set_error(PW_ERR_INVALID_ARG, "%s: no output", op);
  if (!pw::aligned(a.logits, a.dtype == PW_DTYPE_F32 ? 4 : 2))
    return pw::set_error(PW_ERR_INVALID_ARG, "%s: a pointer is not aligned to its values", op);
  for (const void* ptr : {static_cast<const void*>(a.targets), static_cast<const void*>(a.logprobs),
                          static_cast<const void*>(a.lse), static_cast<const void*>(a.entropy),
                          static_cast<const void*>(a.top_ids), static_cast<const void*>(a.top_logprobs)})
    if (!pw::aligned(ptr, 4)) return pw::set_error(PW_ERR_INVALID_ARG, "%s: a pointer is not aligned to its values", op);
  LogprobParams p{};
  p.a = a;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  cudaStream_t s = pw::as_stream(stream);
  if (a.dtype == PW_DTYPE_F16) return launch<__half>(p, s);
  return a.dtype == PW_DTYPE_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}
