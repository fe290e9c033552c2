// Rotary positions on queries and keys, and the append of keys and values to
// the paged cache.
//
// Pair i of a head, at position p, turns by the angle p * f_i:
//   (u, v) -> factor * (u cos - v sin, u sin + v cos)
// The table holds f_i as a fraction of a full turn in units of 2^-64, so
// p * f_i modulo one turn is one 64-bit integer product that wraps: the angle
// keeps its full precision at any position (in 32-bit floating point it would
// lose a digit with every factor of ten in p).
//
// Reads q, k and v once and writes as much: bound by memory bandwidth for
// prompts, by the chain offsets -> length -> page -> store for single tokens.
#include "ops_common.cuh"

namespace {

constexpr int kThreads = 256;

struct RopeParams {
  pw_rope_args a;
  int group_q, group_k;   // work units of one query head, and of one key head
  int groups_v;           // and of one value head
};

template <typename T, int kVec>
struct Vec;
template <typename T>
struct Vec<T, 8> {
  using type = uint4;
};
template <typename T>
struct Vec<T, 4> {
  using type = uint2;
};
template <typename T>
struct Vec<T, 1> {
  using type = uint16_t;
};

template <typename T, int kVec>
union Values {
  typename Vec<T, kVec>::type raw;
  T v[kVec];
  __device__ Values() {}
};

// Unit u of a rotated head: pair units first (two vectors of kVec values that
// hold kVec pairs), then units of kVec values that are copied.
template <typename T, int kVec>
__device__ __forceinline__ void rotate_unit(const T* src, T* dst, int u, int rotary, bool interleaved, float factor,
                                            const float2* cs) {
  using V = typename Vec<T, kVec>::type;
  const int pair_units = rotary / 2 / kVec;
  if (u >= pair_units) {
    const int at = rotary + (u - pair_units) * kVec;
    *reinterpret_cast<V*>(dst + at) = *reinterpret_cast<const V*>(src + at);
    return;
  }
  const int first = interleaved ? 2 * u * kVec : u * kVec;
  const int second = interleaved ? first + kVec : rotary / 2 + u * kVec;
  Values<T, kVec> x, y;
  x.raw = *reinterpret_cast<const V*>(src + first);
  y.raw = *reinterpret_cast<const V*>(src + second);
  if (interleaved && kVec > 1) {
#pragma unroll
    for (int i = 0; i + 1 < kVec; i += 2) {
      const float2 c0 = cs[u * kVec + i / 2], c1 = cs[u * kVec + (kVec + i) / 2];
      const float a0 = pw::to_float(x.v[i]), b0 = pw::to_float(x.v[i + 1]);
      const float a1 = pw::to_float(y.v[i]), b1 = pw::to_float(y.v[i + 1]);
      x.v[i] = pw::from_float<T>(a0 * c0.x - b0 * c0.y);
      x.v[i + 1] = pw::from_float<T>(a0 * c0.y + b0 * c0.x);
      y.v[i] = pw::from_float<T>(a1 * c1.x - b1 * c1.y);
      y.v[i + 1] = pw::from_float<T>(a1 * c1.y + b1 * c1.x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float2 c = cs[u * kVec + i];
      const float a = pw::to_float(x.v[i]), b = pw::to_float(y.v[i]);
      x.v[i] = pw::from_float<T>(a * c.x - b * c.y);
      y.v[i] = pw::from_float<T>(a * c.y + b * c.x);
    }
  }
  *reinterpret_cast<V*>(dst + first) = x.raw;
  *reinterpret_cast<V*>(dst + second) = y.raw;
}

// One CTA per token.
template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  using V = typename Vec<T, kVec>::type;
  extern __shared__ float2 cs[];
  __shared__ int below;
  const pw_rope_args& a = p.a;
  const int tid = threadIdx.x;
  const int t = blockIdx.x;
  // the token's sequence: how many sequences end at or before it
  if (tid == 0) below = 0;
  __syncthreads();
  int n = 0;
  for (int b = tid; b < a.batch; b += kThreads) n += a.q_offsets[b + 1] <= t;
  if (n) atomicAdd(&below, n);
  __syncthreads();
  const int seq = below;
  if (seq >= a.batch || a.q_offsets[seq] > t || a.q_offsets[seq] < 0) {
    if (tid == 0) pw::report_status(a.status, PW_ERR_INVALID_ARG);
    return;
  }
  const int slot = a.kv_lens[seq] - (a.q_offsets[seq + 1] - t);
  const int pos = a.positions ? a.positions[t] : slot;
  const int half = a.rotary_dim / 2;
  for (int i = tid; i < half; i += kThreads) {
    const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(a.turns[i]) * static_cast<uint64_t>(static_cast<int64_t>(pos)));
    float s, c;
    sincospif(static_cast<float>(turn) * 0x1p-63f, &s, &c);   // in half turns, -1 .. 1
    cs[i] = make_float2(c * a.factor, s * a.factor);
  }
  // the slot in the cache
  const T* k_src = nullptr;
  const T* v_src = nullptr;
  T* k_dst = nullptr;
  T* v_dst = nullptr;
  int kv_heads = 0;
  if (a.k) {
    const int index = slot >= 0 ? slot / a.page_size : -1;
    const int page = index >= 0 && index < a.pages_per_seq ? a.page_table[seq * a.page_table_stride + index] : -1;
    if (page < 0 || page >= a.num_pages) {
      if (tid == 0) pw::report_status(a.status, PW_ERR_NOT_RESIDENT);
    } else {
      const int64_t in_page = slot - index * a.page_size;
      kv_heads = a.kv_heads;
      k_src = static_cast<const T*>(a.k) + t * a.k_stride_token;
      v_src = static_cast<const T*>(a.v) + t * a.v_stride_token;
      k_dst = static_cast<T*>(a.k_cache) + page * a.k_cache_stride_page + in_page * a.k_cache_stride_token;
      v_dst = static_cast<T*>(a.v_cache) + page * a.v_cache_stride_page + in_page * a.v_cache_stride_token;
    }
  }
  __syncthreads();
  const int units_q = (a.q ? a.heads : 0) * p.group_q;
  const int units_k = kv_heads * p.group_k;
  const int units = units_q + units_k + kv_heads * p.groups_v;
  for (int w = tid; w < units; w += kThreads) {
    if (w < units_q) {
      const int h = w / p.group_q;
      rotate_unit<T, kVec>(static_cast<const T*>(a.q) + t * a.q_stride_token + h * a.q_stride_head,
                           static_cast<T*>(a.q_out) + t * a.q_out_stride_token + h * a.q_out_stride_head,
                           w - h * p.group_q, a.rotary_dim, a.interleaved, a.factor, cs);
    } else if (w < units_q + units_k) {
      const int h = (w - units_q) / p.group_k;
      rotate_unit<T, kVec>(k_src + h * a.k_stride_head, k_dst + h * a.k_cache_stride_head,
                           w - units_q - h * p.group_k, a.rotary_dim, a.interleaved, a.factor, cs);
    } else {
      const int r = w - units_q - units_k, h = r / p.groups_v, at = (r - h * p.groups_v) * kVec;
      *reinterpret_cast<V*>(v_dst + h * a.v_cache_stride_head + at) =
          *reinterpret_cast<const V*>(v_src + h * a.v_stride_head + at);
    }
  }
}

// Values in one access: 8 where every address and length is a multiple of 8
// values, else 4, else 1.
int vector_width(const pw_rope_args& a) {
  int64_t m = a.head_dim | (a.rotary_dim / 2);
  uintptr_t addr = 0;
  auto add = [&](const void* ptr, int64_t s0, int64_t s1, int64_t s2) {
    addr |= reinterpret_cast<uintptr_t>(ptr);
    m |= s0 | s1 | s2;
  };
  if (a.q) {
    add(a.q, a.q_stride_token, a.q_stride_head, 0);
    add(a.q_out, a.q_out_stride_token, a.q_out_stride_head, 0);
  }
  if (a.k) {
    add(a.k, a.k_stride_token, a.k_stride_head, 0);
    add(a.v, a.v_stride_token, a.v_stride_head, 0);
    add(a.k_cache, a.k_cache_stride_page, a.k_cache_stride_token, a.k_cache_stride_head);
    add(a.v_cache, a.v_cache_stride_page, a.v_cache_stride_token, a.v_cache_stride_head);
  }
  for (int v : {8, 4})
    if (m % v == 0 && addr % (2 * v) == 0) return v;
  return 1;
}

template <typename T, int kVec>
int launch(const pw_rope_args& a, cudaStream_t s) {
  RopeParams p{};
  p.a = a;
  p.group_q = p.group_k = a.rotary_dim / 2 / kVec + (a.head_dim - a.rotary_dim) / kVec;
  p.groups_v = a.head_dim / kVec;
  rope_kernel<T, kVec><<<static_cast<unsigned>(a.tokens), kThreads, sizeof(float2) * (a.rotary_dim / 2 + 1), s>>>(p);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

template <typename T>
int launch_width(const pw_rope_args& a, cudaStream_t s) {
  switch (vector_width(a)) {
    case 8: return launch<T, 8>(a, s);
    case 4: return launch<T, 4>(a, s);
    default: return launch<T, 1>(a, s);
  }
}

}  // namespace

extern "C" {

int pw_rope_turns(int rotary_dim, double base, const pw_rope_scaling* scaling, int64_t* h_turns, float* h_factor) {
  pw_rope_scaling s{};
  if (scaling) s = *scaling;
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 1024)
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_turns: rotary_dim %d", rotary_dim);
  if (!(base > 1.0) || !std::isfinite(base)) return pw::set_error(PW_ERR_INVALID_ARG, "rope_turns: base %g", base);
  if (!h_turns || !h_factor) return pw::set_error(PW_ERR_INVALID_ARG, "rope_turns: NULL output");
  if (s.kind < PW_ROPE_PLAIN || s.kind > PW_ROPE_BANDS)
    return pw::set_error(PW_ERR_UNSUPPORTED, "rope_turns: scaling kind %d", s.kind);
  if (s.kind != PW_ROPE_PLAIN && (!(s.scale >= 1.0) || !std::isfinite(s.scale)))
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_turns: scale %g", s.scale);
  if (s.kind == PW_ROPE_NTK && rotary_dim < 4)
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_turns: the base change needs rotary_dim >= 4");
  if ((s.kind == PW_ROPE_YARN || s.kind == PW_ROPE_BANDS) &&
      (!(s.original_positions > 0) || !(s.fast > s.slow) || !(s.slow > 0)))
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_turns: original_positions %g, fast %g, slow %g", s.original_positions,
                         s.fast, s.slow);
  const double two_pi = 6.283185307179586476925286766559;
  const double d = rotary_dim;
  if (s.kind == PW_ROPE_NTK) base *= std::pow(s.scale, d / (d - 2.0));
  // YARN: the pair that makes n turns over the original length
  auto pair_of = [&](double n) { return d * std::log(s.original_positions / (n * two_pi)) / (2.0 * std::log(base)); };
  double lo = 0, hi = 0;
  if (s.kind == PW_ROPE_YARN) {
    lo = std::fmax(std::floor(pair_of(s.fast)), 0.0);
    hi = std::fmin(std::ceil(pair_of(s.slow)), d - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / d);
    if (s.kind == PW_ROPE_LINEAR) f /= s.scale;
    if (s.kind == PW_ROPE_YARN) {
      const double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
      f = f / s.scale * ramp + f * (1.0 - ramp);
    }
    if (s.kind == PW_ROPE_BANDS) {
      const double turns = s.original_positions * f / two_pi;   // over the original length
      const double keep = std::fmin(std::fmax((turns - s.slow) / (s.fast - s.slow), 0.0), 1.0);
      f = f / s.scale * (1.0 - keep) + f * keep;
    }
    h_turns[i] = static_cast<int64_t>(std::llround(std::ldexp(f / two_pi, 64)));   // f <= 1: below 2^62
  }
  *h_factor = s.kind == PW_ROPE_YARN ? static_cast<float>(0.1 * std::log(s.scale) + 1.0) : 1.0f;
  return PW_OK;
}

int pw_rope_append(const pw_rope_args* args, void* stream) {
  if (!args) return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: NULL argument");
  const pw_rope_args& a = *args;
  if (!pw::is_16bit(a.dtype)) return pw::set_error(PW_ERR_UNSUPPORTED, "rope_append: dtype %d", a.dtype);
  if (a.tokens < 0 || a.batch < 0 || a.heads < 0 || a.kv_heads < 0 || a.head_dim < 1)
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: bad sizes tokens=%d batch=%d heads=%d kv_heads=%d head_dim=%d",
                         a.tokens, a.batch, a.heads, a.kv_heads, a.head_dim);
  if (a.rotary_dim < 0 || a.rotary_dim % 2 || a.rotary_dim > a.head_dim)
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: rotary_dim %d of head_dim %d", a.rotary_dim, a.head_dim);
  if (a.head_dim > 1024 || static_cast<int64_t>(a.heads + 2ll * a.kv_heads) * a.head_dim > (1 << 30))
    return pw::set_error(PW_ERR_UNSUPPORTED, "rope_append: head_dim %d", a.head_dim);
  if (!std::isfinite(a.factor)) return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: factor is not finite");
  if (!a.k != !a.v || !a.k != !a.k_cache || !a.k != !a.v_cache)
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: k, v and the two caches come together");
  if (!a.q != !a.q_out) return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: q and q_out come together");
  if (a.tokens == 0) return PW_OK;
  if (!a.q && !a.k) return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: neither q nor k");
  if (!a.q_offsets || !a.kv_lens || !a.status || (a.rotary_dim && !a.turns) || a.batch < 1)
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: NULL argument");
  if (a.k && (!a.page_table || a.page_size < 1 || a.num_pages < 1 || a.pages_per_seq < 1))
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: page_size %d, num_pages %d, pages_per_seq %d", a.page_size,
                         a.num_pages, a.pages_per_seq);
  if (a.k && a.page_table_stride < a.pages_per_seq)
    return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: page_table_stride");
  for (const void* ptr : {a.q, static_cast<const void*>(a.q_out), a.k, a.v, static_cast<const void*>(a.k_cache),
                          static_cast<const void*>(a.v_cache)})
    if (!pw::aligned(ptr, 2)) return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: misaligned pointer");
  cudaStream_t s = pw::as_stream(stream);
  return a.dtype == PW_DTYPE_F16 ? launch_width<__half>(a, s) : launch_width<__nv_bfloat16>(a, s);
}

}  // extern "C"
