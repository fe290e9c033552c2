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
// prompts (7.3k tokens of 48 + 8 + 8 heads: 40 us, 6.0 TB/s), by the chain
// offsets -> page -> store for single tokens (128 tokens: 3.6 us).  What it takes
// is little arithmetic on places per byte, and many CTAs, so that some wait for
// their tokens' places while others copy: 32 bytes an access and six CTAs an SM
// (with 16 bytes, two units a thread and five CTAs 52 us).
#include "ops_common.cuh"

namespace {

constexpr int kThreads = 256;
template <int kVec>
constexpr int kAhead = kVec == 16 ? 1 : 2;   // units of a thread under way together: 32 bytes
constexpr int kPerCta = 2;
constexpr int kMost = 8;     // tokens of a CTA

// Units of work: a rotated head is pair units, then units of kVec values that
// are copied; a value head is copied units.  A pair unit is one vector where
// pairs are neighbours, else two vectors rotary_dim/2 apart (or two neighbours,
// where an access is one value).
struct RopeParams {
  pw_rope_args a;
  int pair_units;      // of one query or key head
  int head_units;      // pair units and copied ones
  int value_units;     // of one value head
  int units_q, units_k, units;   // of a token: queries, keys, all
  uint32_t head_inv, value_inv, token_inv;   // ceil(2^32 / units): numbers below 2^16 divide by a product
  int per_cta;         // tokens of a CTA
};

template <int kVec>
struct Vec;
struct alignas(32) Words {
  uint32_t r[8];
};
template <>
struct Vec<16> {
  using type = Words;
};
template <>
struct Vec<8> {
  using type = uint4;
};
template <>
struct Vec<4> {
  using type = uint2;
};
template <>
struct Vec<1> {
  using type = uint16_t;
};

template <typename T, int kVec>
union Values {
  typename Vec<kVec>::type raw;
  T v[kVec];
  __device__ Values() {}
};

template <typename V>
__device__ __forceinline__ V load(const void* src) {
  return *static_cast<const V*>(src);
}
template <>
__device__ __forceinline__ Words load<Words>(const void* src) {
  Words w;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w.r[0]), "=r"(w.r[1]), "=r"(w.r[2]), "=r"(w.r[3]), "=r"(w.r[4]), "=r"(w.r[5]), "=r"(w.r[6]), "=r"(w.r[7])
               : "l"(src)
               : "memory");
  return w;
}
template <typename V>
__device__ __forceinline__ void store(void* dst, const V& v) {
  *static_cast<V*>(dst) = v;
}
template <>
__device__ __forceinline__ void store<Words>(void* dst, const Words& w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w.r[0]), "r"(w.r[1]), "r"(w.r[2]),
               "r"(w.r[3]), "r"(w.r[4]), "r"(w.r[5]), "r"(w.r[6]), "r"(w.r[7])
               : "memory");
}

__device__ __forceinline__ int quotient(int n, int d, uint32_t inv) {
  return inv ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), inv)) : n / d;
}

constexpr int kCopied = -1, kNear = -2;   // Unit::second of a copied unit, and of one whose pairs are neighbours

// One unit: what it is, and its values.
template <typename T, int kVec>
struct Unit {
  Values<T, kVec> x, y;
  int token;         // of the CTA's; -1: no unit
  int head;          // of its kind
  int first, second; // offsets of the vectors in the head, or kNear, kCopied
};

// Unit number w of the CTA's tokens, which start at t0 (a token's are those of
// its queries, then keys, then values): loads it.  kind 0, 1, 2: query, key, value.
template <typename T, int kVec>
__device__ __forceinline__ void load_unit(const RopeParams& p, int t0, int w, int total, Unit<T, kVec>& u, int& kind) {
  using V = typename Vec<kVec>::type;
  const pw_rope_args& a = p.a;
  u.token = -1;
  if (w >= total) return;
  u.token = quotient(w, p.units, p.token_inv);
  w -= u.token * p.units;
  const int64_t t = t0 + u.token;
  const T* src;
  if (w < p.units_q + p.units_k) {
    kind = w < p.units_q ? 0 : 1;
    if (kind) w -= p.units_q;
    u.head = quotient(w, p.head_units, p.head_inv);
    const int at = w - u.head * p.head_units;
    src = kind ? static_cast<const T*>(a.k) + t * a.k_stride_token + u.head * a.k_stride_head
               : static_cast<const T*>(a.q) + t * a.q_stride_token + u.head * a.q_stride_head;
    if (at < p.pair_units) {
      const bool near = a.interleaved && kVec > 1;
      u.first = a.interleaved && kVec == 1 ? 2 * at : at * kVec;
      u.second = near ? kNear : a.interleaved ? u.first + 1 : a.rotary_dim / 2 + u.first;
      if (!near) u.y.raw = load<V>(src + u.second);
    } else {
      u.first = a.rotary_dim + (at - p.pair_units) * kVec;
      u.second = kCopied;
    }
  } else {
    kind = 2;
    w -= p.units_q + p.units_k;
    u.head = quotient(w, p.value_units, p.value_inv);
    src = static_cast<const T*>(a.v) + t * a.v_stride_token + u.head * a.v_stride_head;
    u.first = (w - u.head * p.value_units) * kVec;
    u.second = kCopied;
  }
  u.x.raw = load<V>(src + u.first);
}

template <typename T, int kVec>
__device__ __forceinline__ void finish_unit(Unit<T, kVec>& u, T* dst, bool interleaved, const float2* cs) {
  using V = typename Vec<kVec>::type;
  if (kVec > 1 && u.second == kNear) {
#pragma unroll
    for (int i = 0; i + 1 < kVec; i += 2) {
      const float2 c = cs[u.first / 2 + i / 2];
      const float a = pw::to_float(u.x.v[i]), b = pw::to_float(u.x.v[i + 1]);
      u.x.v[i] = pw::from_float<T>(a * c.x - b * c.y);
      u.x.v[i + 1] = pw::from_float<T>(a * c.y + b * c.x);
    }
  } else if (u.second >= 0) {
    const float2* c = cs + (interleaved ? u.first / 2 : u.first);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float a = pw::to_float(u.x.v[i]), b = pw::to_float(u.y.v[i]);
      u.x.v[i] = pw::from_float<T>(a * c[i].x - b * c[i].y);
      u.y.v[i] = pw::from_float<T>(a * c[i].y + b * c[i].x);
    }
    store<V>(dst + u.second, u.y.raw);
  }
  store<V>(dst + u.first, u.x.raw);
}

// A CTA takes p.per_cta tokens.  Their first values are loaded at once: they
// depend on nothing, and the way to their place (sequence, length, page) takes
// two trips to memory.
template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, kVec == 16 ? 6 : 5) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 cs[];
  __shared__ int found[kMost], slots[kMost];
  __shared__ int64_t k_at[kMost], v_at[kMost];   // offsets in the caches; -1: no place
  const pw_rope_args& a = p.a;
  const int tid = threadIdx.x, half = a.rotary_dim / 2;
  const int t0 = blockIdx.x * p.per_cta, tokens = min(p.per_cta, a.tokens - t0), total = tokens * p.units;
  if (tid < kMost) found[tid] = -1;
  constexpr int kUnits = kAhead<kVec>;
  Unit<T, kVec> u[kUnits];
  int kind[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) load_unit<T, kVec>(p, t0, tid + i * kThreads, total, u[i], kind[i]);
  __syncthreads();
  // the tokens' sequences
  for (int b = tid; b < a.batch; b += kThreads) {
    const int lo = a.q_offsets[b], hi = a.q_offsets[b + 1], len = a.kv_lens[b];
    for (int t = max(lo, t0); t < min(hi, t0 + tokens); ++t) {
      found[t - t0] = b;
      slots[t - t0] = len - (hi - t);
    }
  }
  __syncthreads();
  // their places in the cache
  if (tid < tokens) {
    const int seq = found[tid], slot = slots[tid];
    int64_t k_off = -1, v_off = -1;
    if (seq < 0) {
      pw::report_status(a.status, PW_ERR_INVALID_ARG);
    } else if (a.k) {
      const int index = slot >= 0 ? slot / a.page_size : -1, in_page = slot - index * a.page_size;
      if (index < 0 || index >= a.pages_per_seq) {   // a length that the table cannot hold, or below the new tokens
        pw::report_status(a.status, PW_ERR_INVALID_ARG);
      } else {
        const int page = a.page_table[seq * a.page_table_stride + index];
        if (page < 0 || page >= a.num_pages) {
          pw::report_status(a.status, PW_ERR_NOT_RESIDENT);
        } else {
          k_off = page * a.k_cache_stride_page + in_page * a.k_cache_stride_token;
          v_off = page * a.v_cache_stride_page + in_page * a.v_cache_stride_token;
        }
      }
    }
    k_at[tid] = k_off;
    v_at[tid] = v_off;
  }
  for (int i = tid; i < tokens * half; i += kThreads) {
    const int token = i / half, pair = i - token * half;
    const int64_t pos = a.positions ? a.positions[t0 + token] : slots[token];
    const uint64_t turn = static_cast<uint64_t>(a.turns[pair]) * static_cast<uint64_t>(pos);
    float s, c;   // in half turns, -1 .. 1
    sincospif(static_cast<float>(static_cast<int64_t>(turn)) * 0x1p-63f, &s, &c);
    cs[i] = make_float2(c * a.factor, s * a.factor);
  }
  __syncthreads();
  for (int w0 = 0;;) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int token = u[i].token;
      if (token < 0 || found[token] < 0 || (kind[i] && k_at[token] < 0)) continue;
      T* dst = kind[i] == 0   ? static_cast<T*>(a.q_out) + static_cast<int64_t>(t0 + token) * a.q_out_stride_token +
                                  u[i].head * a.q_out_stride_head
               : kind[i] == 1 ? static_cast<T*>(a.k_cache) + k_at[token] + u[i].head * a.k_cache_stride_head
                              : static_cast<T*>(a.v_cache) + v_at[token] + u[i].head * a.v_cache_stride_head;
      finish_unit<T, kVec>(u[i], dst, a.interleaved, cs + token * half);
    }
    w0 += kUnits * kThreads;
    if (w0 >= total) break;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) load_unit<T, kVec>(p, t0, w0 + tid + i * kThreads, total, u[i], kind[i]);
  }
}

// Values in one access: 16 where every address and length is a multiple of 16
// values, else 8, 4 or 1.
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
  for (int v : {16, 8, 4})
    if (m % v == 0 && addr % (2 * v) == 0) return v;
  return 1;
}

template <typename T, int kVec>
int launch(const pw_rope_args& a, cudaStream_t s) {
  RopeParams p{};
  p.a = a;
  p.pair_units = a.interleaved && kVec > 1 ? a.rotary_dim / kVec : a.rotary_dim / 2 / kVec;
  p.head_units = p.pair_units + (a.head_dim - a.rotary_dim) / kVec;
  p.value_units = a.head_dim / kVec;
  p.units_q = a.q ? a.heads * p.head_units : 0;
  p.units_k = a.k ? a.kv_heads * p.head_units : 0;
  p.units = p.units_q + p.units_k + (a.k ? a.kv_heads * p.value_units : 0);
  if (p.units == 0) return PW_OK;   // no heads
  // one token a CTA while they do not fill the SMs, then kPerCta: the search for
  // the place is shared (with halves: 47 us with one, 43 with two, 44 with four)
  const int sms = pw::sm_count();
  p.per_cta = a.tokens > 8 * sms ? kPerCta : 1;
  const bool few = static_cast<int64_t>(p.units) * p.per_cta < (1 << 16);
  auto inverse = [&](int d) { return few && d > 1 ? static_cast<uint32_t>(((1ull << 32) + d - 1) / d) : 0u; };
  p.head_inv = inverse(p.head_units);
  p.value_inv = inverse(p.value_units);
  p.token_inv = inverse(p.units);
  rope_kernel<T, kVec><<<static_cast<unsigned>((a.tokens + p.per_cta - 1) / p.per_cta), kThreads,
                         sizeof(float2) * (p.per_cta * (a.rotary_dim / 2) + 1), s>>>(p);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

template <typename T>
int launch_width(const pw_rope_args& a, cudaStream_t s) {
  switch (vector_width(a)) {
    case 16: return launch<T, 16>(a, s);
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
  for (const void* ptr : {static_cast<const void*>(a.page_table), static_cast<const void*>(a.q_offsets),
                          static_cast<const void*>(a.kv_lens), static_cast<const void*>(a.positions),
                          static_cast<const void*>(a.status)})
    if (!pw::aligned(ptr, 4)) return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: misaligned table, lengths or status");
  if (!pw::aligned(a.turns, 8)) return pw::set_error(PW_ERR_INVALID_ARG, "rope_append: misaligned turns");
  cudaStream_t s = pw::as_stream(stream);
  return a.dtype == PW_DTYPE_F16 ? launch_width<__half>(a, s) : launch_width<__nv_bfloat16>(a, s);
}

}  // extern "C"
