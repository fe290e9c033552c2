// Attention of a chunk of new tokens over a paged key/value cache.
//
//   o = softmax(scale * q k^T + mask) v
// in one pass over the keys with the running maximum m and sum l of each row:
//   m' = max(m, max s),  l' = l 2^(m - m') + sum 2^(s - m'),  o' = o 2^(m - m') + 2^(s - m') v
//
// attn_stream_kernel (here): tiles of 16 rows, for few query rows per
// key/value head (single tokens, drafted tokens).  Each key and value is read
// once and feeds 16 rows of matrix work: memory bandwidth bounds it, and for
// short sequences the chain lengths -> page -> keys -> scores -> join.  A block
// is 64 keys: its four warps take 16 keys each with their own ring of copies
// and their own running maximum, so that nothing but the end of a unit makes
// them wait for each other; three stages of two 4 KB rows of keys and values
// keep 130 KB under way on an SM.  The scores' operand layout is the one that
// the second product wants its weights in, so the weights stay in registers.
// 64 sequences of 4096 keys, one token, 32 heads on 8: 168 us, 6.4 TB/s; 24
// sequences of 17 to 65536 keys, 48 heads on 8: 152 us, 6.3 TB/s; one of 131072
// keys: 91 us, 5.9 TB/s; one of 1021 keys: 9.4 us.  With a window of 4096 and the
// first 67 keys: 64 sequences of 17 to 32768 keys, 48 heads on 8, 101 us, 5.3 TB/s, and
// 168 us, 6.5 TB/s, where all have 8192 and more.
#include "attn_schedule.cuh"
#include "tc_ptx.cuh"

namespace {

using pw_attn::Cursor;
using pw_attn::Params;

constexpr int kTile = 16;            // query rows of a unit
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 16;           // keys of one warp's step
constexpr int kBlock = kChunk * kWarps;
constexpr int kStages = 3;           // chunks in flight per warp

template <int D>
constexpr int stage_bytes() { return 2 * kChunk * D * 2; }   // keys, then values
template <int D>
constexpr int smem_bytes() { return kWarps * kStages * stage_bytes<D>() + kWarps * 8 * D * 4; }
template <int D>
constexpr size_t part_floats() { return static_cast<size_t>(kTile) * (D + 2); }

// Starts the copies of one chunk (keys key0 .. key0+15 of the cursor's
// sequence): rows that the tile does not see are zeros and their pages are not looked up.
template <typename T, int D, bool kSinks>
__device__ __forceinline__ void load_chunk(const Params& p, const Cursor<kSinks>& c, int key0, uint32_t dst) {
  const pw_attn_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const int key = key0 + (lane & 15);
  long long off_k = -1, off_v = -1;
  if (pw_attn::in_sight<kSinks>(p, key, c.r.lo) && key < c.r.hi) {
    const int index = key / a.page_size;
    const int page = a.page_table[c.seq * a.page_table_stride + index];
    if (page >= 0 && page < a.num_pages) {
      const int in_page = key - index * a.page_size;
      off_k = page * a.k_stride_page + in_page * a.k_stride_token + c.head * a.k_stride_head;
      off_v = page * a.v_stride_page + in_page * a.v_stride_token + c.head * a.v_stride_head;
    } else {
      pw::report_status(a.status, PW_ERR_NOT_RESIDENT);
    }
  }
  constexpr int kUnits = D / 8;               // 16-byte units of a row
  constexpr int kRowsAtOnce = 32 / kUnits;
  const int unit = lane % kUnits;
#pragma unroll
  for (int i = 0; i < kChunk; i += kRowsAtOnce) {
    const int row = i + lane / kUnits;
    const long long ok = __shfl_sync(0xFFFFFFFFu, off_k, row), ov = __shfl_sync(0xFFFFFFFFu, off_v, row);
    const uint32_t at = dst + static_cast<uint32_t>(row * D * 2 + ((unit ^ (row & 7)) * 16));
    const uint32_t n = ok >= 0 ? 16 : 0;
    pw::cp_async_16_or_zero(at, static_cast<const T*>(a.k_cache) + (ok >= 0 ? ok : 0) + unit * 8, n);
    pw::cp_async_16_or_zero(at + kChunk * D * 2, static_cast<const T*>(a.v_cache) + (ov >= 0 ? ov : 0) + unit * 8, n);
  }
}

template <typename T, int D>
struct Rows {
  uint32_t q[D / 16][4];   // the tile's queries as matrix operands
  float o[D / 8][4];
  float m[2], l[2];        // of rows g and g + 8; l is this lane's share
};

template <typename T, int D, bool kSinks>
__device__ __forceinline__ void start_unit(const Params& p, const Cursor<kSinks>& c, Rows<T, D>& w) {
  const pw_attn_args& a = p.a;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rows = c.s.q_len * p.group;
  const T* q[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = c.tile * kTile + g + 8 * i;
    const int token = pw_attn::token_of(p, r), h = r - token * p.group;
    q[i] = r < rows ? static_cast<const T*>(a.q) + (c.s.q0 + token) * a.q_stride_token +
                          (c.head * p.group + h) * a.q_stride_head
                    : nullptr;
  }
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const T* row = q[i & 1];
      w.q[k][i] = row ? *reinterpret_cast<const uint32_t*>(row + 16 * k + 2 * t + (i >> 1) * 8) : 0u;
    }
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) w.o[i][j] = 0.0f;
  w.m[0] = w.m[1] = -INFINITY;
  w.l[0] = w.l[1] = 0.0f;
}

template <typename T, int D, bool kSinks>
__device__ __forceinline__ void compute_chunk(const Params& p, const Cursor<kSinks>& c, int key0, uint32_t src,
                                              Rows<T, D>& w) {
  const pw_attn_args& a = p.a;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, mat = lane >> 3, r8 = lane & 7;
  float s[2][4] = {};
  {
    const int row = (mat >> 1) * 8 + r8;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t b[4];
      pw::ldmatrix_x4(src + static_cast<uint32_t>(row * D * 2 + (((2 * k + (mat & 1)) ^ r8) * 16)), b);
      pw::mma_16816<T>(s[0], w.q[k], b[0], b[1]);
      pw::mma_16816<T>(s[1], w.q[k], b[2], b[3]);
    }
  }
  const int rows = c.s.q_len * p.group, base = c.s.kv_len - c.s.q_len;
  uint32_t pr[4];
  float keep[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // the row's visible keys are [lo, hi), and the first ones below hi
    const int r = c.tile * kTile + g + 8 * i;
    const int pos = base + pw_attn::token_of(p, r);
    int hi = a.causal ? min(pos + 1, c.r.hi) : c.r.hi;
    if (r >= rows) hi = 0;
    const int lo = a.causal && a.window ? pos - a.window + 1 : 0;
    float top = w.m[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = key0 + (j >> 1) * 8 + 2 * t + (j & 1);
      float& v = s[j >> 1][2 * i + (j & 1)];
      v = pw_attn::in_sight<kSinks>(p, key, lo) && key < hi ? v * p.scale_log2 : -INFINITY;
      top = fmaxf(top, v);
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const float safe = top == -INFINITY ? 0.0f : top;   // a row that has seen nothing yet
    keep[i] = pw::exp2_fast(w.m[i] - safe);
    w.m[i] = top;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float& v = s[j >> 1][2 * i + (j & 1)];
      v = pw::exp2_fast(v - safe);
      sum += v;
    }
    w.l[i] = w.l[i] * keep[i] + sum;
    // The weights are rounded to the values' type, which both operands of the instruction have: half a step each,
    // against one rounding of the result; their sum is not.
    pr[i] = pw::pack2<T>(s[0][2 * i], s[0][2 * i + 1]);
    pr[2 + i] = pw::pack2<T>(s[1][2 * i], s[1][2 * i + 1]);
  }
  const int row = (mat & 1) * 8 + r8;
#pragma unroll
  for (int n = 0; n < D / 16; ++n) {
    uint32_t b[4];
    pw::ldmatrix_x4_trans(src + static_cast<uint32_t>(kChunk * D * 2 + row * D * 2 + (((2 * n + (mat >> 1)) ^ r8) * 16)),
                          b);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float(&o)[4] = w.o[2 * n + j];
      o[0] *= keep[0];
      o[1] *= keep[0];
      o[2] *= keep[1];
      o[3] *= keep[1];
      pw::mma_16816<T>(o, pr, b[2 * j], b[2 * j + 1]);
    }
  }
}

struct Shared {
  float m[kWarps][kTile], l[kWarps][kTile];
  int last;
};

// End of a CTA's work on a unit: the warps' states are joined, and the rows
// are written, or left as a partial result whose last piece joins them all.
template <typename T, int D, bool kSinks>
__device__ __forceinline__ void finish_unit(const Params& p, const Cursor<kSinks>& c, long long begin, long long seg_begin,
                                            long long seg_end, const pw_attn::Cut& cut, Rows<T, D>& w, Shared& sh,
                                            float* buf) {
  const pw_attn_args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rows = min(kTile, c.s.q_len * p.group - c.tile * kTile);
  const long long unit_end = begin + pw_attn::blocks_of(c.r);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float l = w.l[i];
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
    if (t == 0) {
      sh.m[warp][g + 8 * i] = w.m[i];
      sh.l[warp][g + 8 * i] = l;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float top = -INFINITY;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) top = fmaxf(top, sh.m[x][g + 8 * i]);
    const float mine = pw::exp2_fast(w.m[i] - (top == -INFINITY ? 0.0f : top));
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      w.o[n][2 * i] *= mine;
      w.o[n][2 * i + 1] *= mine;
    }
  }
  // The warps' outputs are added through shared memory, eight rows at a time:
  // a thread owns four columns of a row.
  const bool whole = seg_begin == begin && seg_end == unit_end;
  constexpr size_t kFloats = part_floats<D>();
  constexpr int kRowItems = D / 4;
  // a piece: slot 0 of the CTA when it continues a unit or starts exactly at
  // its stretch's begin, slot 1 otherwise
  const bool at_start = seg_begin == cut.most * blockIdx.x;
  float* part = p.part + (2 * static_cast<size_t>(blockIdx.y * gridDim.x + blockIdx.x) + (at_start ? 0 : 1)) * kFloats;
  for (int r0 = 0; r0 < rows; r0 += 8) {
    const int i = r0 >> 3, live = min(8, rows - r0);
    if (g < live) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(buf + (warp * 8 + g) * D + 8 * n + 2 * t) =
            i ? make_float2(w.o[n][2], w.o[n][3]) : make_float2(w.o[n][0], w.o[n][1]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < live * kRowItems; e += kThreads) {
      const int row = e / kRowItems, d = (e % kRowItems) * 4;
      float4 o = *reinterpret_cast<const float4*>(buf + row * D + d);
#pragma unroll
      for (int x = 1; x < kWarps; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(buf + (x * 8 + row) * D + d);
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) top = fmaxf(top, sh.m[x][r0 + row]);
      const float safe = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) sum += sh.l[x][r0 + row] * pw::exp2_fast(sh.m[x][r0 + row] - safe);
      if (whole) {
        const int r = c.tile * kTile + r0 + row, t0 = pw_attn::token_of(p, r), token = c.s.q0 + t0;
        const int h = c.head * p.group + r - t0 * p.group;
        const float inv = pw_attn::inverse_sum(sum);
        T* out = static_cast<T*>(a.out) + token * a.out_stride_token + h * a.out_stride_head + d;
        *reinterpret_cast<uint2*>(out) = make_uint2(pw::pack2<T>(o.x * inv, o.y * inv), pw::pack2<T>(o.z * inv, o.w * inv));
        if (a.lse && d == 0) a.lse[static_cast<int64_t>(token) * a.heads + h] = pw_attn::log_sum(top, sum);
      } else {
        *reinterpret_cast<float4*>(part + (r0 + row) * D + d) = o;
        if (d == 0) {
          part[kTile * D + r0 + row] = top;
          part[kTile * D + kTile + r0 + row] = sum;
        }
      }
    }
    __syncthreads();
  }
  if (whole) return;
  static_assert(pw_attn::state_entries(pw_attn::kMaxCtas, kTile) * sizeof(float2) <= kWarps * 8 * D * 4, "state");
  pw_attn::join<kTile, D, true, kThreads, 1, 8>(
      p, cut, begin, unit_end, rows, reinterpret_cast<float2*>(buf), sh.last, [] { __syncthreads(); },
      [&](int row, int d, const float4* o, float top, float sum) {
        const int r = c.tile * kTile + row, t0 = pw_attn::token_of(p, r), token = c.s.q0 + t0;
        const int h = c.head * p.group + r - t0 * p.group;
        const float inv = pw_attn::inverse_sum(sum);
        T* out = static_cast<T*>(a.out) + token * a.out_stride_token + h * a.out_stride_head + d;
        *reinterpret_cast<uint2*>(out) = make_uint2(pw::pack2<T>(o->x * inv, o->y * inv), pw::pack2<T>(o->z * inv, o->w * inv));
        if (a.lse && d == 0) a.lse[static_cast<int64_t>(token) * a.heads + h] = pw_attn::log_sum(top, sum);
      });
}

template <typename T, int D, bool kSinks>
__global__ void __launch_bounds__(kThreads) attn_stream_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5;
  const uint32_t ring = pw::smem_u32(smem) + static_cast<uint32_t>(warp * kStages * stage_bytes<D>());
  float* buf = reinterpret_cast<float*>(smem + kWarps * kStages * stage_bytes<D>());
  Cursor<kSinks> c;
  pw_attn::Cut cut;
  if (!pw_attn::find_start<kTile, kBlock, kThreads, 1>(p, c, cut)) return;
  Cursor<kSinks> ahead = c;   // the copies run kStages - 1 blocks ahead of the arithmetic
  int fill = 0;
  auto load_next = [&]() {
    if (!ahead.done()) {
      load_chunk<T, D>(p, ahead, ahead.r.block_at(ahead.block) * kBlock + warp * kChunk,
                       ring + static_cast<uint32_t>(fill * stage_bytes<D>()));
      ++ahead.pos;
      if (++ahead.block >= pw_attn::blocks_of(ahead.r) && !ahead.done()) pw_attn::next_unit<kTile, kBlock>(p, ahead);
    }
    fill = fill + 1 == kStages ? 0 : fill + 1;
    pw::cp_async_commit();
  };
  for (int i = 0; i < kStages - 1; ++i) load_next();
  Rows<T, D> w;
  start_unit<T, D>(p, c, w);
  long long seg_begin = c.pos;
  int use = 0;
  while (!c.done()) {
    pw::cp_async_wait<kStages - 2>();
    __syncwarp();
    load_next();   // into the stage that the last step has left
    compute_chunk<T, D>(p, c, c.r.block_at(c.block) * kBlock + warp * kChunk,
                        ring + static_cast<uint32_t>(use * stage_bytes<D>()), w);
    __syncwarp();
    use = use + 1 == kStages ? 0 : use + 1;
    const long long begin = c.unit_begin();
    ++c.pos;
    ++c.block;
    const bool unit_done = c.block >= pw_attn::blocks_of(c.r);
    if (unit_done || c.done()) {
      finish_unit<T, D>(p, c, begin, seg_begin, c.pos, cut, w, sh, buf);
      if (!c.done()) {
        pw_attn::next_unit<kTile, kBlock>(p, c);
        start_unit<T, D>(p, c, w);
        seg_begin = c.pos;
      }
    }
  }
  pw::cp_async_wait<0>();
}

template <typename T, int D, bool kSinks>
int launch_stream(const Params& p, cudaStream_t s) {
  constexpr int kDevs = 64;
  static bool attr_done[kDevs] = {};
  int dev = 0;
  PW_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= kDevs || !attr_done[dev]) {
    PW_CUDA_TRY(cudaFuncSetAttribute(attn_stream_kernel<T, D, kSinks>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D>()));
    if (dev < kDevs) attr_done[dev] = true;
  }
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  // two CTAs an SM, but no more than there are blocks to share out
  const long long tiles = (static_cast<long long>(p.a.tokens) * p.group + kTile - 1) / kTile + p.a.batch;
  const long long blocks = tiles * ((p.a.max_kv_len + kBlock - 1) / kBlock + 1);
  const dim3 grid = pw_attn::grid_of(2ll * sms < pw_attn::kMaxCtas ? 2ll * sms : pw_attn::kMaxCtas, blocks, p.a.kv_heads);
  attn_stream_kernel<T, D, kSinks><<<grid, kThreads, smem_bytes<D>(), s>>>(p);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

template <typename T>
int launch(const Params& p, cudaStream_t s) {
  if (pw_attn::tile_kernel_takes(p)) return pw_attn::launch_tile_kernel(p, s);
  if (p.sinks) return p.a.head_dim == 64 ? launch_stream<T, 64, true>(p, s) : launch_stream<T, 128, true>(p, s);
  return p.a.head_dim == 64 ? launch_stream<T, 64, false>(p, s) : launch_stream<T, 128, false>(p, s);
}

constexpr size_t kCounterBytes = 4096;   // the counters, rounded up
static_assert(kCounterBytes >= 2 * 4 * pw_attn::kMaxCtas, "counters");

bool head_dim_ok(int d) { return d == 64 || d == 128; }

}  // namespace

extern "C" {

size_t pw_paged_attention_workspace(int tokens, int batch, int heads, int kv_heads, int head_dim) {
  if (tokens < 0 || batch < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || !head_dim_ok(head_dim)) return 0;
  const size_t stream = 2 * pw_attn::kMaxCtas * static_cast<size_t>(kTile) * (head_dim + 2);
  const size_t tile = pw_attn::kMaxCtas * pw_attn::tile_part_floats(head_dim);   // one CTA an SM
  return kCounterBytes + sizeof(float) * (stream > tile ? stream : tile);
}

int pw_paged_attention(const pw_attn_args* args, void* d_ws, size_t ws_bytes, void* stream) {
  return pw_paged_attention_ex(args, nullptr, d_ws, ws_bytes, stream);
}

int pw_paged_attention_ex(const pw_attn_args* args, const pw_attn_options* options, void* d_ws, size_t ws_bytes, void* stream) {
  if (!args) return pw::set_error(PW_ERR_INVALID_ARG, "paged_attention: NULL argument");
  const pw_attn_args& a = *args;
  if (!pw::is_16bit(a.dtype)) return pw::set_error(PW_ERR_UNSUPPORTED, "paged_attention: dtype %d", a.dtype);
  if (a.tokens < 0 || a.batch < 0 || a.heads < 1 || a.kv_heads < 1 || a.heads % a.kv_heads || a.max_q_len < 0 ||
      a.max_kv_len < 0)
    return pw::set_error(PW_ERR_INVALID_ARG,
                         "paged_attention: bad sizes tokens=%d batch=%d heads=%d kv_heads=%d max_q_len=%d max_kv_len=%d",
                         a.tokens, a.batch, a.heads, a.kv_heads, a.max_q_len, a.max_kv_len);
  if (!head_dim_ok(a.head_dim))
    return pw::set_error(PW_ERR_UNSUPPORTED, "paged_attention: head_dim %d (64 or 128)", a.head_dim);
  if (static_cast<long long>(a.tokens) * a.heads > (1ll << 30) || a.batch > (1 << 20))
    return pw::set_error(PW_ERR_UNSUPPORTED, "paged_attention: problem too large");
  if (a.window < 0 || a.window > (1 << 30) || (a.window && !a.causal))
    return pw::set_error(PW_ERR_INVALID_ARG, "paged_attention: window %d (needs causal)", a.window);
  const int sinks = options ? options->sinks : 0;
  if (sinks < 0 || sinks > (1 << 30)) return pw::set_error(PW_ERR_INVALID_ARG, "paged_attention: %d first keys", sinks);
  if (options)
    for (int32_t r : options->reserved)
      if (r) return pw::set_error(PW_ERR_INVALID_ARG, "paged_attention: a reserved option is set");
  if (!std::isfinite(a.scale)) return pw::set_error(PW_ERR_INVALID_ARG, "paged_attention: scale is not finite");
  if (a.tokens == 0 || a.batch == 0) return PW_OK;
  if (a.page_size < 1 || a.num_pages < 1 || a.pages_per_seq < 1 || a.page_table_stride < a.pages_per_seq)
    return pw::set_error(PW_ERR_INVALID_ARG, "paged_attention: page_size %d, num_pages %d, pages_per_seq %d", a.page_size,
                         a.num_pages, a.pages_per_seq);
  if (static_cast<long long>(a.page_size) * a.pages_per_seq > (1ll << 30))
    return pw::set_error(PW_ERR_UNSUPPORTED, "paged_attention: sequences of more than 2^30 keys");
  if (!a.q || !a.out || !a.k_cache || !a.v_cache || !a.page_table || !a.q_offsets || !a.kv_lens || !a.status || !d_ws)
    return pw::set_error(PW_ERR_INVALID_ARG, "paged_attention: NULL argument");
  int64_t strides = a.q_stride_token | a.q_stride_head | a.out_stride_token | a.out_stride_head | a.k_stride_page |
                    a.k_stride_token | a.k_stride_head | a.v_stride_page | a.v_stride_token | a.v_stride_head;
  if (strides % 8 || !pw::aligned(a.q, 16) || !pw::aligned(a.out, 16) || !pw::aligned(a.k_cache, 16) ||
      !pw::aligned(a.v_cache, 16))
    return pw::set_error(PW_ERR_INVALID_ARG, "paged_attention: every head's row must be 16-byte aligned");
  for (const void* ptr : {static_cast<const void*>(a.page_table), static_cast<const void*>(a.q_offsets),
                          static_cast<const void*>(a.kv_lens), static_cast<const void*>(a.lse),
                          static_cast<const void*>(a.status)})
    if (!pw::aligned(ptr, 4))
      return pw::set_error(PW_ERR_INVALID_ARG, "paged_attention: misaligned table, lengths, lse or status");
  const size_t need = pw_paged_attention_workspace(a.tokens, a.batch, a.heads, a.kv_heads, a.head_dim);
  if (ws_bytes < need || !pw::aligned(d_ws, 256))
    return pw::set_error(PW_ERR_WORKSPACE, "paged_attention: workspace needs %zu bytes, 256-byte aligned (got %zu)", need,
                         ws_bytes);
  Params p{};
  p.a = a;
  // no sequence is longer than its table; a bound of 2^31 - 1 ("any") would wrap where it is rounded up to blocks
  const int holds = a.page_size * a.pages_per_seq;
  if (p.a.max_kv_len > holds) p.a.max_kv_len = holds;
  p.group = a.heads / a.kv_heads;
  // n * group_inv / 2^32 is exact while n times the excess of group_inv stays below 2^32 / group
  p.group_inv = static_cast<uint32_t>(((1ull << 32) + p.group - 1) / p.group);
  p.group_max = p.group > 1 ? static_cast<int>(((1ull << 31) - 1) / p.group) : -1;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.sinks = a.window ? sinks : 0;   // without a window every token sees them anyway
  p.arrived = static_cast<uint32_t*>(d_ws);
  p.part = reinterpret_cast<float*>(static_cast<char*>(d_ws) + kCounterBytes);
  cudaStream_t s = pw::as_stream(stream);
  return a.dtype == PW_DTYPE_F16 ? launch<__half>(p, s) : launch<__nv_bfloat16>(p, s);
}

}  // extern "C"
