// Division of a paged-attention call into equal shares of key blocks.
//
// A unit is one tile of query rows of one sequence for one key/value head; a
// row is a (token, query head) pair of that head's group.  A unit reads its
// visible keys in blocks of kBlock; the blocks of all units, head by head, form
// one line that the CTAs cut into equal stretches.  So a batch of ragged
// lengths and one long sequence both load every SM alike.  A unit that a cut
// crosses leaves a partial result (row maximum, sum and unnormalised output)
// with each CTA that worked on it; the last of them to arrive joins the pieces
// in the order of the CTAs, which does not depend on who is last.  Many pieces
// of many rows are joined in groups first, each by its last CTA.
//
// The grid is (CTAs, kv_heads) with each head's part of the line cut by itself,
// where the CTAs divide evenly among the heads and the longest stretch is no
// longer for it: fewer CTAs then have two units to finish (24 sequences of 17 to
// 65536 keys, one token each: 152 us, 164 cut as one line).  Otherwise it is
// (CTAs, 1).
//
// kSinks: calls whose tokens see the first keys of their sequence beside the
// window's.  A unit's blocks are then the window's, and after them those of the
// first keys, as far as they lie before the window's first block.  (The few keys
// of that last block seldom move the running maximum; in front, they set one that the
// window's keys move again: chunks of 2048 tokens with a window of 4096 and 1, 4 and
// 64 such keys take 387, 376 and 392 us, 425, 390 and 372 in front.  These are keys drawn
// alike.  Where the first ones' scores stand 5 to 10 above all others, they hold nearly every
// row's maximum and the last block moves it once more: 378, 382 and 375 us, against 376, 378 and 375
// of keys drawn alike in that run; in front was not timed there.)  The kernels are compiled
// apart, so that the other calls do not pay for the second range.
#pragma once

#include "ops_common.cuh"

namespace pw_attn {

struct Params {
  pw_attn_args a;
  int group;          // query heads per key/value head
  uint32_t group_inv; // ceil(2^32 / group): rows up to group_max divide by a product
  int group_max;
  float scale_log2;   // scale * log2(e): the softmax runs in powers of two
  int sinks;          // first keys that every token of a sequence sees; 0 without a window
  uint32_t* arrived;  // two counters per CTA, all 0 between calls
  float* part;        // 2 partial results per CTA
};

constexpr int kMaxCtas = 320;   // at most two CTAs on each of 160 SMs

__device__ __forceinline__ float inverse_sum(float l) { return l > 0.0f || l != l ? 1.0f / l : 0.0f; }
// Logarithm of the softmax's sum l * 2^m.
__device__ __forceinline__ float log_sum(float m, float l) {
  return l > 0.0f || l != l ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// The tcgen05 kernel (attention_tile.cu): whether it can take the call, the
// floats of one partial result, and the launch.
bool tile_kernel_takes(const Params& p);
size_t tile_part_floats(int head_dim);
int launch_tile_kernel(const Params& p, cudaStream_t s);

// Row number to token.
__device__ __forceinline__ int token_of(const Params& p, int row) {
  return row <= p.group_max ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.group_inv)) : row / p.group;
}

struct Sequence {
  int q0, q_len, kv_len;
};
// First key that any of the call's tokens sees: the pages before it may be gone.
__device__ __forceinline__ int first_key(const pw_attn_args& a, const Sequence& s) {
  return a.causal && a.window ? max(0, s.kv_len - s.q_len - a.window + 1) : 0;
}

// Lengths of sequence b; what the call's arrays cannot hold is reported and
// left out (a sequence without tokens, or keys past its page table).
__device__ __forceinline__ Sequence sequence(const pw_attn_args& a, int b, bool report) {
  Sequence s;
  s.q0 = a.q_offsets[b];
  s.q_len = a.q_offsets[b + 1] - s.q0;
  s.kv_len = a.kv_lens[b];
  if (s.q0 < 0 || s.q_len < 0 || s.q0 > a.tokens - s.q_len) {
    if (report) pw::report_status(a.status, PW_ERR_INVALID_ARG);
    s.q0 = s.q_len = 0;
  }
  const int64_t most = static_cast<int64_t>(a.pages_per_seq) * a.page_size;
  if (s.kv_len < 0 || s.kv_len > most) {
    if (report) pw::report_status(a.status, PW_ERR_INVALID_ARG);
    s.kv_len = s.kv_len < 0 ? 0 : static_cast<int>(most);
  }
  return s;
}

// Whether a key, not past the call's last token, is one that a row whose window starts at `lo` sees.
template <bool kSinks>
__device__ __forceinline__ bool in_sight(const Params& p, int key, int lo) {
  return key >= lo || (kSinks && key < p.sinks);
}

// Key range [lo, hi) that the rows of a tile see, and its blocks b0 .. b1-1;
// with first keys, the blocks 0 .. first-1 come after them.
template <bool kSinks>
struct Range {
  int lo, hi, b0, b1;
  __device__ __forceinline__ int blocks() const { return b1 - b0; }
  __device__ __forceinline__ int block_at(int i) const { return b0 + i; }
};
template <>
struct Range<true> {
  int lo, hi, b0, b1, first;
  __device__ __forceinline__ int blocks() const { return b1 - b0 + first; }
  __device__ __forceinline__ int block_at(int i) const { return i < b1 - b0 ? b0 + i : i - (b1 - b0); }
};
template <int kTile, int kBlock, bool kSinks>
__device__ __forceinline__ Range<kSinks> tile_range(const Params& p, const Sequence& s, int tile) {
  const int rows = s.q_len * p.group;
  const int first = tile * kTile, last = min(rows, first + kTile) - 1;
  const int base = s.kv_len - s.q_len;
  Range<kSinks> r;
  r.hi = p.a.causal ? max(0, base + token_of(p, last) + 1) : s.kv_len;
  r.lo = p.a.causal && p.a.window ? max(0, base + token_of(p, first) - p.a.window + 1) : 0;
  if (r.lo >= r.hi) r.lo = r.hi = 0;
  r.b0 = r.lo / kBlock;
  r.b1 = (r.hi + kBlock - 1) / kBlock;
  if constexpr (kSinks) r.first = min(r.b0, (p.sinks + kBlock - 1) / kBlock);
  return r;
}
// A unit whose rows see nothing still takes one (empty) block: its zeros have
// to be written.
template <bool kSinks>
__device__ __forceinline__ int blocks_of(const Range<kSinks>& r) {
  return max(1, r.blocks());
}

template <int kTile>
__device__ __forceinline__ int tiles_of(const Params& p, const Sequence& s) {
  return (s.q_len * p.group + kTile - 1) / kTile;
}

template <int kTile, int kBlock, bool kSinks>
__device__ __forceinline__ long long sequence_blocks(const Params& p, const Sequence& s) {
  const int tiles = tiles_of<kTile>(p, s);
  long long n = 0;
  for (int i = 0; i < tiles; ++i) n += blocks_of(tile_range<kTile, kBlock, kSinks>(p, s, i));
  return n;
}

// Where a CTA is on the line.
template <bool kSinks>
struct Cursor {
  Sequence s;
  Range<kSinks> r;
  int head, seq, tile;
  int block;                // next block of the unit, 0 .. blocks_of(r) - 1
  long long pos, end;       // its position on the line, and the end of the CTA's stretch
  __device__ __forceinline__ bool done() const { return pos >= end; }
  // the unit's blocks on the line are [unit_begin, unit_end)
  __device__ __forceinline__ long long unit_begin() const { return pos - block; }
  __device__ __forceinline__ long long unit_end() const { return pos - block + blocks_of(r); }
};

// Moves to the first block of the next unit; pos is that block's already.
template <int kTile, int kBlock, bool kSinks>
__device__ __forceinline__ void next_unit(const Params& p, Cursor<kSinks>& c) {
  ++c.tile;
  while (c.tile >= tiles_of<kTile>(p, c.s)) {
    c.tile = 0;
    if (++c.seq >= p.a.batch) {
      c.seq = 0;
      if (++c.head >= p.a.kv_heads) {   // only past the end of the line
        c.end = c.pos;
        return;
      }
    }
    c.s = sequence(p.a, c.seq, false);
  }
  c.r = tile_range<kTile, kBlock, kSinks>(p, c.s, c.tile);
  c.block = 0;
}

// 64-bit quotient; short operands, the usual case, take a short division.
__device__ __forceinline__ long long quotient(long long n, long long d) {
  return (n | d) >> 31 ? n / d : static_cast<long long>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d));
}

// The cut of a line, or of one head's part of it: every CTA takes `most`
// consecutive blocks, the last one what is left.
struct Cut {
  long long most;
  __device__ __forceinline__ int cta_of(long long w) const { return static_cast<int>(quotient(w, most)); }
};

// Grid of at most `ctas` CTAs, for at most `blocks` blocks per head.
inline dim3 grid_of(long long ctas, long long blocks, int kv_heads) {
  const bool by_head = ctas % kv_heads == 0;
  const long long n = by_head ? ctas / kv_heads : ctas, most = by_head ? blocks : blocks * kv_heads;
  return dim3(static_cast<unsigned>(n < most ? n : most < 1 ? 1 : most), by_head ? static_cast<unsigned>(kv_heads) : 1u);
}

// The cursor of this CTA, found by all its kThreads threads.  Returns false
// when it has no stretch.
template <int kTile, int kBlock, int kThreads, int kLeast, bool kSinks>
__device__ __forceinline__ bool find_start(const Params& p, Cursor<kSinks>& c, Cut& cut) {
  constexpr int kWarps = kThreads / 32;
  __shared__ long long warp_sum[2][kWarps];
  __shared__ long long sh_rest;
  __shared__ int sh_seq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // blocks of one head, and (batch <= kThreads) the prefix of this thread's sequence
  long long mine = 0;
  for (int b = tid; b < p.a.batch; b += kThreads)
    mine += sequence_blocks<kTile, kBlock, kSinks>(p, sequence(p.a, b, blockIdx.x + blockIdx.y == 0));
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sum[0][warp] = incl;
  __syncthreads();
  long long per_head = 0, base = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i == warp) base = per_head;
    per_head += warp_sum[0][i];
  }
  const bool by_head = gridDim.y > 1;
  const long long span = by_head ? per_head : per_head * p.a.kv_heads;
  cut.most = max(static_cast<long long>(kLeast), quotient(span + gridDim.x - 1, gridDim.x));
  c.pos = cut.most * blockIdx.x;
  if (c.pos >= span) return false;   // the same for every thread
  c.end = min(span, c.pos + cut.most);
  c.head = by_head ? static_cast<int>(blockIdx.y) : static_cast<int>(quotient(c.pos, per_head));
  const long long want = by_head ? c.pos : c.pos - c.head * per_head;
  // the sequence that holds position `want` of the head's blocks
  if (p.a.batch <= kThreads) {
    const long long lo = base + incl - mine;
    if (mine > 0 && lo <= want && want < lo + mine) {
      sh_seq = tid;
      sh_rest = want - lo;
    }
  } else {
    long long before = 0;
    for (int b0 = 0, turn = 1; b0 < p.a.batch; b0 += kThreads, turn ^= 1) {
      const int b = b0 + tid;
      const long long n = b < p.a.batch ? sequence_blocks<kTile, kBlock, kSinks>(p, sequence(p.a, b, false)) : 0;
      incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += u;
      }
      if (lane == 31) warp_sum[turn][warp] = incl;
      __syncthreads();   // two buffers in turn: the one written next was last read before this
      long long lo = before + incl - n;
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) lo += warp_sum[turn][i];
        before += warp_sum[turn][i];
      }
      if (n > 0 && lo <= want && want < lo + n) {
        sh_seq = b;
        sh_rest = want - lo;
      }
    }
  }
  __syncthreads();
  c.seq = sh_seq;
  c.s = sequence(p.a, c.seq, false);
  long long rest = sh_rest;
  c.tile = 0;
  c.r = tile_range<kTile, kBlock, kSinks>(p, c.s, 0);
  while (rest >= blocks_of(c.r)) {
    rest -= blocks_of(c.r);
    c.r = tile_range<kTile, kBlock, kSinks>(p, c.s, ++c.tile);
  }
  c.block = static_cast<int>(rest);
  return true;
}

// ---------------------------------------------------------------- joining the pieces of a unit
// A piece is kTile x D outputs, kTile maxima (in powers of two) and kTile sums;
// kColumnsInside: the outputs lie [row][D], otherwise [D / 4][row][4].
template <int kTile, int D, bool kColumnsInside>
__device__ __forceinline__ int piece_at(int row, int d) {
  return kColumnsInside ? row * D + d : (d * kTile / 4 + row) * 4;
}

// Whether this CTA is the last of `n` that come here; all its threads get the
// answer, and what the others wrote before they came is visible to them.
template <typename Sync>
__device__ __forceinline__ bool last_of(uint32_t* counter, int n, int& flag, Sync sync) {
  __threadfence();
  sync();
  if (threadIdx.x == 0) {
    const bool last = atomicAdd(counter, 1u) == static_cast<uint32_t>(n - 1);
    if (last) *counter = 0;
    flag = last;
    __threadfence();
  }
  sync();
  const bool last = flag;
  sync();
  return last;
}

// Adds `count` pieces in order; f(row, d, o, m, l) gets kColumns x 4 columns
// of every row at a time.  Maxima and sums come into shared memory in one round trip; then a
// thread has the loads of kColumns x 4 columns of kAtOnce pieces under way
// together.
template <int kTile, int D, bool kColumnsInside, int kThreads, int kColumns, int kAtOnce, typename Piece, typename Sync,
          typename F>
__device__ __forceinline__ void combine(int count, int rows, float2* state, Piece piece, Sync sync, F f) {
  const int tid = threadIdx.x;
  const int bits = rows > 1 ? 32 - __clz(rows - 1) : 0, mask = (1 << bits) - 1;   // rows, rounded up to a power of two
  const int step = kThreads >> bits;
  if ((tid & mask) < rows)
    for (int x0 = tid >> bits; x0 < count; x0 += 4 * step) {
      float2 t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = x0 + j * step;
        const float* src = piece(x < count ? x : x0) + kTile * D + (tid & mask);
        t[j] = make_float2(__ldcg(src), __ldcg(src + kTile));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (x0 + j * step < count) state[(x0 + j * step) * rows + (tid & mask)] = t[j];
    }
  sync();
  constexpr int kItems = D / (4 * kColumns);   // of a row
  const int items = kColumnsInside ? rows * kItems : kItems << bits;
  float top = -INFINITY, safe = 0.0f, sum = 0.0f;
#pragma unroll 1
  for (int e = tid; e < items; e += kThreads) {
    const int row = kColumnsInside ? e / kItems : e & mask;
    const int d = 4 * kColumns * (kColumnsInside ? e % kItems : e >> bits);
    if (row >= rows) continue;
    if (kColumnsInside || e == tid) {   // otherwise a thread keeps its row
      top = -INFINITY;
      sum = 0.0f;
      for (int x = 0; x < count; ++x) top = fmaxf(top, state[x * rows + row].x);
      safe = top == -INFINITY ? 0.0f : top;
      if (!kColumnsInside)
        for (int x = 0; x < count; ++x) sum += pw::exp2_fast(state[x * rows + row].x - safe) * state[x * rows + row].y;
    }
    float4 o[kColumns];
#pragma unroll
    for (int k = 0; k < kColumns; ++k) o[k] = make_float4(0, 0, 0, 0);
#pragma unroll 1
    for (int x = 0; x < count; x += kAtOnce) {
      float4 v[kAtOnce][kColumns];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
        for (int k = 0; k < kColumns; ++k)
          v[j][k] = x + j < count ? __ldcg(reinterpret_cast<const float4*>(
                                        piece(x + j) + piece_at<kTile, D, kColumnsInside>(row, d + 4 * k)))
                                  : make_float4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (x + j >= count) break;
        const float2 t = state[(x + j) * rows + row];
        const float w = pw::exp2_fast(t.x - safe);
        if (kColumnsInside) sum += w * t.y;
#pragma unroll
        for (int k = 0; k < kColumns; ++k) {
          o[k].x += w * v[j][k].x;
          o[k].y += w * v[j][k].y;
          o[k].z += w * v[j][k].z;
          o[k].w += w * v[j][k].w;
        }
      }
    }
    f(row, d, o, top, sum);
  }
  sync();   // the state is free again
}

// Number of pieces that are joined at a time.  Few, or of few rows: all, in one
// step; else about the square root of their number, so that both steps are
// alike.  A CTA adds 130 KB in about 1 us, as long as a second step takes to
// begin (64 tokens over 8192 keys, 16 pieces of 256 rows a head: 42 us in two
// steps, 54 in one; one token, 32 pieces of 4 rows: 16.8 and 18.8 in one and two).
constexpr int kPiecesAtOnce = 6, kRowsAtOnce = 256;
__device__ __forceinline__ int group_of(int pieces, int rows) {
  if (pieces <= kPiecesAtOnce || pieces * rows <= kRowsAtOnce) return pieces;
  int n = 3;
  while (n * n < pieces) ++n;
  return n;
}
// Entries of the shared state for tiles of `rows` rows on at most `ctas` CTAs.
constexpr int state_entries(int ctas, int rows) {
  int n = 4;
  while (n * n < ctas) ++n;
  return n * rows > kRowsAtOnce ? n * rows : kRowsAtOnce;
}

// This CTA has written its piece of the unit whose blocks are [begin, end).
// The last CTA of each group adds its pieces into the group's first, the last
// of those adds the groups; f as above.  (A CTA is the first of at most one cut
// unit, and of at most one group of two and more: the counters need no other
// index.)
template <int kTile, int D, bool kColumnsInside, int kThreads, int kColumns, int kAtOnce, typename Sync, typename F>
__device__ __forceinline__ void join(const Params& p, const Cut& cut, long long begin, long long end, int rows, float2* state,
                                     int& flag, Sync sync, F f) {
  constexpr size_t kFloats = static_cast<size_t>(kTile) * (D + 2);
  const int c0 = cut.cta_of(begin), n = cut.cta_of(end - 1) - c0 + 1;
  const int first = static_cast<int>(blockIdx.y * gridDim.x) + c0, first_slot = begin == cut.most * c0 ? 0 : 1;
  auto piece = [&](int x) { return p.part + (2 * static_cast<size_t>(first + x) + (x == 0 ? first_slot : 0)) * kFloats; };
  const int size = group_of(n, rows), groups = (n + size - 1) / size;
  const int lead = (static_cast<int>(blockIdx.x) - c0) / size * size, members = min(size, n - lead);
  if (members > 1 && !last_of(p.arrived + first + lead, members, flag, sync)) return;
  if (groups > 1) {
    if (members > 1) {
      float* sum = piece(lead);
      combine<kTile, D, kColumnsInside, kThreads, kColumns, kAtOnce>(
          members, rows, state, [&](int x) { return piece(lead + x); }, sync,
          [&](int row, int d, const float4* o, float m, float l) {
#pragma unroll
            for (int k = 0; k < kColumns; ++k)
              *reinterpret_cast<float4*>(sum + piece_at<kTile, D, kColumnsInside>(row, d + 4 * k)) = o[k];
            if (d == 0) {
              sum[kTile * D + row] = m;
              sum[kTile * D + kTile + row] = l;
            }
          });
    }
    if (!last_of(p.arrived + kMaxCtas + first, groups, flag, sync)) return;
  }
  const int step = groups > 1 ? size : 1;
  combine<kTile, D, kColumnsInside, kThreads, kColumns, kAtOnce>(
      groups > 1 ? groups : n, rows, state, [&](int x) { return piece(x * step); }, sync, f);
}

}  // namespace pw_attn
