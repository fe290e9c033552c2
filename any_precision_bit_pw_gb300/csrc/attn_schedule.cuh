// Division of a paged-attention call into equal shares of key blocks.
//
// A unit is one tile of query rows of one sequence for one key/value head; a
// row is a (token, query head) pair of that head's group.  A unit reads its
// visible keys in blocks of kBlock; the blocks of all units, head by head, form
// one line that the CTAs cut into equal stretches.  So a batch of ragged
// lengths and one long sequence both load every SM alike.  A unit that a cut
// crosses leaves a partial result (row maximum, sum and unnormalised output)
// with each CTA that worked on it; the last of them to arrive joins the pieces
// in the order of the CTAs, which does not depend on who is last.
#pragma once

#include "ops_common.cuh"

namespace pw_attn {

struct Params {
  pw_attn_args a;
  int group;          // query heads per key/value head
  uint32_t group_inv; // ceil(2^32 / group): rows up to group_max divide by a product
  int group_max;
  float scale_log2;   // scale * log2(e): the softmax runs in powers of two
  uint32_t* arrived;  // one counter per CTA, all 0 between calls
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

// Key range [lo, hi) that the rows of a tile see, and its blocks.
struct Range {
  int lo, hi, b0, b1;
};
template <int kTile, int kBlock>
__device__ __forceinline__ Range tile_range(const Params& p, const Sequence& s, int tile) {
  const int rows = s.q_len * p.group;
  const int first = tile * kTile, last = min(rows, first + kTile) - 1;
  const int base = s.kv_len - s.q_len;
  Range r;
  r.hi = p.a.causal ? max(0, base + token_of(p, last) + 1) : s.kv_len;
  r.lo = p.a.causal && p.a.window ? max(0, base + token_of(p, first) - p.a.window + 1) : 0;
  if (r.lo >= r.hi) r.lo = r.hi = 0;
  r.b0 = r.lo / kBlock;
  r.b1 = (r.hi + kBlock - 1) / kBlock;
  return r;
}
// A unit whose rows see nothing still takes one (empty) block: its zeros have
// to be written.
__device__ __forceinline__ int blocks_of(const Range& r) { return max(1, r.b1 - r.b0); }

template <int kTile>
__device__ __forceinline__ int tiles_of(const Params& p, const Sequence& s) {
  return (s.q_len * p.group + kTile - 1) / kTile;
}

template <int kTile, int kBlock>
__device__ __forceinline__ long long sequence_blocks(const Params& p, const Sequence& s) {
  const int tiles = tiles_of<kTile>(p, s);
  long long n = 0;
  for (int i = 0; i < tiles; ++i) n += blocks_of(tile_range<kTile, kBlock>(p, s, i));
  return n;
}

// Where a CTA is on the line.
struct Cursor {
  Sequence s;
  Range r;
  int head, seq, tile;
  int block;                // next block of the unit, 0 .. blocks_of(r) - 1
  long long pos, end;       // its position on the line, and the end of the CTA's stretch
  __device__ __forceinline__ bool done() const { return pos >= end; }
  // the unit's blocks on the line are [unit_begin, unit_end)
  __device__ __forceinline__ long long unit_begin() const { return pos - block; }
  __device__ __forceinline__ long long unit_end() const { return pos - block + blocks_of(r); }
};

// Moves to the first block of the next unit; pos is that block's already.
template <int kTile, int kBlock>
__device__ __forceinline__ void next_unit(const Params& p, Cursor& c) {
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
  c.r = tile_range<kTile, kBlock>(p, c.s, c.tile);
  c.block = 0;
}

// 64-bit quotient; short operands, the usual case, take a short division.
__device__ __forceinline__ long long quotient(long long n, long long d) {
  return (n | d) >> 31 ? n / d : static_cast<long long>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d));
}

// The line's cut: the first `extra` CTAs take q + 1 blocks, the others q.
struct Cut {
  long long q;
  int extra;
  __device__ __forceinline__ long long begin(int cta) const { return q * cta + min(cta, extra); }
  __device__ __forceinline__ int cta_of(long long w) const {
    const long long big = (q + 1) * extra;
    return static_cast<int>(w < big ? quotient(w, q + 1) : extra + quotient(w - big, q));
  }
};

// The cursor of CTA `cta` of `ctas`, found by the whole CTA (kThreads
// threads).  Returns false when it has no stretch: there are never more
// stretches than blocks.
template <int kTile, int kBlock, int kThreads>
__device__ __forceinline__ bool find_start(const Params& p, int cta, int ctas, Cursor& c, Cut& cut) {
  constexpr int kWarps = kThreads / 32;
  __shared__ long long warp_sum[2][kWarps];
  __shared__ long long sh_rest;
  __shared__ int sh_seq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // blocks of one head, and (batch <= kThreads) the prefix of this thread's sequence
  long long mine = 0;
  for (int b = tid; b < p.a.batch; b += kThreads)
    mine += sequence_blocks<kTile, kBlock>(p, sequence(p.a, b, cta == 0));
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
  const long long line = per_head * p.a.kv_heads;
  if (line < ctas) ctas = static_cast<int>(line);
  if (cta >= ctas) return false;   // the same for every thread
  cut.q = quotient(line, ctas);
  cut.extra = static_cast<int>(line - cut.q * ctas);
  c.pos = cut.begin(cta);
  c.end = cut.begin(cta + 1);
  c.head = static_cast<int>(quotient(c.pos, per_head));
  const long long want = c.pos - c.head * per_head;
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
      const long long n = b < p.a.batch ? sequence_blocks<kTile, kBlock>(p, sequence(p.a, b, false)) : 0;
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
  c.r = tile_range<kTile, kBlock>(p, c.s, 0);
  while (rest >= blocks_of(c.r)) {
    rest -= blocks_of(c.r);
    c.r = tile_range<kTile, kBlock>(p, c.s, ++c.tile);
  }
  c.block = static_cast<int>(rest);
  return true;
}

}  // namespace pw_attn
