// Attention of a chunk of new tokens over a paged cache, for many query rows
// per key/value head: tcgen05 matrix instructions on tiles of 2 x 128 rows by
// 128 keys (attention.cu holds the formulas and the kernel for few rows).
//
// The two halves of a tile take turns: while the tensor cores multiply one
// half's weights with the values and its queries with the next keys, four
// warps turn the other half's scores into weights.  A thread owns one row, so
// maximum and sum need no exchange.  Scores S and outputs O live in Tensor
// Memory; the weights P overwrite S in 16 bits and feed the second product
// from there.
//
// The running maximum moves only when a row's new maximum exceeds it by 2^8
// (by 2^15 inside a block): until then the weights stay in the 16-bit range and
// need no common factor, so the output is rescaled a few times per row instead
// of at every block.
//
// Keys and values arrive by TMA, a box per page piece, into 128-byte swizzled
// rows.  Values outside the visible keys are zeros in shared memory (a weight
// of 0 does not hide a NaN).
//
// A block is 2 x 2 products of 128 x 128 x 128, 2048 cycles of the tensor pipe
// if nothing holds it up; it takes about 2630.  The first product reads both
// operands from shared memory at its full rate while the copies of the next
// block write to it, and the softmax of a half (128 exponentials a row) has to
// fit under the other half's products.  256 rows a tile are what one SM's
// Tensor Memory holds (two S and two O of 128 columns each), and they halve the
// key reads of a 128-row tile.  Four chunks of 1500 to 2048 tokens over 4096 to
// 16384 keys, 32 heads on 8: 1131 us, 1.31 PFLOP/s, at the clocks that the
// power limit leaves (about 1.6 GHz).
#include <numeric>

#include "attn_schedule.cuh"
#include "umma.cuh"

namespace {

using pw_attn::Cursor;
using pw_attn::Params;

constexpr int kHalf = 128;             // rows of half a tile: the lanes of Tensor Memory
constexpr int kTile = 2 * kHalf;
constexpr int kBlock = 128;            // keys of a block
constexpr int kKeySlots = 2, kValueSlots = 3;   // rings of key and value blocks in shared memory
// A piece of a tile costs its join as much as a block of keys costs the matrix
// units: no CTA takes fewer blocks (64 tokens over 1000 keys: 23 us, 29 with 1).
constexpr int kLeast = 3;
constexpr int kSoftmaxWarps = 8;
constexpr int kKeyWarp = 8, kValueWarp = 9, kMmaWarp = 10;
constexpr int kThreads = 384;
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr float kLazy = 8.0f;          // log2 of what a weight may grow to, from block to block
constexpr float kLazyInside = 15.0f;   // and inside a block
constexpr int kHalfRow = kBlock * 128; // bytes of 64 values of 128 rows

template <int D>
constexpr int tile_bytes() { return (D / 64) * kHalfRow; }
template <int D>
constexpr int smem_bytes() { return (2 + kKeySlots + kValueSlots) * tile_bytes<D>() + 1024; }

struct alignas(8) Shared {
  uint64_t q_full[2], k_full[kKeySlots], k_empty[kKeySlots], v_full[kValueSlots], v_empty[kValueSlots];
  uint64_t drained, s_full[2], p_full[2][2], o_half[2], o_done[2];   // p_full: weights of the first and the last 64 keys
  uint32_t tmem;
  int dead;
  int last;
};

struct Maps {
  CUtensorMap k, v;
  int box;   // rows of a box: a divisor of the page size and of a block
};

__device__ __forceinline__ bool wait(const uint64_t& bar, uint32_t parity, Shared& sh, const Params& p) {
  return pw::warp_wait(&bar, parity, &sh.dead, p.a.status);
}
__device__ __forceinline__ uint32_t bar(const uint64_t& b) { return pw::smem_u32(&b); }

// Number of 128-row halves with rows.
template <bool kSinks>
__device__ __forceinline__ int halves_of(const Params& p, const Cursor<kSinks>& c) {
  return pw::uniform(c.s.q_len * p.group - c.tile * kTile > kHalf ? 2 : 1);
}

// Walks the units of the CTA's stretch: f(cursor, first block, end block) with
// block numbers of the unit.
template <bool kSinks, typename F>
__device__ __forceinline__ void for_units(const Params& p, Cursor<kSinks> c, F f) {
  while (pw::uniform(!c.done())) {
    const int b0 = pw::uniform(c.block), n = pw_attn::blocks_of(c.r);
    const long long room = c.end - c.pos;
    const int b1 = pw::uniform(room < n - b0 ? b0 + static_cast<int>(room) : n);
    if (!f(c, b0, b1)) return;
    c.pos += b1 - b0;
    c.block = b1;
    if (!c.done()) pw_attn::next_unit<kTile, kBlock>(p, c);
  }
}

// ---------------------------------------------------------------- copies (a warp for keys, a warp for values)
// Rows of values that no token of the call sees have to be zero: past the
// sequence's end, and before every window, after the first keys.  They occur in the
// blocks at those places only: there the boxes that hold such rows are copied row by
// row, with zeros for the others.
template <int D, bool kSinks>
__device__ __forceinline__ void copy_rows(const Params& p, const Cursor<kSinks>& c, int key0, int first, int rows, int page,
                                          int begin, unsigned char* dst) {
  const pw_attn_args& a = p.a;
  constexpr int kUnits = D / 8, kAtOnce = 8;   // (the loads of a turn before its stores: one latency a turn)
  const int lane = threadIdx.x & 31;
  for (int i0 = lane; i0 < rows * kUnits; i0 += 32 * kAtOnce) {
    uint4 v[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int i = i0 + 32 * j, row = first + i / kUnits, unit = i % kUnits, key = key0 + row;
      v[j] = make_uint4(0, 0, 0, 0);
      if (i < rows * kUnits && page >= 0 && pw_attn::in_sight<kSinks>(p, key, begin) && key < c.s.kv_len)
        v[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v_cache) + page * a.v_stride_page +
                                               (key % a.page_size) * a.v_stride_token + c.head * a.v_stride_head + unit * 8);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int i = i0 + 32 * j, row = first + i / kUnits, unit = i % kUnits;
      if (i < rows * kUnits)
        *reinterpret_cast<uint4*>(dst + (unit >> 3) * kHalfRow + row * 128 + (((unit & 7) ^ (row & 7)) << 4)) = v[j];
    }
  }
}

template <int D, bool kValues, bool kSinks>
__device__ __forceinline__ void load_role(const Params& p, const Cursor<kSinks>& start, const Maps& maps, Shared& sh,
                                          unsigned char* ring) {
  const pw_attn_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const int box = maps.box, boxes = kBlock / box;   // at most 16 boxes of 64 values
  const uint32_t every = (1u << boxes) - 1u;
  const int step_pages = kBlock / a.page_size, step_rows = kBlock % a.page_size;
  uint64_t* const fulls = kValues ? sh.v_full : sh.k_full;
  uint64_t* const empties = kValues ? sh.v_empty : sh.k_empty;
  constexpr uint32_t kSlots = kValues ? kValueSlots : kKeySlots;
  pw::Ring<kSlots> slot;
  uint32_t x = 0;                                   // blocks started
  for_units(p, start, [&](const Cursor<kSinks>& c, int b0, int b1) {
    const int32_t* table = a.page_table + c.seq * a.page_table_stride;
    // this lane's box: its first key, and where that is in the page table
    int key0 = c.r.block_at(b0) * kBlock, key = key0 + lane * box;
    int index = key / a.page_size, in_page = key - index * a.page_size;
    const int begin = pw_attn::first_key(a, c.s), end = c.s.kv_len;
    auto wanted = [&]() { return lane < boxes && key < end && (key + box > begin || (kSinks && key < p.sinks)); };
    int page = wanted() ? table[index] : -1;
    for (int b = b0; b < b1; ++b, ++x) {
      const bool want = wanted();
      const int this_page = page, row = in_page;
      bool take = want && this_page >= 0 && this_page < a.num_pages;
      if (want && !take && !kValues) pw::report_status(a.status, PW_ERR_NOT_RESIDENT);
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, take);
      // every row is visible to some token
      if (kValues) take = take && (key >= begin || (kSinks && key + box <= p.sinks)) && key + box <= end;
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, take);
      // the next block's page: its latency passes during this block's waits
      key += kBlock;
      index += step_pages;
      in_page += step_rows;
      if (in_page >= a.page_size) {
        in_page -= a.page_size;
        ++index;
      }
      const bool back = kSinks && b + 1 == c.r.b1 - c.r.b0;   // from the window to the first keys
      if (back) {
        key = lane * box;
        index = key / a.page_size;
        in_page = key - index * a.page_size;
      }
      page = b + 1 < b1 && wanted() ? table[index] : -1;
      if (x >= kSlots && !wait(empties[slot.at], slot.parity ^ 1u, sh, p)) return false;
      const uint32_t full = bar(fulls[slot.at]);
      unsigned char* dst = ring + slot.at * tile_bytes<D>();
      slot.next();
      if (kValues && mask != every) {
        for (int i = 0; i < boxes; ++i)
          if (!(mask >> i & 1u))
            copy_rows<D>(p, c, key0, i * box, box, __shfl_sync(0xFFFFFFFFu, live >> lane & 1u ? this_page : -1, i), begin, dst);
        pw::fence_proxy_async_smem();
        __syncwarp();
      }
      if (pw::elect_one())
        pw::mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(mask)) * static_cast<uint32_t>(box * 2 * D));
      __syncwarp();
      for (int i = 0; i < boxes; ++i) {
        const int pg = __shfl_sync(0xFFFFFFFFu, this_page, i), at = __shfl_sync(0xFFFFFFFFu, row, i);
        if ((mask >> i & 1u) && pw::elect_one()) {
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            pw::tma_load_4d(pw::smem_u32(dst) + h * kHalfRow + i * box * 128, kValues ? &maps.v : &maps.k, 64 * h, at,
                            c.head, pg, full);
        }
        __syncwarp();
      }
      key0 = back ? 0 : key0 + kBlock;
    }
    return true;
  });
  __syncwarp();
  // No copy may be in flight when the CTA leaves: in a call that went well the
  // matrix instructions have waited for every one of them.
  if (*reinterpret_cast<volatile int*>(&sh.dead))
    for (uint32_t i = x > kSlots ? x - kSlots : 0; i < x; ++i)
      pw::mbar_wait(bar(fulls[i % kSlots]), (i / kSlots) & 1u, kDrainNs);
}

// ---------------------------------------------------------------- matrix instructions (one warp)
// The tensor cores queue a few instructions only, so what this warp does
// between two groups of them is time in which they run dry: addresses and
// descriptors are made beforehand, the halves are written out.  (One issuing
// warp a half instead lets the halves' products alternate, and both finish
// late: 1330 us against 1257 on 7.2k tokens over 16k keys.)
template <int D, bool kBf16, bool kSinks>
__device__ __forceinline__ void mma_role(const Params& p, const Cursor<kSinks>& start, Shared& sh, uint32_t tmem,
                                         uint32_t q_smem, uint32_t k_ring, uint32_t v_ring) {
  constexpr uint32_t kScores = pw::idesc_f32(kHalf, kBlock, kBf16, false);
  constexpr uint32_t kValues = pw::idesc_f32(kHalf, D, kBf16, true);
  constexpr uint32_t kStep = tile_bytes<D>() >> 4;
  const uint64_t q_desc = pw::sdesc_kmajor_sw128(q_smem), k_desc = pw::sdesc_kmajor_sw128(k_ring);
  const uint64_t v_desc = pw::sdesc_nmajor_sw128(v_ring, kHalfRow);
  pw::Ring<kKeySlots> keys;
  pw::Ring<kValueSlots> vals;
  uint32_t q_parity = 0, p_parity = 0;   // a bit a half
  bool ok = true;
  auto scores = [&](int h, bool free_after) {   // S_h = Q_h K^T
    const uint64_t q = q_desc + h * kStep, k = k_desc + keys.at * kStep;
    if (pw::elect_one()) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint64_t at = (i / 4) * (kHalfRow >> 4) + (i % 4) * 2;
        pw::tc_mma_f16(tmem + h * kBlock, q + at, k + at, kScores, i);
      }
      pw::tc_commit(bar(sh.s_full[h]));
      if (free_after) pw::tc_commit(bar(sh.k_empty[keys.at]));
    }
    __syncwarp();
  };
  // O_h (+)= P_h V, the first or the last 64 keys
  auto values = [&](int h, int part, bool first, bool free_after) {
    const uint64_t v = v_desc + vals.at * kStep;
    if (pw::elect_one()) {
#pragma unroll
      for (int j = 0; j < kBlock / 32; ++j) {
        const int i = part * (kBlock / 32) + j;
        pw::tc_mma_ts(tmem + 2 * kBlock + h * D, tmem + h * kBlock + 8 * i, v + i * (2048 >> 4), kValues,
                      !first || part > 0 || j > 0);
      }
      // o_done last: the CTA leaves after it, and no arrival may find it gone
      if (part && free_after) pw::tc_commit(bar(sh.v_empty[vals.at]));
      pw::tc_commit(bar(part ? sh.o_done[h] : sh.o_half[h]));
    }
    __syncwarp();
  };
  auto both = [&](const uint64_t& b1, uint32_t parity1, const uint64_t& b2, uint32_t parity2) {
    ok = pw::warp_wait2(&b1, parity1, &b2, parity2, &sh.dead, p.a.status);
    pw::tc_fence_after();
    return ok;
  };
  for_units(p, start, [&](const Cursor<kSinks>& c, int b0, int b1) {
    const bool two = halves_of(p, c) == 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !two) break;
      if (!both(sh.k_full[keys.at], keys.parity, sh.q_full[h], (q_parity >> h) & 1u)) return false;
      q_parity ^= 1u << h;
      scores(h, h == 1 || !two);
    }
    keys.next();
    for (int b = b0; b < b1; ++b) {
      const bool more = b + 1 < b1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !two) break;
        const bool last = h == 1 || !two;
        const uint32_t parity = (p_parity >> h) & 1u;
        if (!both(sh.p_full[h][0], parity, sh.v_full[vals.at], vals.parity)) return false;
        values(h, 0, b == b0, false);
        if (!both(sh.p_full[h][1], parity, more ? sh.k_full[keys.at] : sh.p_full[h][1], more ? keys.parity : parity))
          return false;
        values(h, 1, b == b0, last);
        p_parity ^= 1u << h;
        if (more) scores(h, last);
      }
      vals.next();
      if (more) keys.next();
    }
    return true;
  });
  if (!ok) {   // Tensor Memory goes back only when nothing writes it
    if (pw::elect_one()) pw::tc_commit(bar(sh.drained));
    __syncwarp();
    pw::mbar_wait(bar(sh.drained), 0, kDrainNs);
  }
}

// ---------------------------------------------------------------- softmax (four warps a half)
template <typename T, int D, bool kSinks>
__device__ __forceinline__ void write_queries(const Params& p, const Cursor<kSinks>& c, int h, int tid, unsigned char* q_smem) {
  constexpr int kUnits = D / 8;             // 16-byte units of a row
  constexpr int kStep = kHalf / kUnits;     // rows at once
  const pw_attn_args& a = p.a;
  const int rows = c.s.q_len * p.group, unit = tid % kUnits, first = tid / kUnits;
  const int r0 = c.tile * kTile + h * kHalf + first;
  int token = pw_attn::token_of(p, r0), head = r0 - token * p.group;
  const int token_step = kStep / p.group, head_step = kStep % p.group;
  const T* base = static_cast<const T*>(a.q) + c.s.q0 * a.q_stride_token + c.head * p.group * a.q_stride_head + unit * 8;
  // all loads at once: each queues behind the copies of keys and values
  uint4 v[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (r0 + i * kStep < rows)
      v[i] = __ldg(reinterpret_cast<const uint4*>(base + token * a.q_stride_token + head * a.q_stride_head));
    token += token_step;
    head += head_step;
    if (head >= p.group) {
      head -= p.group;
      ++token;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int row = first + i * kStep;
    *reinterpret_cast<uint4*>(q_smem + h * tile_bytes<D>() + (unit >> 3) * kHalfRow + row * 128 +
                              (((unit & 7) ^ (row & 7)) << 4)) = v[i];
  }
}

template <typename T, int D, bool kSinks>
__device__ __forceinline__ void softmax_role(const Params& p, const Cursor<kSinks>& start, const pw_attn::Cut& cut, Shared& sh,
                                             uint32_t tmem, unsigned char* q_smem) {
  const pw_attn_args& a = p.a;
  const int h = threadIdx.x / kHalf, tid = threadIdx.x % kHalf, lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
  const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
  const uint32_t s_tmem = tmem + lanes + h * kBlock, o_tmem = tmem + lanes + 2 * kBlock + h * D;
  const size_t part_floats = static_cast<size_t>(kTile) * (D + 2);
  uint32_t blocks = 0;   // of this half so far
  for_units(p, start, [&](const Cursor<kSinks>& c, int b0, int b1) {
    const int rows = c.s.q_len * p.group, r = c.tile * kTile + tid + h * kHalf;
    const bool live = r < rows;
    float m = -INFINITY, l = 0.0f;
    const bool active = h < halves_of(p, c);
    if (active) {
      write_queries<T, D>(p, c, h, tid, q_smem);
      pw::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) pw::mbar_arrive(bar(sh.q_full[h]));
      const int pos = c.s.kv_len - c.s.q_len + pw_attn::token_of(p, r);
      const uint64_t scale2 = pw::pack_f32x2(__float_as_uint(p.scale_log2), __float_as_uint(p.scale_log2));
      // the row's visible keys; a row past the end takes all of them and is not written
      const int hi = !live ? 0x7FFFFFFF : a.causal ? min(pos + 1, c.r.hi) : c.r.hi;
      const int lo = live && a.causal && a.window ? pos - a.window + 1 : 0;
      for (int b = b0; b < b1; ++b, ++blocks) {
        const int key0 = c.r.block_at(b) * kBlock;
        wait(sh.s_full[h], blocks & 1u, sh, p);
        pw::tc_fence_after();
        // no mask in this block
        const bool all = __all_sync(0xFFFFFFFFu, (lo <= key0 || (kSinks && p.sinks >= key0 + kBlock)) && hi >= key0 + kBlock);
        // 64 scores at a time: their maximum, then their weights, so that the
        // second product can start on the first 64 keys (with the maximum of all
        // 128 first it starts 350 cycles later, and the period is longer by as
        // much).
        uint64_t sum[2] = {0, 0};
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          uint32_t s[2][32];
          pw::tmem_ld_x32(s_tmem + 64 * i, s[0]);
          pw::tmem_ld_x32(s_tmem + 64 * i + 32, s[1]);
          pw::tmem_ld_wait();
          if (!all) {
            const int from = lo - key0 - 64 * i, to = hi - key0 - 64 * i, first = kSinks ? p.sinks - key0 - 64 * i : 0;
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if ((j < from && (!kSinks || j >= first)) || j >= to) s[j >> 5][j & 31] = 0xFF800000u;   // -inf
          }
          float most[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            most[j] = fmaxf(__uint_as_float(s[j >> 1][16 * (j & 1)]), __uint_as_float(s[j >> 1][16 * (j & 1) + 1]));
#pragma unroll
          for (int k = 2; k < 16; k += 2)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              most[j] = pw::max3(most[j], __uint_as_float(s[j >> 1][16 * (j & 1) + k]),
                                 __uint_as_float(s[j >> 1][16 * (j & 1) + k + 1]));
          const float top = fmaxf(pw::max3(most[0], most[1], most[2]), most[3]);
          // m follows the maximum in steps of at least 2^8 (and at once from
          // -inf); between a block's two parts only where the weights would
          // leave the 16-bit range otherwise.
          const bool moves = top > m && !((top - m) * p.scale_log2 <= (i ? kLazyInside : kLazy));
          if (__any_sync(0xFFFFFFFFu, moves)) {
            const bool scales = moves && m != -INFINITY;   // else there is nothing to scale
            float keep = 1.0f;
            if (moves) {
              keep = pw::exp2_fast((m - top) * p.scale_log2);
              m = top;
              l *= keep;
            }
            if (__any_sync(0xFFFFFFFFu, scales)) {
              if (!scales) keep = 1.0f;
              // the sum so far of this block's first part
              if (i) {
                float s0, s1;
                pw::unpack_f32x2(pw::add_f32x2(sum[0], sum[1]), s0, s1);
                l += (s0 + s1) * keep;
                sum[0] = sum[1] = 0;
              }
              // O has to be complete up to here before it is scaled
              wait(i ? sh.o_half[h] : sh.o_done[h], (i ? blocks : blocks - 1) & 1u, sh, p);
              pw::tc_fence_after();
#pragma unroll 1
              for (int j = 0; j < D / 16; ++j) {
                uint32_t o[16];
                pw::tmem_ld_x16(o_tmem + 16 * j, o);
                pw::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                pw::tmem_st_x16(o_tmem + 16 * j, o);
              }
              pw::tmem_st_wait();
            }
          }
          const float off = m == -INFINITY ? 0.0f : -m * p.scale_log2;
          const uint64_t off2 = pw::pack_f32x2(__float_as_uint(off), __float_as_uint(off));
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const uint32_t* src = &s[j >> 4][2 * (j & 15)];
            float e0, e1;
            pw::unpack_f32x2(pw::fma_f32x2(pw::pack_f32x2(src[0], src[1]), scale2, off2), e0, e1);
            e0 = pw::exp2_fast(e0);
            e1 = pw::exp2_fast(e1);
            sum[j & 1] = pw::add_f32x2(sum[j & 1], pw::pack_f32x2(__float_as_uint(e0), __float_as_uint(e1)));
            w[j] = pw::pack2<T>(e0, e1);   // in the values' type, as the instruction wants it; the sum is of the unrounded
          }
          pw::tmem_st_x32(s_tmem + 32 * i, w);
          pw::tmem_st_wait();
          pw::tc_fence_before();
          __syncwarp();
          if (lane == 0) pw::mbar_arrive(bar(sh.p_full[h][i]));
        }
        float s0, s1;
        pw::unpack_f32x2(pw::add_f32x2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      wait(sh.o_done[h], (blocks - 1) & 1u, sh, p);
      pw::tc_fence_after();
    }
    const float m2 = m * p.scale_log2;   // in powers of two
    const long long begin = c.unit_begin(), unit_end = c.unit_end();
    const bool whole = b0 == 0 && begin + b1 == unit_end;
    const int t0 = pw_attn::token_of(p, r), token = c.s.q0 + t0, head = c.head * p.group + r - t0 * p.group;
    T* out = static_cast<T*>(a.out) + token * a.out_stride_token + head * a.out_stride_head;
    const bool dead = *reinterpret_cast<volatile int*>(&sh.dead) != 0;
    if (whole) {
      if (active) {
        const float inv = pw_attn::inverse_sum(l);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t o[16];
          pw::tmem_ld_x16(o_tmem + 16 * i, o);
          pw::tmem_ld_wait();
          if (live && !dead) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pw::pack2<T>(__uint_as_float(o[8 * j + 2 * k]) * inv, __uint_as_float(o[8 * j + 2 * k + 1]) * inv);
              *reinterpret_cast<uint4*>(out + 16 * i + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (live && !dead && a.lse) a.lse[static_cast<int64_t>(token) * a.heads + head] = pw_attn::log_sum(m2, l);
        pw::tc_fence_before();
      }
      return true;
    }
    // a piece: [d / 4][row] of four values, so that neighbouring rows are
    // neighbours in memory; slot 0 when it starts at the stretch's begin
    const bool at_start = begin + b0 == cut.most * blockIdx.x;
    float* part = p.part + (2 * static_cast<size_t>(blockIdx.y * gridDim.x + blockIdx.x) + (at_start ? 0 : 1)) * part_floats;
    const int slot_row = h * kHalf + tid;
    if (active) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t o[16];
        pw::tmem_ld_x16(o_tmem + 16 * i, o);
        pw::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(part + ((4 * i + j) * kTile + slot_row) * 4) =
              make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
      }
      part[kTile * D + slot_row] = m2;
      part[kTile * D + kTile + slot_row] = l;
      pw::tc_fence_before();
    }
    // All eight warps add the pieces, whichever half has rows; the queries' part
    // of shared memory, read to the end by now, holds the joined state.
    static_assert(pw_attn::state_entries(pw_attn::kMaxCtas / 2, kTile) * sizeof(float2) <= 2 * tile_bytes<D>(), "state");
    pw_attn::join<kTile, D, false, 32 * kSoftmaxWarps, 8, 2>(
        p, cut, begin, unit_end, min(kTile, c.s.q_len * p.group - c.tile * kTile), reinterpret_cast<float2*>(q_smem), sh.last,
        [] { pw::bar_sync(1, 32 * kSoftmaxWarps); },
        [&](int row, int d, const float4* o, float top, float total) {
          if (*reinterpret_cast<volatile int*>(&sh.dead)) return;
          const int jr = c.tile * kTile + row, jt = pw_attn::token_of(p, jr), to = c.s.q0 + jt;
          const int hd = c.head * p.group + jr - jt * p.group;
          const float inv = pw_attn::inverse_sum(total);
          T* dst = static_cast<T*>(a.out) + to * a.out_stride_token + hd * a.out_stride_head + d;
#pragma unroll
          for (int k = 0; k < 8; k += 2)
            *reinterpret_cast<uint4*>(dst + 4 * k) =
                make_uint4(pw::pack2<T>(o[k].x * inv, o[k].y * inv), pw::pack2<T>(o[k].z * inv, o[k].w * inv),
                           pw::pack2<T>(o[k + 1].x * inv, o[k + 1].y * inv), pw::pack2<T>(o[k + 1].z * inv, o[k + 1].w * inv));
          if (a.lse && d == 0) a.lse[static_cast<int64_t>(to) * a.heads + hd] = pw_attn::log_sum(top, total);
        });
    return true;
  });
}

template <typename T, int D, bool kBf16, bool kSinks>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tile_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ Shared sh;
  unsigned char* smem = smem_raw + ((1024u - (pw::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = pw::uniform(static_cast<int>(threadIdx.x >> 5));
  Cursor<kSinks> c;
  pw_attn::Cut cut;
  if (!pw_attn::find_start<kTile, kBlock, kThreads, kLeast>(p, c, cut)) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKeySlots; ++i) {
      pw::mbar_init(bar(sh.k_full[i]), 1);
      pw::mbar_init(bar(sh.k_empty[i]), 1);
    }
    for (int i = 0; i < kValueSlots; ++i) {
      pw::mbar_init(bar(sh.v_full[i]), 1);
      pw::mbar_init(bar(sh.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      pw::mbar_init(bar(sh.q_full[i]), 4);
      pw::mbar_init(bar(sh.s_full[i]), 1);
      pw::mbar_init(bar(sh.p_full[i][0]), 4);
      pw::mbar_init(bar(sh.p_full[i][1]), 4);
      pw::mbar_init(bar(sh.o_half[i]), 1);
      pw::mbar_init(bar(sh.o_done[i]), 1);
    }
    pw::mbar_init(bar(sh.drained), 1);
    sh.dead = 0;
    pw::mbar_init_fence();
  }
  if (warp == kMmaWarp) {
    pw::tmem_alloc(pw::smem_u32(&sh.tmem), 512);
    pw::tmem_relinquish();
  }
  pw::tc_fence_before();
  __syncthreads();
  pw::tc_fence_after();
  const uint32_t tmem = pw::uniform(sh.tmem);
  unsigned char* k_ring = smem + 2 * tile_bytes<D>();
  unsigned char* v_ring = k_ring + kKeySlots * tile_bytes<D>();
  if (warp < kSoftmaxWarps) {
    softmax_role<T, D>(p, c, cut, sh, tmem, smem);
  } else if (warp == kKeyWarp) {
    load_role<D, false>(p, c, maps, sh, k_ring);
  } else if (warp == kValueWarp) {
    load_role<D, true>(p, c, maps, sh, v_ring);
  } else if (warp == kMmaWarp) {
    mma_role<D, kBf16>(p, c, sh, tmem, pw::smem_u32(smem), pw::smem_u32(k_ring), pw::smem_u32(v_ring));
  }
  __syncwarp();
  pw::tc_fence_before();
  __syncthreads();
  pw::tc_fence_after();
  if (warp == kMmaWarp) pw::tmem_dealloc(tmem, 512);
}

int encode_cache(CUtensorMap* m, const pw_attn_args& a, const void* base, int64_t page, int64_t token, int64_t head,
                 int box, bool bf16) {
  const uint64_t dims[4] = {static_cast<uint64_t>(a.head_dim), static_cast<uint64_t>(a.page_size),
                            static_cast<uint64_t>(a.kv_heads), static_cast<uint64_t>(a.num_pages)};
  // the stride of a dimension of one is never used, but the map wants a valid one
  const uint64_t strides[3] = {a.page_size > 1 ? 2ull * token : 256, a.kv_heads > 1 ? 2ull * head : 256,
                               a.num_pages > 1 ? 2ull * page : 256};
  const uint32_t bx[4] = {64, static_cast<uint32_t>(box), 1, 1};
  return pw::encode_tensor_map(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base, dims,
                               strides, bx);
}

template <typename T, int D, bool kBf16, bool kSinks>
int launch(const Params& p, cudaStream_t s) {
  constexpr int kDevs = 64;
  static bool attr_done[kDevs] = {};
  int dev = 0;
  PW_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= kDevs || !attr_done[dev]) {
    PW_CUDA_TRY(cudaFuncSetAttribute(attn_tile_kernel<T, D, kBf16, kSinks>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     smem_bytes<D>()));
    if (dev < kDevs) attr_done[dev] = true;
  }
  const int sms = pw::sm_count();
  if (sms < 1) return pw::set_error(PW_ERR_CUDA, "could not query the SM count");
  const pw_attn_args& a = p.a;
  Maps maps;
  maps.box = std::gcd(a.page_size, kBlock);
  if (int e = encode_cache(&maps.k, a, a.k_cache, a.k_stride_page, a.k_stride_token, a.k_stride_head, maps.box, kBf16))
    return e;
  if (int e = encode_cache(&maps.v, a, a.v_cache, a.v_stride_page, a.v_stride_token, a.v_stride_head, maps.box, kBf16))
    return e;
  const long long tiles = (static_cast<long long>(a.tokens) * p.group + kTile - 1) / kTile + a.batch;
  const long long blocks = tiles * ((a.max_kv_len + kBlock - 1) / kBlock + 1);
  const dim3 grid = pw_attn::grid_of(sms < pw_attn::kMaxCtas / 2 ? sms : pw_attn::kMaxCtas / 2, blocks, a.kv_heads);
  attn_tile_kernel<T, D, kBf16, kSinks><<<grid, kThreads, smem_bytes<D>(), s>>>(p, maps);
  PW_CUDA_TRY(cudaGetLastError());
  return PW_OK;
}

}  // namespace

namespace pw_attn {

size_t tile_part_floats(int head_dim) { return static_cast<size_t>(kTile) * (head_dim + 2); }

bool tile_kernel_takes(const Params& p) {
  const pw_attn_args& a = p.a;
  // More rows per key/value head than one 16-row tile: the other kernel would
  // read the keys once per 16 rows (64 sequences of 4096 keys, 4 query heads to
  // a key head: 8 tokens 185 us here, 333 there; 4 tokens 184 and 177).  A
  // positive scale (the running maximum is kept on unscaled scores); boxes of
  // whole 8-row swizzle groups; strides that a tensor map can hold.
  if (static_cast<long long>(a.max_q_len) * p.group <= 16 || !(a.scale > 0.0f)) return false;
  if (std::gcd(a.page_size, kBlock) < 8) return false;
  const int64_t most = 1ll << 38;
  for (int64_t st : {a.k_stride_page, a.k_stride_token, a.k_stride_head, a.v_stride_page, a.v_stride_token, a.v_stride_head})
    if (st < 1 || st > most) return false;
  return true;
}

template <bool kSinks>
int launch_tile(const Params& p, cudaStream_t s) {
  if (p.a.dtype == PW_DTYPE_F16)
    return p.a.head_dim == 64 ? launch<__half, 64, false, kSinks>(p, s) : launch<__half, 128, false, kSinks>(p, s);
  return p.a.head_dim == 64 ? launch<__nv_bfloat16, 64, true, kSinks>(p, s) : launch<__nv_bfloat16, 128, true, kSinks>(p, s);
}
int launch_tile_kernel(const Params& p, cudaStream_t s) {
  return p.sinks ? launch_tile<true>(p, s) : launch_tile<false>(p, s);
}

}  // namespace pw_attn
