// More of the Blackwell features, for the operators outside the fused layer
// (tc_ptx.cuh has the barriers, copies and Tensor Memory of the layer itself):
// matrix instructions with both operands in shared memory, tiled copies of two
// to four dimensions, wide Tensor Memory loads and packed 32-bit arithmetic.
// Inline PTX written from the public PTX ISA description.
#pragma once

#include <cstdint>

#include "ops_common.cuh"
#include "tc_ptx.cuh"
#include "umma_host.h"

namespace pw {

// ---------------------------------------------------------------- warp-uniform code
// The matrix instructions and copies take uniform registers.  A role that the
// whole warp runs, with loop bounds and addresses known to be the same in all
// lanes and only the instructions themselves behind elect_one, keeps its
// operands there; a role inside `if (lane == 0)` moves each of them at every
// instruction (measured: 100 instead of 64 cycles per 128 x 128 x 16 step).
__device__ __forceinline__ bool elect_one() {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(v));
  return v != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// ---------------------------------------------------------------- bounded waits
// A whole warp waits for phase `parity`.  Each try sleeps up to 1 us; after
// kWaitTries of them (80 ms at the least, seconds in practice; the waits here
// are for the CTA's own work and take microseconds) the wait reports
// PW_ERR_TIMEOUT and sets the CTA's `dead` word, which ends every other wait of
// the CTA: the caller stops issuing work, lets its own finish and returns.  The
// lanes leave together.  Kept this short because every role holds copies of it
// in the instruction cache.
constexpr int kWaitTries = 1 << 22;
__device__ __forceinline__ bool warp_wait(const uint64_t* bar, uint32_t parity, int* dead, int32_t* status) {
  const uint32_t b = smem_u32(bar);
  int tries = 0;
  while (!__all_sync(0xFFFFFFFFu, mbar_try_wait_hint(b, parity, 1000))) {
    if (__any_sync(0xFFFFFFFFu, ++tries > kWaitTries || *reinterpret_cast<volatile int*>(dead))) {
      if (atomicExch(dead, 1) == 0) atomicCAS(status, 0, PW_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// Two barriers in one step, for a role whose waits are on its critical path.
__device__ __forceinline__ bool warp_wait2(const uint64_t* bar1, uint32_t parity1, const uint64_t* bar2, uint32_t parity2,
                                           int* dead, int32_t* status) {
  const bool one = mbar_try_wait(smem_u32(bar1), parity1), two = mbar_try_wait(smem_u32(bar2), parity2);
  if (__all_sync(0xFFFFFFFFu, one && two)) return true;
  return warp_wait(bar1, parity1, dead, status) && warp_wait(bar2, parity2, dead, status);
}

// A position in a ring of kSize barriers and the parity of its current use.
template <uint32_t kSize>
struct Ring {
  uint32_t at = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if (++at == kSize) {
      at = 0;
      parity ^= 1u;
    }
  }
};

// ---------------------------------------------------------------- matrix instructions
// D[tmem] (+)= A[smem] x B[smem]^T, e4m3 operands (K = 32 a step), fp32 accumulate.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same for fp16 or bf16 operands (K = 16 a step).
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same by a pair of CTAs: 256 rows of A (128 in each CTA's shared memory),
// N rows of B (half in each), and each CTA's Tensor Memory gets its 128 rows.
// One thread of the pair's first CTA issues it.
__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs of the pair once the
// thread's matrix instructions have completed.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Arrives on a barrier of any CTA of the cluster.  Orders nothing but this
// thread's tcgen05 work (with the fence before it): a release at cluster scope
// costs over 1000 cycles and has no memory to publish here.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t cluster_addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Instruction descriptor: D fp32, A K-major, shape M x N.  kind::f8f6f4 with
// both operands e4m3 has the same bits as kind::f16 with both fp16 (format 0).
constexpr uint32_t idesc_f32(int M, int N, bool bf16, bool b_mn_major) {
  return (1u << 4)                                    // D format: f32
         | (bf16 ? (1u << 7) | (1u << 10) : 0u)       // A, B format
         | (b_mn_major ? 1u << 16 : 0u)               // B is N-major
         | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Shared-memory descriptor of an N-major operand (rows of K, 64 values of N to
// a 128-byte swizzled row): 8-row groups of K are 1024 bytes apart, the next 64
// values of N `n_stride` bytes.  A step of 16 K advances the address by 2048.
__device__ __forceinline__ uint64_t sdesc_nmajor_sw128(uint32_t smem_addr, uint32_t n_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(n_stride >> 4) << 16;           // leading byte offset
  d |= static_cast<uint64_t>(1024u >> 4) << 32;              // stride byte offset
  d |= static_cast<uint64_t>(1u) << 46;                      // descriptor version
  d |= static_cast<uint64_t>(2u) << 61;                      // 128-byte swizzle
  return d;
}

// ---------------------------------------------------------------- tiled copies (TMA)
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// A copy into this CTA's shared memory that completes on a barrier of the
// pair's first CTA (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, int c0, int c1, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(c0), "r"(c1), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The thread's stores have read their shared memory / are complete.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// ---------------------------------------------------------------- Tensor Memory
// 32 lanes x 32 consecutive columns.
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---------------------------------------------------------------- packed fp32
// Two 32-bit operations in one instruction.
__device__ __forceinline__ uint64_t pack_f32x2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t twice(float v) { return pack_f32x2(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Divisor's quotients, of two values.
struct PairDivisor {
  uint64_t s, inv, neg;
  __device__ __forceinline__ explicit PairDivisor(const Divisor& by) : s(twice(by.s)), inv(twice(by.inv)), neg(twice(-by.inv)) {}
  __device__ __forceinline__ uint64_t operator()(uint64_t v) const {
    const uint64_t q = mul_f32x2(v, inv);
    return fma_f32x2(fma_f32x2(q, s, v ^ 0x8000000080000000ull), neg, q);
  }
};
// e4m3 codes of four values.
__device__ __forceinline__ uint32_t e4m3_pairs(uint64_t a, uint64_t b) {
  float f[4];
  unpack_f32x2(a, f[0], f[1]);
  unpack_f32x2(b, f[2], f[3]);
  return e4m3x4(f[0], f[1], f[2], f[3]);
}

}  // namespace pw
