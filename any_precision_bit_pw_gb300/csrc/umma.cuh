// More of the Blackwell features, for the operators outside the fused layer
// (tc_ptx.cuh has the barriers, copies and Tensor Memory of the layer itself):
// matrix instructions with both operands in shared memory, tiled copies of two
// to four dimensions, wide Tensor Memory loads and packed 32-bit arithmetic.
// Inline PTX written from the public PTX ISA description.
#pragma once

#include <cstdint>

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
// Waits for phase `parity`, at most `limit_ns`.  A wait that runs out reports
// PW_ERR_TIMEOUT and sets the CTA's `dead` word, which ends every other wait of
// the CTA: the caller stops issuing work, lets its own finish and returns.
__device__ __forceinline__ bool wait_or_dead(const uint64_t* bar, uint32_t parity, int* dead, int32_t* status,
                                             uint64_t limit_ns) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait_hint(b, parity, 1000)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait_hint(b, parity, 1000)) {
    if (*reinterpret_cast<volatile int*>(dead)) return false;
    if (global_ns() - t0 > limit_ns) {
      *reinterpret_cast<volatile int*>(dead) = 1;
      if (status) atomicCAS(status, 0, PW_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// The same for a whole warp: its lanes leave together (one may see the
// barrier, another the failure).
__device__ __forceinline__ bool warp_wait_or_dead(const uint64_t* bar, uint32_t parity, int* dead, int32_t* status,
                                                  uint64_t limit_ns) {
  return __all_sync(0xFFFFFFFFu, wait_or_dead(bar, parity, dead, status, limit_ns));
}

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
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace pw
