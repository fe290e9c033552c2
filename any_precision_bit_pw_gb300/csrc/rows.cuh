// Rows of 16-bit values in the registers of a CTA: a thread holds units of eight
// columns.  Shared by norm_quant.cu and norm_add_norm.cu.
#pragma once

#include "ops_common.cuh"

namespace pw {

constexpr int kVec = 8;               // values of a unit: 16 bytes

// Eight values at columns c .. c+7 of a row, packed; columns past the end are 0.
template <typename T, bool kAligned>
__device__ __forceinline__ uint4 load8(const T* row, int c, int cols) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (kAligned) {
    if (c < cols) u = *reinterpret_cast<const uint4*>(row + c);
  } else {
    const uint16_t* v = reinterpret_cast<const uint16_t*>(row) + c;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (c + 2 * i < cols ? v[2 * i] : 0u) | (c + 2 * i + 1 < cols ? static_cast<uint32_t>(v[2 * i + 1]) << 16 : 0u);
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return u;
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[kVec]) {
  unpack2<T>(u.x, v[0], v[1]);
  unpack2<T>(u.y, v[2], v[3]);
  unpack2<T>(u.z, v[4], v[5]);
  unpack2<T>(u.w, v[6], v[7]);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&v)[kVec]) {
  return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}
template <typename T, bool kAligned>
__device__ __forceinline__ void store8(T* row, int c, int cols, const float (&v)[kVec]) {
  if (kAligned) {
    if (c < cols) *reinterpret_cast<uint4*>(row + c) = pack8<T>(v);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (c + i < cols) row[c + i] = from_float<T>(v[i]);
  }
}
template <bool kAligned>
__device__ __forceinline__ void store8_e4m3(uint8_t* row, int c, int cols, const float (&v)[kVec], const Divisor& by) {
  const uint32_t lo = e4m3x4(by(v[0]), by(v[1]), by(v[2]), by(v[3]));
  const uint32_t hi = e4m3x4(by(v[4]), by(v[5]), by(v[6]), by(v[7]));
  if (kAligned) {
    if (c < cols) *reinterpret_cast<uint2*>(row + c) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (c + i < cols) row[c + i] = static_cast<uint8_t>((i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) & 0xFFu);
  }
}

// Rows at any address of a 16-bit value.  The row's memory is cut into granules of
// 16 bytes at 16-byte addresses: with s values of granule 0 before the row,
// granule j holds columns 8j - s .. 8j - s + 7.  Granules inside the row move in one
// access, the two at its ends value by value; neighbouring lanes hold neighbouring
// units, and exchange what a granule has of its neighbour's unit.
__device__ __forceinline__ int row_shift(const void* row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1 & 7);
}
template <typename T>
__device__ __forceinline__ uint4 load_granule(const T* row, int c, int cols) {   // columns c .. c+7, c may be negative
  if (c >= 0 && c + kVec <= cols) return *reinterpret_cast<const uint4*>(row + c);
  const uint16_t* v = reinterpret_cast<const uint16_t*>(row);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = c + 2 * i;
    w[i] = (k >= 0 && k < cols ? v[k] : 0u) | (k + 1 >= 0 && k + 1 < cols ? static_cast<uint32_t>(v[k + 1]) << 16 : 0u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Values `off` .. off+7 of the sixteen of a and b; off is the same in the warp.
__device__ __forceinline__ uint4 eight_of(const uint4& a, const uint4& b, int off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (off & 2) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (off & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __byte_perm(w[i], w[i + 1], 0x5432);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 shift_down(const uint4& v) {
  return make_uint4(__shfl_down_sync(0xFFFFFFFFu, v.x, 1), __shfl_down_sync(0xFFFFFFFFu, v.y, 1),
                    __shfl_down_sync(0xFFFFFFFFu, v.z, 1), __shfl_down_sync(0xFFFFFFFFu, v.w, 1));
}
__device__ __forceinline__ uint4 shift_up(const uint4& v) {
  return make_uint4(__shfl_up_sync(0xFFFFFFFFu, v.x, 1), __shfl_up_sync(0xFFFFFFFFu, v.y, 1),
                    __shfl_up_sync(0xFFFFFFFFu, v.z, 1), __shfl_up_sync(0xFFFFFFFFu, v.w, 1));
}
// The unit at column c from the granules that the warp's lanes have loaded.  (The
// last lane's second granule is its next neighbour's first one: in L1 by now.)
template <typename T>
__device__ __forceinline__ uint4 unit_of(const uint4& granule, const T* row, int c, int cols) {
  const int s = row_shift(row);
  uint4 next = shift_down(granule);
  if ((threadIdx.x & 31) == 31 && s) next = load_granule(row, c + kVec - s, cols);
  return eight_of(granule, next, s);
}
template <typename T>
__device__ __forceinline__ void store_unit(T* row, int c, int cols, const float (&v)[kVec]) {
  const int s = row_shift(row), lane = threadIdx.x & 31;
  const uint4 own = pack8<T>(v), before = shift_up(own);
  // the granule at column c - s; what the warp's ends have of one goes value by value
  const uint4 w = s ? eight_of(before, own, kVec - s) : own;
  const int from = c - s, lo = lane == 0 ? c : max(from, 0), hi = min(from + kVec, cols);
  uint16_t* out = reinterpret_cast<uint16_t*>(row);
  if (lo == from && hi == from + kVec) {
    *reinterpret_cast<uint4*>(row + from) = w;
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (from + i >= lo && from + i < hi) out[from + i] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
  }
  if (lane == 31) {
    const uint32_t u[4] = {own.x, own.y, own.z, own.w};
#pragma unroll
    for (int i = 1; i < kVec; ++i)
      if (i >= kVec - s && c + i < cols) out[c + i] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
  }
}

// Scale of a group of 128 columns that 16 neighbouring threads hold, 8 each: its
// largest value is four shuffles away.
__device__ __forceinline__ float group_scale(const float (&v)[kVec]) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) top = max_nan(top, fabsf(v[i]));
#pragma unroll
  for (int o = 8; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  return max_nan(top / kE4m3Max, kMinScale);
}

// 16-byte accesses of 16-bit rows need the address, the stride and the width
// in multiples of 8 values; 8-byte accesses of codes the same in bytes.
inline bool rows_aligned(const void* ptr, int64_t stride, int cols) {
  return !ptr || (aligned(ptr, 16) && stride % kVec == 0 && cols % kVec == 0);
}
inline bool codes_aligned(const void* ptr, int64_t stride) { return !ptr || (aligned(ptr, 8) && stride % 8 == 0); }

inline int check_matrix(const char* op, const char* name, int64_t stride, int cols) {
  if (stride < cols)
    return set_error(PW_ERR_INVALID_ARG, "%s: row stride %lld of %s is below the %d columns", op,
                     static_cast<long long>(stride), name, cols);
  return PW_OK;
}

}  // namespace pw
