// Rows of 16-bit values in the registers of a CTA: a thread holds units of eight
// columns.  Shared by norm_quant.cu and norm_add_norm.cu.
#pragma once

#include "ops_common.cuh"
#include "umma.cuh"

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
template <typename T, bool kAligned>
__device__ __forceinline__ void store8(T* row, int c, int cols, const float (&v)[kVec]) {
  if (kAligned) {
    if (c < cols) *reinterpret_cast<uint4*>(row + c) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                                      pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
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

// Sixteen neighbouring columns of a row, packed, and as pairs of 32-bit numbers.
// Rows may start at any address of a 16-bit value; how they are accessed:
//  kWide     rows and widths of whole 32 bytes: one access
//  kHalves   of whole 16 bytes: two
//  kSame     all rows with the same number s of values between a 32-byte address
//            and their first column: a thread takes columns 16i - s .. 16i - s + 15,
//            those of one 32-byte cell.  What the first and the last cell of a row
//            hold of its neighbours is loaded with them, unless the matrix may end
//            there, and dropped; they are stored value by value
//  kShifted  any.  The row's memory is cut into granules of 16 bytes at 16-byte
//            addresses: with s values of the first one before the row, granule j
//            holds columns 8j - s .. 8j - s + 7.  Granules inside the row move in one
//            access, those at its ends value by value; neighbouring lanes hold
//            neighbouring columns, and exchange what a granule has of both.
enum class Access { kWide, kHalves, kSame, kShifted };
struct Sixteen {
  uint4 lo, hi;
};

__device__ __forceinline__ int row_shift(const void* row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1 & 7);
}
// Columns c .. c+7 (c may be negative): value by value, or in one access where they are a granule of the row.
template <typename T>
__device__ __forceinline__ uint4 by_value8(const T* row, int c, int cols) {
  const uint16_t* v = reinterpret_cast<const uint16_t*>(row);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = c + 2 * i;
    w[i] = (k >= 0 && k < cols ? v[k] : 0u) | (k + 1 >= 0 && k + 1 < cols ? static_cast<uint32_t>(v[k + 1]) << 16 : 0u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ uint4 load_granule(const T* row, int c, int cols) {
  return c >= 0 && c + kVec <= cols ? *reinterpret_cast<const uint4*>(row + c) : by_value8(row, c, cols);
}
template <typename T>
__device__ __forceinline__ void store_by_value8(T* row, int c, int lo, int hi, const uint4& w) {   // of c .. c+7 those in [lo, hi)
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint16_t* out = reinterpret_cast<uint16_t*>(row);
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (c + i >= lo && c + i < hi) out[c + i] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
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

// What the thread of columns c .. c+15 loads of the row: those columns, or
// (kShifted) two granules.
template <typename T, Access kAccess>
__device__ __forceinline__ Sixteen load16(const T* row, int c, int cols) {
  Sixteen v{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if constexpr (kAccess == Access::kWide) {
    if (c < cols)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v.lo.x), "=r"(v.lo.y), "=r"(v.lo.z), "=r"(v.lo.w), "=r"(v.hi.x), "=r"(v.hi.y), "=r"(v.hi.z), "=r"(v.hi.w)
                   : "l"(row + c)
                   : "memory");
  } else if constexpr (kAccess == Access::kHalves) {
    if (c < cols) v.lo = *reinterpret_cast<const uint4*>(row + c);
    if (c + kVec < cols) v.hi = *reinterpret_cast<const uint4*>(row + c + kVec);
  } else {
    const int s = row_shift(row);
    v.lo = load_granule(row, c - s, cols);
    v.hi = load_granule(row, c + kVec - s, cols);
  }
  return v;
}
// The thread's sixteen values of what load16 gave.  (The last lane's third granule
// is its neighbour's first one: in L1 by now.)
template <typename T, Access kAccess>
__device__ __forceinline__ Sixteen columns16(const Sixteen& v, const T* row, int c, int cols) {
  if constexpr (kAccess != Access::kShifted) {
    return v;
  } else {
    const int s = row_shift(row);
    uint4 next = shift_down(v.lo);
    if ((threadIdx.x & 31) == 31 && s) next = load_granule(row, c + 2 * kVec - s, cols);
    return Sixteen{eight_of(v.lo, v.hi, s), eight_of(v.hi, next, s)};
  }
}
// Stores columns c .. c+15; all lanes of the warp come here.
template <typename T, Access kAccess>
__device__ __forceinline__ void store16(T* row, int c, int cols, const Sixteen& v) {
  if constexpr (kAccess == Access::kWide || kAccess == Access::kSame) {
    if (kAccess == Access::kWide ? c < cols : c >= 0 && c + 16 <= cols) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + c), "r"(v.lo.x), "r"(v.lo.y),
                   "r"(v.lo.z), "r"(v.lo.w), "r"(v.hi.x), "r"(v.hi.y), "r"(v.hi.z), "r"(v.hi.w)
                   : "memory");
    } else if (kAccess == Access::kSame && c < cols) {
      store_by_value8(row, c, 0, cols, v.lo);
      store_by_value8(row, c + kVec, 0, cols, v.hi);
    }
  } else if constexpr (kAccess == Access::kHalves) {
    if (c < cols) *reinterpret_cast<uint4*>(row + c) = v.lo;
    if (c + kVec < cols) *reinterpret_cast<uint4*>(row + c + kVec) = v.hi;
  } else {
    const int s = row_shift(row), lane = threadIdx.x & 31;
    auto granule = [&](const uint4& w, int from, int lo) {            // from column lo on
      if (lo <= from && from >= 0 && from + kVec <= cols)
        *reinterpret_cast<uint4*>(row + from) = w;
      else
        store_by_value8(row, from, max(lo, 0), cols, w);
    };
    const uint4 before = shift_up(v.hi);
    const int off = (kVec - s) & 7;
    granule(s ? eight_of(before, v.lo, off) : v.lo, c - s, lane ? 0 : c);   // the first lane has nothing of its neighbour's
    granule(s ? eight_of(v.lo, v.hi, off) : v.hi, c + kVec - s, 0);
    if (lane == 31 && s) store_by_value8(row, c + kVec, c + 2 * kVec - s, cols, v.hi);   // and the last lane's end is nobody else's
  }
}
// kSame: the cell of columns c .. c+15 (c may be negative); `whole`: all of it lies in
// the matrix.  (One load, whose values are dropped where they are used: loads of
// single values are packed at once, which waits for each of them in the warps at
// the row's ends, and the others wait for these at the barrier: a third of all
// stalls.)
template <typename T>
__device__ __forceinline__ Sixteen load_cell(const T* row, int c, int cols, bool whole) {
  Sixteen v{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (c >= cols) return v;
  if (!whole) return Sixteen{by_value8(row, c, cols), by_value8(row, c + kVec, cols)};
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.lo.x), "=r"(v.lo.y), "=r"(v.lo.z), "=r"(v.lo.w), "=r"(v.hi.x), "=r"(v.hi.y), "=r"(v.hi.z), "=r"(v.hi.w)
               : "l"(row + c)
               : "memory");
  return v;
}
// Values outside the row to 0.
__device__ __forceinline__ void clip_cell(Sixteen& v, int c, int cols) {
  if (c >= 0 && c + 16 <= cols) return;
  uint32_t w[8] = {v.lo.x, v.lo.y, v.lo.z, v.lo.w, v.hi.x, v.hi.y, v.hi.z, v.hi.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] &= (c + 2 * i >= 0 && c + 2 * i < cols ? 0xFFFFu : 0u) | (c + 2 * i + 1 >= 0 && c + 2 * i + 1 < cols ? 0xFFFF0000u : 0u);
  v = Sixteen{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}
template <typename T>
__device__ __forceinline__ void unpack16(const Sixteen& u, uint64_t (&v)[8]) {
  const uint32_t w[8] = {u.lo.x, u.lo.y, u.lo.z, u.lo.w, u.hi.x, u.hi.y, u.hi.z, u.hi.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo, hi;
    unpack2<T>(w[i], lo, hi);
    v[i] = pack_f32x2(__float_as_uint(lo), __float_as_uint(hi));
  }
}
template <typename T>
__device__ __forceinline__ Sixteen pack16(const uint64_t (&v)[8]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo, hi;
    unpack_f32x2(v[i], lo, hi);
    w[i] = pack2<T>(lo, hi);
  }
  return Sixteen{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}

// The codes of columns c .. c+15, at a multiple of `align` (16, 8 or 1); c may be negative.
__device__ __forceinline__ void store_codes16(uint8_t* row, int c, int cols, const uint32_t (&code)[4], int align) {
  if (align == 16 && c >= 0 && c + 16 <= cols) {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(code[0], code[1], code[2], code[3]);
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (align >= 8 && c >= 0 && c + 8 * h + 8 <= cols) {
      *reinterpret_cast<uint2*>(row + c + 8 * h) = make_uint2(code[2 * h], code[2 * h + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + 8 * h + i >= 0 && c + 8 * h + i < cols) row[c + 8 * h + i] = static_cast<uint8_t>(code[2 * h + (i >> 2)] >> (8 * (i & 3)));
    }
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
