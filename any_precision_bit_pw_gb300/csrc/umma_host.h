// Tensor maps (host side).
#pragma once

#include <cuda.h>

#include <cstdint>

#include "pw_internal.h"

namespace pw {

// Tiled tensor map; with the 128-byte swizzle `box[0]` elements are 128 bytes.
// strides[i] is the byte stride of dimension i + 1.
int encode_tensor_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const uint64_t* dims,
                      const uint64_t* strides, const uint32_t* box, bool swizzle = true);

}  // namespace pw
