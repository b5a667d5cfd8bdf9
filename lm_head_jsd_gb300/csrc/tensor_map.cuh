// TMA tensor maps (internal).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace fljsd {

enum class MapType { kBf16, kF32, kU8 };

// 2-D map over a row-major [outer x inner] matrix with row stride ld elements:
// boxes of box_outer rows x box_inner elements, 128-byte swizzle or none, zeros past
// the edges. ptr and the row stride in bytes must be multiples of 16.
bool make_tensor_map(CUtensorMap* m, MapType type, const void* ptr, int64_t inner, int64_t outer,
                     int64_t ld, int box_inner, int box_outer, bool swizzle = true);

}  // namespace fljsd
