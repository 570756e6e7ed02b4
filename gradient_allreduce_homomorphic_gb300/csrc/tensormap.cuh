// tensormap.cuh -- host side of the TMA tile loads: a map of a matrix whose rows
// are contiguous, its tiles laid out in shared memory with the 128-byte swizzle.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace gar {

// The matrix has `outer` rows of `inner` elements, a row every `stride` bytes
// (base and stride multiples of 16 bytes); a tile is box_outer rows of box_inner
// elements (128 bytes).  What lies outside the matrix loads as zero.
int encode_tile_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner, int64_t outer, int64_t stride,
                    int box_inner, int box_outer);

}  // namespace gar
