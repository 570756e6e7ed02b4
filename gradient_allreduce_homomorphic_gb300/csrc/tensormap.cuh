// tensormap.cuh -- host side of the TMA tile loads: a map of a matrix whose rows
// are contiguous, its tiles laid out in shared memory with a swizzle (of 128 bytes
// unless told otherwise).
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace gar {

// The matrix has `outer` rows of `inner` elements, a row every `stride` bytes
// (base and stride multiples of 16 bytes); a tile is box_outer rows of box_inner
// elements (128 bytes).  What lies outside the matrix loads as zero.
int encode_tile_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner, int64_t outer, int64_t stride,
                    int box_inner, int box_outer, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

// The same matrix cut into columns of 128 bytes (inner a multiple of them): a tile is
// box_outer rows of box_columns such columns, column by column.
int encode_column_map(CUtensorMap *map, CUtensorMapDataType type, int elem, const void *base, int64_t inner, int64_t outer,
                      int64_t stride, int box_columns, int box_outer);

}  // namespace gar
