// fp8.cuh -- what the block-scaled 8-bit operators share.
//
// The scales of a matrix of `rows` rows, in blocks of 128 columns, are bytes
// in the order [ceil(blocks / 4)][rows][4]: the four blocks of 512 columns of
// one row make one 32-bit word, and neighbouring rows neighbouring words, so a
// tile of rows reads its scales coalesced and the tensor core takes each
// word's byte by its index.  Blocks past the last one hold 1, the scale of an
// all-zero block (any value but NaN's would do).
#pragma once

#include "common.cuh"

namespace gar {

__device__ __forceinline__ float load_f32(const float *p) { return *p; }
__device__ __forceinline__ float load_f32(const uint16_t *p) { return bf16_one(*p); }
__device__ __forceinline__ void store_f32(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_f32(uint16_t *p, float v) { *p = to_bf16(v); }

// Scale byte of block `blk` of `row`; the last block also fills its word.
__device__ __forceinline__ void store_scale(uint8_t *scale, int64_t rows, int64_t row, int64_t blk, int64_t blocks,
                                            uint32_t byte) {
    uint8_t *word = scale + ((blk >> 2) * rows + row) * 4;
    word[blk & 3] = static_cast<uint8_t>(byte);
    if (blk == blocks - 1)
        for (int i = static_cast<int>(blk & 3) + 1; i < 4; ++i) word[i] = 1;
}

}  // namespace gar
