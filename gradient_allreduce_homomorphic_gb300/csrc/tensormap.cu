// tensormap.cu -- tensor maps for TMA, through the driver's entry point (looked
// up once, so the library does not link against the driver).
#include "tensormap.cuh"

#include <atomic>

namespace gar {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

}  // namespace

namespace {

int encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
           const cuuint32_t *boxes, CUtensorMapSwizzle swizzle) {
    EncodeTiled fn = encode_tiled();
    if (!fn) return fail(GAR_ECUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint32_t elem[3] = {1, 1, 1};
    const CUresult r = fn(map, type, static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, boxes, elem,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(GAR_ECUDA, "cuTensorMapEncodeTiled: %d", static_cast<int>(r));
    return GAR_OK;
}

}  // namespace

int encode_tile_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner, int64_t outer, int64_t stride,
                    int box_inner, int box_outer, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
    const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
    return encode(map, type, 2, base, dims, strides, boxes, swizzle);
}

int encode_column_map(CUtensorMap *map, CUtensorMapDataType type, int elem, const void *base, int64_t inner, int64_t outer,
                      int64_t stride, int box_columns, int box_outer) {
    const int wide = 128 / elem;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(wide), static_cast<cuuint64_t>(outer), static_cast<cuuint64_t>(inner / wide)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride), 128};
    const cuuint32_t boxes[3] = {static_cast<cuuint32_t>(wide), static_cast<cuuint32_t>(box_outer), static_cast<cuuint32_t>(box_columns)};
    return encode(map, type, 3, base, dims, strides, boxes, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace gar
