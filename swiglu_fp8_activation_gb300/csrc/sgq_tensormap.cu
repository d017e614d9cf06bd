// sgq_tensormap.cu -- tensor maps for the bulk tensor copies of the grouped
// products and of paged_attention.
#include "sgq_cache.cuh"

namespace sgq {

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (no link to the driver library).
EncodeTiled encoder() {
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

}  // namespace

bool encode_rows(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, int box_rows) {
    const EncodeTiled f = encoder();
    if (!f) return false;
    const cuuint64_t strides[2] = {dims[0], rank == 3 ? dims[0] * dims[1] : 0};
    const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_tiles512(CUtensorMap* m, const void* base, int64_t tiles) {
    const EncodeTiled f = encoder();
    if (!f) return false;
    const cuuint64_t dims[2] = {128, (cuuint64_t)tiles}, strides[1] = {512};
    const cuuint32_t box[2] = {128, 1}, step[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_cache(CUtensorMap* m, const CacheArgs& c, const void* rows, int tokens, int block, int elem) {
    const EncodeTiled f = encoder();
    if (!f) return false;
    const cuuint64_t width = (cuuint64_t)c.D * elem, apart = (width + 15) / 16 * 16;     // an axis of one has no stride of its own
    const cuuint64_t dims[4] = {width, c.page.d, (cuuint64_t)c.heads, (cuuint64_t)c.pages};
    const cuuint64_t strides[3] = {c.ts ? (cuuint64_t)c.ts : apart, c.hs ? (cuuint64_t)c.hs : apart, c.ps ? (cuuint64_t)c.ps : apart};
    const cuuint32_t box[4] = {(cuuint32_t)block, (cuuint32_t)tokens, 1, 1}, step[4] = {1, 1, 1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(rows), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             block == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sgq
