// sgq_tensormap.cu -- tensor maps for the bulk tensor copies of the grouped
// products.
#include "sgq_group.cuh"

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

}  // namespace sgq
