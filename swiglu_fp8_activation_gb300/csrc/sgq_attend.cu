// sgq_attend.cu -- the kernels of paged_attention by the cache's format and the
// 16-bit type beside it, one translation unit each.
#include "sgq_attend.cuh"

namespace sgq {

cudaError_t launch_attend(int fmt, int dt, const Device& dev, const AttendArgs& a, cudaStream_t stream) {
    if (fmt == FMT_PT) return dt == DT_F16 ? attend::launch_fp8_f16(dev, a, stream) : attend::launch_fp8_bf16(dev, a, stream);
    return dt == DT_F16 ? attend::launch_f16(dev, a, stream) : attend::launch_bf16(dev, a, stream);
}

cudaError_t attend_gave_up(uint32_t* n) {
    *n = 0;
    for (const auto f : {attend::gave_up_bf16, attend::gave_up_f16, attend::gave_up_fp8_bf16, attend::gave_up_fp8_f16}) {
        uint32_t k = 0;
        const cudaError_t e = f(&k);
        if (e != cudaSuccess) return e;
        *n += k;
    }
    return cudaSuccess;
}

}  // namespace sgq
