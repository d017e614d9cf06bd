// sgq_attend_fp8_f16.cu -- paged_attention's kernels for E4M3 rows beside fp16 queries.
#include "sgq_attend.cuh"

namespace sgq {

cudaError_t attend::launch_fp8_f16(const Device& dev, const AttendArgs& a, cudaStream_t stream) {
    return launch_kind<FP8_F16>(dev, a, stream);
}

cudaError_t attend::gave_up_fp8_f16(uint32_t* n) { return read_gave_up(n); }

}  // namespace sgq
