// sgq_attend_f16.cu -- paged_attention's kernels for fp16 rows.
#include "sgq_attend.cuh"

namespace sgq {

cudaError_t attend::launch_f16(const Device& dev, const AttendArgs& a, cudaStream_t stream) {
    return launch_kind<F16>(dev, a, stream);
}

cudaError_t attend::gave_up_f16(uint32_t* n) { return read_gave_up(n); }

}  // namespace sgq
