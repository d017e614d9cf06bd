// sgq_attend_bf16.cu -- paged_attention's kernels for bf16 rows.
#include "sgq_attend.cuh"

namespace sgq {

cudaError_t attend::launch_bf16(const Device& dev, const AttendArgs& a, cudaStream_t stream) {
    return launch_kind<BF16>(dev, a, stream);
}

cudaError_t attend::gave_up_bf16(uint32_t* n) { return read_gave_up(n); }

}  // namespace sgq
