// sgq_attend_bf16.cu -- paged_attention's kernels for bf16 rows.
#include "sgq_attend.cuh"

namespace sgq {

cudaError_t attend::launch_bf16(const Device& dev, const AttendArgs& a, cudaStream_t stream) {
    return launch_kind<BF16>(dev, a, stream);
}

}  // namespace sgq
