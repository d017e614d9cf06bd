// sgq_combine.cu -- the weighted sum of each token's rows (include/sgq_group.h,
// combine_rows).
//
// One pass: a thread owns 8 columns of one token and sums the k rows' chunks
// in fp32, in order of j. Bound by memory: every row of y is read once in
// 16-byte loads, and the loads of up to 8 rows are issued before the first is
// used, so that k does not multiply the latency.
#include "sgq_group.cuh"

namespace sgq {

namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;          // rows whose loads are in flight together

// 16-byte read of data that is read once.
__device__ __forceinline__ uint4 ld16_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x / (uint32_t)a.nblk;
    const int n = ((int)(blockIdx.x % (uint32_t)a.nblk) * kThreads + (int)threadIdx.x) * 8;
    if (n >= a.N) return;
    const int32_t* slots = a.slots + t * a.k;
    const float* weights = a.weights ? a.weights + t * a.k : nullptr;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
        int64_t s[kAhead];
        float c[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            s[j] = j0 + j < a.k ? slots[j0 + j] : -1;
            c[j] = weights && j0 + j < a.k ? weights[j0 + j] : 1.0f;
        }
        uint4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (s[j] >= 0 && s[j] < a.S) v[j] = ld16_once(a.y + s[j] * a.N + n);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (s[j] >= 0 && s[j] < a.S) {
                float f[8];
                load8<DT>(v[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = fmaf(c[j], f[i], sum[i]);
            }
        }
    }
    st16_if(a.out + t * a.N + n, pack8<DT>(sum), true);
}

}  // namespace

cudaError_t launch_combine(int dt, const Device& dev, const CombineArgs& a, cudaStream_t stream) {
    CombineArgs b = a;
    b.nblk = (a.N / 8 + kThreads - 1) / kThreads;
    const int64_t ctas = a.T * b.nblk;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_grid(dt == DT_F16 ? combine_kernel<DT_F16> : combine_kernel<DT_BF16>, dim3((unsigned)ctas), kThreads, 0,
                       1, dev.id, b, stream);
}

}  // namespace sgq
