// sgq_lora.cu -- low-rank adapters of many requests, added to a shared
// projection's output (include/sgq_group.h, lora_add).
//
// A first form, right for every case: a warp a (slot, rank) dot product into
// the workspace, then a thread a (slot, column).
#include "sgq_group.cuh"

namespace sgq {

namespace {

template <int DT>
__device__ __forceinline__ float value16(uint16_t v) {
    return DT == DT_BF16 ? __uint_as_float((uint32_t)v << 16) : f16x2_to_f32x2(v).x;
}

// The group of slot s (the last whose range holds it), or -1.
__device__ int group_of_slot(const LoraArgs& a, int s) {
    int prev = 0;
    for (int g = 0; g < a.groups; ++g) {
        const int lo = held(a.offsets[g], prev, a.S), hi = held(a.offsets[g + 1], lo, a.S);
        if (s >= lo && s < hi) return g;
        prev = lo;
    }
    return -1;
}

// The row of slot s, or -1 where it is outside or its token's slot is another.
__device__ int64_t row_of_slot(const LoraArgs& a, int s) {
    if (!a.rows) return s;
    const int64_t t = a.rows[s];
    return t >= 0 && t < a.T && a.slots[t] == s ? t : -1;
}

template <int DT>
__global__ void __launch_bounds__(128) lora_shrink_kernel(const LoraArgs a) {
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.x, g = group_of_slot(a, s);
    const int64_t t = row_of_slot(a, s);
    if (g < 0 || t < 0) return;
    for (int r = threadIdx.x / 32; r < a.R; r += 4) {
        float sum = 0;
        for (int k = threadIdx.x % 32; k < a.K; k += 32)
            sum = fmaf(value16<DT>(a.x[t * a.K + k]), value16<DT>(a.a[((int64_t)g * a.R + r) * a.K + k]), sum);
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (threadIdx.x % 32 == 0) a.v[(int64_t)s * a.R + r] = sum;
    }
}

template <int DT>
__global__ void __launch_bounds__(128) lora_expand_kernel(const LoraArgs a) {
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.x, g = group_of_slot(a, s);
    const int64_t t = row_of_slot(a, s);
    if (g < 0 || t < 0) return;
    const float c = a.scaling ? a.scaling[g] : 1.0f;
    for (int n = threadIdx.x; n < a.N; n += 128) {
        float sum = 0;
        for (int r = 0; r < a.R; ++r)
            sum = fmaf(a.v[(int64_t)s * a.R + r], value16<DT>(a.b[((int64_t)g * a.N + n) * a.R + r]), sum);
        const float y = fmaf(c, sum, value16<DT>(a.y[t * a.N + n]));
        a.y[t * a.N + n] = (uint16_t)(DT == DT_F16 ? f32x2_to_f16x2(y, 0.0f) : f32x2_to_bf16x2(y, 0.0f));
    }
}

}  // namespace

cudaError_t launch_lora(int dt, const Device& dev, const LoraArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)a.S);
    const cudaError_t e = launch_grid(dt == DT_F16 ? lora_shrink_kernel<DT_F16> : lora_shrink_kernel<DT_BF16>, grid, 128, 0,
                                      1, dev.id, a, stream);
    if (e != cudaSuccess) return e;
    return launch_grid(dt == DT_F16 ? lora_expand_kernel<DT_F16> : lora_expand_kernel<DT_BF16>, grid, 128, 0, 1, dev.id, a,
                       stream);
}

}  // namespace sgq
