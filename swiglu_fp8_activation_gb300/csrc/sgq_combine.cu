// sgq_combine.cu -- the weighted sum of each token's rows (include/sgq_group.h,
// combine_rows).
//
// One pass: a thread owns 16 columns of one token (8 where rows are not 32-byte
// aligned) and sums the k rows' pieces in fp32, in order of j. Bound by memory:
// every row of y is read once, in 32-byte loads, and several rows' loads are
// issued before the first is used, so that k does not multiply the latency.
// 8192 tokens x 8 rows of 6144, 95 of 100 of them there: 16-byte loads 8 ahead 149 us,
// 32-byte loads 8 ahead 132.6, 4 ahead 125.5 (866 MB, 6904 GB/s), where more CTAs
// fit a multiprocessor; 64 tokens of 4096, where they do not matter: 2.2, 2.06
// and 2.29.
#include "sgq_group.cuh"

namespace sgq {

namespace {

constexpr int kThreads = 64;

// PIECES 16-byte reads, side by side, of data that is read once. (Not by the
// read-only path: the kernel before may still write y when this one starts.)
template <int PIECES>
__device__ __forceinline__ void load_once(const void* p, uint4 (&v)[PIECES]) {
    if (PIECES == 2)
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[PIECES - 1].x), "=r"(v[PIECES - 1].y),
                       "=r"(v[PIECES - 1].z), "=r"(v[PIECES - 1].w)
                     : "l"(p)
                     : "memory");
    else
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w)
                     : "l"(p)
                     : "memory");
}

template <int DT, int PIECES, int AHEAD>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x / (uint32_t)a.nblk;
    const int n = ((int)(blockIdx.x % (uint32_t)a.nblk) * kThreads + (int)threadIdx.x) * 8 * PIECES;
    if (n >= a.N) return;
    const int32_t* slots = a.slots + t * a.k;
    const float* weights = a.weights ? a.weights + t * a.k : nullptr;
    float sum[PIECES][8] = {};
    for (int j0 = 0; j0 < a.k; j0 += AHEAD) {
        int64_t s[AHEAD];
        float c[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            s[j] = j0 + j < a.k ? slots[j0 + j] : -1;
            c[j] = weights && j0 + j < a.k ? weights[j0 + j] : 1.0f;
        }
        uint4 v[AHEAD][PIECES];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (s[j] >= 0 && s[j] < a.S) load_once<PIECES>(a.y + s[j] * a.N + n, v[j]);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (s[j] >= 0 && s[j] < a.S) {
#pragma unroll
                for (int p = 0; p < PIECES; ++p) {
                    float f[8];
                    load8<DT>(v[j][p], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[p][i] = fmaf(c[j], f[i], sum[p][i]);
                }
            }
        }
    }
#pragma unroll
    for (int p = 0; p < PIECES; ++p) st16_if(a.out + t * a.N + n + 8 * p, pack8<DT>(sum[p]), true);
}

template <int DT>
auto pick(bool wide, bool many) {
    return wide ? (many ? combine_kernel<DT, 2, 4> : combine_kernel<DT, 2, 8>) : combine_kernel<DT, 1, 8>;
}

}  // namespace

cudaError_t launch_combine(int dt, const Device& dev, const CombineArgs& a, cudaStream_t stream) {
    CombineArgs b = a;
    const bool wide = a.N % 16 == 0 && (reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.out)) % 32 == 0;
    const int columns = kThreads * (wide ? 16 : 8);
    b.nblk = (a.N + columns - 1) / columns;
    const int64_t ctas = a.T * b.nblk;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const bool many = ctas > 8 * (int64_t)dev.sms;
    return launch_grid(dt == DT_F16 ? pick<DT_F16>(wide, many) : pick<DT_BF16>(wide, many), dim3((unsigned)ctas), kThreads, 0, 1,
                       dev.id, b, stream);
}

}  // namespace sgq
