// sgq_ragged.cuh -- what the products over ragged groups share on the device:
// the scan of the offsets that gives every CTA the tiles, and the loads of
// row chunks.
#pragma once

#include "sgq_group.cuh"

namespace sgq {

constexpr int kChunk = 128;        // bytes of K a chunk: one row of a 128-byte swizzled operand

// Warp-wide and block-wide inclusive scan (maximum or sum) of one value a thread.
template <bool MAX>
__device__ __forceinline__ int block_scan(int v, int* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v = MAX ? max(v, o) : v + o;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before = MAX ? max(before, part[w]) : before + part[w];
    __syncthreads();
    return MAX ? max(v, before) : v + before;
}

// lo[g] = the held offset of group g (g = 0 .. G), first[g] = tiles of bn
// slots in the groups before g. All threads of the block.
__device__ inline void scan_groups(const int32_t* offsets, int G, int S, int bn, int* lo, int* first, int* part) {
    const int per = (G + (int)blockDim.x) / (int)blockDim.x;                   // of G + 1 offsets, per a thread
    const int b = threadIdx.x * per, e = min(b + per, G + 1);
    int run = 0;
    for (int g = b; g < e; ++g) {
        run = max(run, held(offsets[g], 0, S));
        lo[g] = run;
    }
    const int upto = block_scan<true>(run, part);                 // includes this thread's own
    // earlier threads' maximum: the scan without this thread's values
    first[threadIdx.x] = upto;
    __syncthreads();
    const int before = threadIdx.x ? first[threadIdx.x - 1] : 0;
    __syncthreads();
    for (int g = b; g < e; ++g) lo[g] = max(lo[g], before);
    __syncthreads();
    int sum = 0;
    for (int g = b; g < e && g < G; ++g) sum += (lo[g + 1] - lo[g] + bn - 1) / bn;
    int at = block_scan<false>(sum, part) - sum;
    for (int g = b; g < e; ++g) {
        first[g] = at;
        if (g < G) at += (lo[g + 1] - lo[g] + bn - 1) / bn;
    }
    __syncthreads();
}

}  // namespace sgq
