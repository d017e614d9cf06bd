// sgq_ragged.cuh -- what the products over ragged groups share on the device:
// the scan of the offsets that gives every CTA the tiles, and the loads of
// row chunks.
#pragma once

#include "sgq_group.cuh"

namespace sgq {

constexpr int kChunk = 128;        // bytes of K a chunk: one row of a 128-byte swizzled operand

// Exclusive scan (maximum or sum) over the block of one value >= 0 a thread;
// part: an int a warp.
template <bool MAX>
__device__ __forceinline__ int block_scan(int v, int* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v = MAX ? max(v, o) : v + o;
    }
    if (lane == 31) part[warp] = v;
    v = __shfl_up_sync(0xFFFFFFFFu, v, 1);
    if (lane == 0) v = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v = MAX ? max(v, part[w]) : v + part[w];
    __syncthreads();
    return v;
}

// lo[g] = the held offset of group g (g = 0 .. G), first[g] = tiles of bn
// slots in the groups before g. All threads of the block; tables of G + 1.
// Up to 127 groups one warp does it in shuffles (0.9 us with the loads at 64
// groups; the whole block, with its six barriers, 1.3).
__device__ inline void scan_groups(const int32_t* offsets, int G, int S, int bn, int* lo, int* first, int* part) {
    if (G < 128) {
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x;
            int v[4], carry = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = i * 32 + lane <= G ? held(offsets[i * 32 + lane], 0, S) : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, v[i], d);
                    if (lane >= d) v[i] = max(v[i], o);
                }
                v[i] = max(v[i], carry);
                carry = __shfl_sync(0xFFFFFFFFu, v[i], 31);
                if (i * 32 + lane <= G) lo[i * 32 + lane] = v[i];
            }
            carry = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // the next entry is the next lane's, or lane 0's of the next 32
                int next = __shfl_down_sync(0xFFFFFFFFu, v[i], 1);
                const int head = i < 3 ? __shfl_sync(0xFFFFFFFFu, v[i < 3 ? i + 1 : 3], 0) : 0;
                if (lane == 31) next = head;
                const int mine = i * 32 + lane < G ? (next - v[i] + bn - 1) / bn : 0;
                int sum = mine;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                    if (lane >= d) sum += o;
                }
                if (i * 32 + lane <= G) first[i * 32 + lane] = carry + sum - mine;
                carry += __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
        }
        __syncthreads();
        return;
    }
    const int per = (G + (int)blockDim.x) / (int)blockDim.x;     // of G + 1 offsets, per a thread
    const int b = threadIdx.x * per, e = min(b + per, G + 1);
    int run = 0;
    for (int g = b; g < e; ++g) {
        run = max(run, held(offsets[g], 0, S));
        lo[g] = run;
    }
    const int before = block_scan<true>(run, part);              // the earlier threads' maximum
    for (int g = b; g < e; ++g) lo[g] = max(lo[g], before);
    __syncthreads();
    int sum = 0;
    for (int g = b; g < e && g < G; ++g) sum += (lo[g + 1] - lo[g] + bn - 1) / bn;
    int at = block_scan<false>(sum, part);
    for (int g = b; g < e; ++g) {
        first[g] = at;
        if (g < G) at += (lo[g + 1] - lo[g] + bn - 1) / bn;
    }
    __syncthreads();
}

// Stores into the copy of the shared memory at p that the cluster's CTA `rank` holds.
__device__ __forceinline__ void st_cluster16(const void* p, uint32_t rank, float4 v) {
    const uint32_t local = (uint32_t)__cvta_generic_to_shared(p);
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(remote), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

__device__ __forceinline__ void st_cluster4(const void* p, uint32_t rank, float v) {
    const uint32_t local = (uint32_t)__cvta_generic_to_shared(p);
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(v) : "memory");
}

// Entries of a table of the groups' offsets in shared memory (16-byte multiple).
__host__ __device__ constexpr int table_ints(int groups) { return (groups + 8 + 3) & ~3; }

// The group and slots [s0, s0 + m) of tile q of bn slots; false behind the
// last. Binary search in the scanned offsets.
__device__ __forceinline__ bool find_tile(const int* lo, const int* first, int G, int bn, int q, int& g, int& s0, int& m) {
    if (q >= first[G]) return false;
    int a = 0, b = G;                // first[a] <= q < first[b]
    while (b - a > 1) {
        const int c = (a + b) >> 1;
        if (first[c] <= q) a = c;
        else b = c;
    }
    g = a;
    s0 = lo[a] + (q - first[a]) * bn;
    m = min(bn, lo[a + 1] - s0);
    return true;
}

}  // namespace sgq
