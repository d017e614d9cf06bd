// sgq_group_rows.cu -- group ids -> rows in group order (include/sgq_group.h,
// group_rows).
//
// A stable counting sort in one launch. The ids are cut into contiguous
// pieces, one per warp of a cluster of up to 8 CTAs. With c[w][g] the number
// of ids g in warp w's piece, an id's slot is
//
//   start[g] + sum of c[w'][g] over earlier warps w' + earlier ids g in its piece,
//
// start[g] being the exclusive sum over groups of all warps' counts. A warp
// reads 32 ids at a time; match.any gives every lane the lanes that hold its
// id, so a rank inside the 32 is a popcount and only the first of equal lanes
// touches the warp's own counter: no atomics, the same order on every run.
// The CTAs of the cluster exchange their counts through distributed shared
// memory.
//
// The data is small (12 bytes an id), so latency bounds it: two passes over
// the ids with one exchange between them, and a warp's ids held in registers
// between the passes where they fit.
#include "sgq_group.cuh"

namespace sgq {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 16;          // ids a lane keeps between the two passes

__device__ __forceinline__ int load_id(const GroupRowsArgs& a, uint32_t i) {
    if (i >= a.n) return -1;
    if (a.wide) {
        const long long v = static_cast<const long long*>(a.ids)[i];
        return v >= 0 && v < a.groups ? (int)v : -1;
    }
    const int v = static_cast<const int*>(a.ids)[i];
    return v >= 0 && v < a.groups ? v : -1;
}

// The value at p in CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* p, uint32_t rank) {
    const uint32_t local = (uint32_t)__cvta_generic_to_shared(p);
    uint32_t remote, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
    return v;
}

// Shared memory: count [warps][groups], total [groups] (this CTA's), 32 words.
__global__ void __launch_bounds__(kThreads) group_rows_kernel(const GroupRowsArgs a) {
    extern __shared__ uint32_t sm[];
    const int G = a.groups, warps = blockDim.x >> 5;
    uint32_t* count = sm;
    uint32_t* total = sm + (size_t)warps * G;
    uint32_t* part = total + G;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ctas = cluster_ctas(), me = cluster_rank();
    for (int i = tid; i < warps * G; i += blockDim.x) count[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    // this warp's piece: `len` ids (a multiple of 32) from `first`
    const uint32_t pieces = ctas * warps;
    const uint32_t len = ((a.n + pieces - 1) / pieces + 31) & ~31u;
    const uint64_t first64 = (uint64_t)len * (me * warps + warp);
    const uint32_t first = first64 < a.n ? (uint32_t)first64 : a.n;
    const uint32_t steps = first < a.n ? ((a.n - first < len ? a.n - first : len) + 31) >> 5 : 0;
    uint32_t* mine = count + (size_t)warp * G;

    int id[kHeld];
    if (steps <= kHeld) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) id[j] = j < (int)steps ? load_id(a, first + 32 * j + lane) : -1;
    }
    auto each = [&](auto&& body) {      // body(step, id) for the piece's 32-id steps in order
        if (steps <= kHeld) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j)
                if (j < (int)steps) body((uint32_t)j, id[j]);
        } else {
            for (uint32_t j = 0; j < steps; ++j) body(j, load_id(a, first + 32 * j + lane));
        }
    };
    each([&](uint32_t, int g) {
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, g);
        if (g >= 0 && lane == __ffs(same) - 1) mine[g] += __popc(same);
        __syncwarp();
    });
    __syncthreads();
    // counts -> sums over this CTA's earlier warps
    for (int g = tid; g < G; g += blockDim.x) {
        uint32_t run = 0;
        for (int w = 0; w < warps; ++w) {
            const uint32_t c = count[(size_t)w * G + g];
            count[(size_t)w * G + g] = run;
            run += c;
        }
        total[g] = run;
    }
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // exclusive sum over the groups (at most 1024, so one a thread: blocks of
    // warps * 32 groups in turn), plus the earlier CTAs' counts
    uint32_t carry = 0;
    for (int g0 = 0; g0 < G; g0 += blockDim.x) {
        const int g = g0 + tid;
        uint32_t all = 0, before = 0;
        if (g < G) {
            for (uint32_t c = 0; c < ctas; ++c) {
                const uint32_t v = ctas > 1 ? ld_cluster_u32(total + g, c) : total[g];
                if (c < me) before += v;
                all += v;
            }
        }
        uint32_t incl = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += v;
        }
        if (lane == 31) part[warp] = incl;
        __syncthreads();
        uint32_t earlier = 0, whole = 0;
        for (int w = 0; w < warps; ++w) {
            const uint32_t v = part[w];
            if (w < warp) earlier += v;
            whole += v;
        }
        const uint32_t start = carry + earlier + incl - all;
        if (g < G) {
            if (me == 0) a.offsets[g] = (int32_t)start;
            for (int w = 0; w < warps; ++w) count[(size_t)w * G + g] += start + before;
        }
        carry += whole;
        __syncthreads();
    }
    if (me == 0 && tid == 0) a.offsets[G] = (int32_t)carry;
    __syncthreads();

    each([&](uint32_t j, int g) {
        const uint32_t i = first + 32 * j + lane;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, g);
        uint32_t slot = 0xFFFFFFFFu;
        if (g >= 0) {
            slot = mine[g] + __popc(same & ((1u << lane) - 1));
            a.rows[slot] = (int32_t)(i / a.k);
        }
        if (i < a.n && a.slots) a.slots[i] = (int32_t)slot;
        __syncwarp();
        if (g >= 0 && lane == __ffs(same) - 1) mine[g] += __popc(same);
        __syncwarp();
    });
    for (uint64_t s = carry + (uint64_t)me * blockDim.x + tid; s < a.n; s += (uint64_t)ctas * blockDim.x) a.rows[s] = -1;
    if (ctas > 1) {                    // no CTA leaves while another reads its counts
        cluster_arrive();
        cluster_wait();
    }
}

}  // namespace

cudaError_t launch_group_rows(const Device& dev, const GroupRowsArgs& a, cudaStream_t stream) {
    // one warp a 32 ids up to 32 warps; more CTAs once a lane would hold more than 4 ids
    int warps = (int)((a.n + 31) / 32 < (uint32_t)kWarps ? (a.n + 31) / 32 : (uint32_t)kWarps);
    if (warps < 4) warps = 4;
    int ctas = 1;
    while (ctas < kMaxCluster && (uint64_t)ctas * kThreads * 4 < a.n) ctas *= 2;
    const int smem = 4 * (warps * a.groups + a.groups + kWarps);
    return launch_grid(group_rows_kernel, dim3((unsigned)ctas), warps * 32, smem, ctas, dev.id, a, stream);
}

}  // namespace sgq
