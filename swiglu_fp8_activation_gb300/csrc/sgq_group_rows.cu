// sgq_group_rows.cu -- group ids -> rows in group order (include/sgq_group.h,
// group_rows).
//
// A stable counting sort in one launch. The ids are cut into contiguous
// pieces, one per warp of a cluster of up to 16 CTAs. With c[w][g] the number
// of ids g in warp w's piece, an id's slot is
//
//   start[g] + sum of c[w'][g] over earlier warps w' + earlier ids g in its piece,
//
// start[g] being the exclusive sum over groups of all warps' counts. A warp
// takes 32 ids at a time and finds for every lane the lanes that hold its id,
// one ballot a bit of the group number, so that a rank inside the 32 is a
// popcount and only the first of equal lanes touches the warp's own counter: no
// atomics, the same order on every run. (match.any in place of the ballots
// took 48 cycles a warp of the whole multiprocessor: 131072 ids of 160 groups
// ran in 38 us with it.) The ranks stay in registers between the passes where
// they fit. The CTAs exchange their counts through distributed shared memory.
//
// The data is small (12 bytes an id), so latency bounds it: launch, one read
// of the ids, one exchange, the writes. With several CTAs each puts its rows in
// group order in shared memory first and writes them as runs, a warp a group: as
// 32 separate 4-byte stores an instruction the writes took half of the time.
// 131072 ids of 160 groups: 12.7 us (17.8 with 8 CTAs at most), 2^20 of 128: 94 (180).
#include "sgq_group.cuh"

#include <atomic>

namespace sgq {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 16;       // of the cluster (8 where the device has no room for 16)
constexpr int kHeld = 16;          // ids a lane keeps between the two passes

// The group of id i, G (none of them) where it is outside [0, G) or i is behind the last.
template <bool WIDE>
__device__ __forceinline__ uint32_t load_id(const GroupRowsArgs& a, uint64_t i) {
    const uint32_t G = (uint32_t)a.groups;
    if (WIDE) {
        const unsigned long long v = i < a.n ? static_cast<const unsigned long long*>(a.ids)[i] : G;
        return v < G ? (uint32_t)v : G;
    }
    const uint32_t v = i < a.n ? static_cast<const uint32_t*>(a.ids)[i] : G;
    return v < G ? v : G;
}

// The lanes whose g is this lane's; g < 2^BITS.
template <int BITS>
__device__ __forceinline__ uint32_t lanes_with(uint32_t g) {
    uint32_t same = 0xFFFFFFFFu;
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
        const bool bit = g & (1u << b);
        const uint32_t set = __ballot_sync(0xFFFFFFFFu, bit);
        same &= bit ? set : ~set;
    }
    return same;
}

// The value at p in CTA `rank`'s shared memory.
__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* p, uint32_t rank) {
    const uint32_t local = (uint32_t)__cvta_generic_to_shared(p);
    uint32_t remote, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
    return v;
}

// Shared memory: count [warps][groups], total, base and local [groups] (of this
// CTA), two words a warp, and with several CTAs that hold their ids sorted [32 kHeld warps].
template <bool WIDE, int BITS>
__global__ void __launch_bounds__(kThreads) group_rows_kernel(const GroupRowsArgs a) {
    extern __shared__ uint32_t sm[];
    const int G = a.groups, warps = blockDim.x >> 5;
    uint32_t* count = sm;
    uint32_t* total = sm + (size_t)warps * G;
    uint32_t* base = total + G;
    uint32_t* local = base + G;      // first of a group's rows in `sorted`
    uint32_t* part = local + G;
    uint32_t* sorted = part + 2 * kWarps;
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
    const bool held = len <= 32 * kHeld, runs = held && ctas > 1;
    uint32_t* mine = count + (size_t)warp * G;
    const uint32_t earlier_lanes = (1u << lane) - 1;
    // rank of this lane's id among the piece's ids of its group so far, and the piece's counts
    auto take = [&](uint32_t g) {
        const uint32_t same = lanes_with<BITS>(g);
        const uint32_t before = g < (uint32_t)G ? mine[g] : 0;
        __syncwarp();
        if (g < (uint32_t)G && (same & earlier_lanes) == 0) mine[g] = before + __popc(same);
        __syncwarp();
        return before + __popc(same & earlier_lanes);
    };

    uint32_t id[kHeld], rank[kHeld];
    if (held) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) id[j] = load_id<WIDE>(a, j < (int)steps ? (uint64_t)first + 32 * j + lane : a.n);
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (j < (int)steps) rank[j] = take(id[j]);
    } else {
        for (uint32_t j = 0; j < steps; ++j) take(load_id<WIDE>(a, (uint64_t)first + 32 * (uint64_t)j + lane));
    }
    __syncthreads();
    // counts -> sums over this CTA's earlier warps
    for (int g = tid; g < G; g += blockDim.x) {
        uint32_t run = 0;
#pragma unroll 8
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
    // exclusive sum over the groups (blocks of as many as there are threads),
    // plus the earlier CTAs' counts
    uint32_t carry = 0, carry_own = 0;
    for (int g0 = 0; g0 < G; g0 += blockDim.x) {
        const int g = g0 + tid;
        uint32_t all = 0, before = 0;
        if (g < G) {
#pragma unroll
            for (uint32_t c = 0; c < (uint32_t)kMaxCtas; ++c) {
                const uint32_t v = c >= ctas ? 0 : ctas > 1 ? ld_cluster_u32(total + g, c) : total[g];
                if (c < me) before += v;
                all += v;
            }
        }
        const uint32_t own = g < G ? total[g] : 0;
        uint32_t incl = all, incl_own = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d), o = __shfl_up_sync(0xFFFFFFFFu, incl_own, d);
            if (lane >= d) {
                incl += v;
                incl_own += o;
            }
        }
        if (lane == 31) {
            part[warp] = incl;
            part[kWarps + warp] = incl_own;
        }
        __syncthreads();
        const uint32_t sums = lane < warps ? part[lane] : 0, sums_own = lane < warps ? part[kWarps + lane] : 0;
        uint32_t upto = sums, upto_own = sums_own;                       // of the warps
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, d), o = __shfl_up_sync(0xFFFFFFFFu, upto_own, d);
            if (lane >= d) {
                upto += v;
                upto_own += o;
            }
        }
        const uint32_t start = carry + __shfl_sync(0xFFFFFFFFu, upto - sums, warp) + incl - all;
        const uint32_t start_own = carry_own + __shfl_sync(0xFFFFFFFFu, upto_own - sums_own, warp) + incl_own - own;
        if (g < G) {
            if (me == 0) a.offsets[g] = (int32_t)start;
            base[g] = start + before;
            local[g] = start_own;
        }
        carry += __shfl_sync(0xFFFFFFFFu, upto, 31);
        carry_own += __shfl_sync(0xFFFFFFFFu, upto_own, 31);
        __syncthreads();
    }
    if (me == 0 && tid == 0) a.offsets[G] = (int32_t)carry;

    // id i is token i / k, counted along in steps of 32
    uint32_t i = first + lane, token = i / a.k, left = i - token * a.k;
    const uint32_t step_q = 32 / a.k, step_r = 32 - step_q * a.k;
    auto put = [&](uint32_t g, uint32_t rank_in_piece) {
        uint32_t slot = 0xFFFFFFFFu;
        if (g < (uint32_t)G) {
            const uint32_t at = mine[g] + rank_in_piece;
            slot = base[g] + at;
            if (runs) sorted[local[g] + at] = token;
            else a.rows[slot] = (int32_t)token;
        }
        if (i < a.n && a.slots) a.slots[i] = (int32_t)slot;
        i += 32;
        token += step_q;
        left += step_r;
        if (left >= a.k) {
            left -= a.k;
            ++token;
        }
    };
    if (held) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (j < (int)steps) put(id[j], rank[j]);
    } else {
        for (uint32_t j = 0; j < steps; ++j) {
            // `mine` holds the sums of the earlier warps and counts on from there
            const uint32_t g = load_id<WIDE>(a, (uint64_t)first + 32 * (uint64_t)j + lane);
            const uint32_t slot_in_cta = take(g);
            put(g, g < (uint32_t)G ? slot_in_cta - mine[g] : 0);
            __syncwarp();
        }
    }
    if (runs) {
        __syncthreads();
        for (int g = warp; g < G; g += warps)
            for (uint32_t j = lane; j < total[g]; j += 32) a.rows[base[g] + j] = (int32_t)sorted[local[g] + j];
    }
    for (uint64_t s = carry + (uint64_t)me * blockDim.x + tid; s < a.n; s += (uint64_t)ctas * blockDim.x) a.rows[s] = -1;
    if (ctas > 1) {                    // no CTA leaves while another reads its counts
        cluster_arrive();
        cluster_wait();
    }
}

using Kernel = void (*)(const GroupRowsArgs);

// Whether the device runs clusters of 16 of these CTAs, whatever shared memory
// they take: asked once a kernel and device, which also allows the size for the kernel.
bool runs_16(Kernel k, int which, int device) {
    constexpr int kDevices = 64;
    static std::atomic<int> seen[kDevices][6];       // 0: not asked yet, 1: no, 2: yes
    if (device < 0 || device >= kDevices) return false;
    int v = seen[device][which].load(std::memory_order_acquire);
    if (v == 0) {
        const void* f = reinterpret_cast<const void*>(k);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kMaxDynamicSmem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 16;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        const bool ok = ensure_dynamic_smem(f, device, kMaxDynamicSmem) == cudaSuccess &&
                        cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                        cudaOccupancyMaxActiveClusters(&n, k, &cfg) == cudaSuccess && n > 0;
        if (!ok) (void)cudaGetLastError();
        v = ok ? 2 : 1;
        seen[device][which].store(v, std::memory_order_release);
    }
    return v == 2;
}

}  // namespace

cudaError_t launch_group_rows(const Device& dev, const GroupRowsArgs& a, cudaStream_t stream) {
    // one warp a 32 ids up to 32 warps; more CTAs once a lane would hold more than 2 ids
    int warps = (int)((a.n + 31) / 32 < (uint32_t)kWarps ? (a.n + 31) / 32 : (uint32_t)kWarps);
    if (warps < 4) warps = 4;
    // bits that tell 0 .. groups apart (groups itself stands for no group)
    const int bits = a.groups < 64 ? 0 : a.groups < 256 ? 1 : 2;
    static constexpr Kernel kernels[2][3] = {{group_rows_kernel<false, 6>, group_rows_kernel<false, 8>, group_rows_kernel<false, 11>},
                                             {group_rows_kernel<true, 6>, group_rows_kernel<true, 8>, group_rows_kernel<true, 11>}};
    const Kernel k = kernels[a.wide != 0][bits];
    int ctas = 1;
    while (ctas < kMaxCtas && (uint64_t)ctas * kThreads * 2 < a.n) ctas *= 2;
    if (ctas > 8 && !runs_16(k, (a.wide != 0) * 3 + bits, dev.id)) ctas = 8;
    const int smem = 4 * (warps * a.groups + 3 * a.groups + 2 * kWarps + (ctas > 1 ? 32 * kHeld * warps : 0));
    return launch_grid(k, dim3((unsigned)ctas), warps * 32, smem, ctas, dev.id, a, stream);
}

}  // namespace sgq
