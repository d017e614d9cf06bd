// sgq_attend.cuh -- attention of one new token a sequence over a paged cache
// (include/sgq_cache.h, paged_attention).
//
// Reading the cache bounds it: every key and value row is used by `group` heads
// of q, 4 to 16 operations a byte up to groups of 8.
//
// An item is a sequence and a head of the cache (a chunk of its group of q heads, where
// there are more than a CTA's columns); its tiles are 64 tokens, 128 of E4M3 rows of
// up to 128. Two ways of sharing them out, by the sizes that the host knows (attend_split):
//   * A cluster of 1 to 8 CTAs takes an item, each CTA an equal run of its tiles, and joins
//     in its shared memory. One launch.
//   * All items' tiles stand in one row, an item's end counted as some tiles more, and CTA c of G
//     takes those from c total / G on, total / G of them, rounded up or down; a second launch
//     joins what several CTAs have computed of one item. Empty sequences are not in the row.
// Lengths are read on the device in both, so a captured graph follows them.
//
// Inside a CTA each of four groups of warps takes a quarter of every tile's tokens, and each warp of a
// group 8 or 16 columns of them. A group runs by itself: its own copies, several tiles
// ahead and across the items' borders; a warp has its own running maximum and sums. All warps meet where an
// item ends, to add up.
//
// Products, transposed so that a small group wastes little of a tile: the tokens are
// the 16 rows of S = K q^T, the heads its 8 columns. p comes out of S with a
// token's row in a group of lanes and is turned in registers (movmatrix) into
// the right operand of O = V^T p. mma.sync and not tcgen05: its smallest tile of 64 by 8
// would need p in shared memory or FP8 q and p, and the products are not what bounds it.
//
// E4M3 rows become fp16, exactly, on their way into registers; each row's k scale multiplies its
// row of S, its v scale its p. The order in which the columns of q and k are
// summed, and in which the rows of V^T stand in their tiles, is free: both
// follow what a lane's 16-byte reads bring, so no byte is moved twice.
//
// The running maximum is a reference that is moved only when a weight exceeds it some 512
// times, so most tiles need no reduction over lanes and no rescaling.
#pragma once

#include "sgq_cache.cuh"
#include "sgq_tc.cuh"

// A test that makes a wait run out says here which copies come late or not at all, and how long waits are.
#ifndef SGQ_ATTEND_COPIES
#define SGQ_ATTEND_COPIES(item, part, tile) true
#define SGQ_ATTEND_WAIT sgq::tc::kWaitCycles
#endif

namespace sgq {
namespace attend {

constexpr int kParts = 4;                        // of a tile's tokens, a group of warps each
// Entries of items that CTAs share: one an item (few items, each of many CTAs), or one a CTA.
enum Joined : int { kByCta = 1, kByItem = 2 };
constexpr int kEnd = kAttendEnd;
constexpr int kStages = 8;                       // tiles copied ahead, at most (and 2 at least)
constexpr float kNone = -3.0e38f;                // below every logit
// Of a tile's p in a lane, with E4M3 rows: w does not bound it where a row's scale is small or 0. An item's longest sum, 2^24 tiles of a lane, stays finite.
constexpr float kMostSum = 0x1p40f;
// The powers of two that w is divided by: of normal numbers, up and down; rows of zeros alone, which have no size, come to the least.
constexpr float kLeastExp = -124.0f, kMostExp = 126.0f;

// Kinds of rows and queries.
enum Kind : int { BF16 = 0, F16 = 1, FP8_BF16 = 2, FP8_F16 = 3 };

// Columns: NT times 8 a warp, CG warps side by side. DIRECT: see attend_kernel.
template <int KIND, int DP, int CG, int NT, bool DIRECT>
struct Shape {
    static constexpr bool fp8 = KIND >= FP8_BF16;
    static constexpr int warps = kParts * CG, threads = warps * 32;
    static constexpr int tokens = attend_tokens(fp8, DP);            // of a tile
    static constexpr int rows = tokens / kParts;                 // that a warp takes at a time, 16 of them a product
    static constexpr int halves = rows / 16;
    static constexpr uint32_t full = rows == 32 ? 0xFFFFFFFFu : 0xFFFFu;         // the mask of rows that are all there
    static constexpr int elem = fp8 ? 1 : 2;
    // Rows in shared memory: blocks of 128 bytes (64: narrow E4M3 heads) of all rows, their 16-byte pieces in the order
    // that the copy engine's swizzle gives them.
    static constexpr int block = DP * elem < 128 ? 64 : 128, blocks = DP * elem / block;
    static constexpr int half = rows * DP * elem, slot = 2 * half;               // k's rows, and v's behind them
    static constexpr int scales = fp8 ? 2 * rows * 4 : 0;
    static constexpr int step = kParts * slot;                   // bytes of a tile: its parts' slots side by side
    static constexpr int ctas = attend_resident(fp8, DP, CG * NT * 8, DIRECT);
    // Tiles that fit in shared memory where n CTAs share a multiprocessor.
    static constexpr int bytes(int n) { return n * (step + kParts * scales) + 1024; }    // dynamic shared memory of n tiles
    static constexpr int fit(int n) { return (227 * 1024 / n - 4096) / (step + kParts * scales); }
    static constexpr int parts = KIND == FP8_BF16 ? 1 : 2;       // 16-bit parts of p
    // bytes of a column's sums: 4 lanes' columns meet no bank twice, where a slot has room for that
    static constexpr int line = (DP + (8 * (DP + 4) * 4 <= slot ? 4 : 0)) * 4;
    static constexpr int at_once = slot / (8 * line) < CG ? slot / (8 * line) : CG;      // groups of columns whose sums pass through a slot
    static_assert(at_once >= 1 && CG % at_once == 0 && fit(ctas) >= 2, "");
    // Where piece p (of 16 bytes) of row r lies, from the first row's beginning: two bits of the row, or three, turn the
    // pieces' order. Eight rows' pieces of one number meet no bank twice; of E4M3 k rows, read four pieces of two rows at a time, two do.
    static __device__ __forceinline__ int piece_at(int r, int p) {
        return block == 64 ? r * 64 + ((p << 4) ^ turn(r)) : (p >> 3) * (rows * 128) + r * 128 + (((p & 7) << 4) ^ turn(r));
    }
    static __device__ __forceinline__ int turn(int r) { return block == 64 ? ((r >> 1) & 3) << 4 : (r & 7) << 4; }
    static constexpr int pieces = DP * elem / 16;                // of a row
};

template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ void ldmatrix4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float lds_f32(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void sts16(uint32_t at, float4 v) {
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

__device__ __forceinline__ void sts_f32(uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }

// Four E4M3 codes -> two fp16 pairs, exactly.
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
                 ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// n bytes, a multiple of 16, from and to multiples of 16.
__device__ __forceinline__ void load_bytes(uint32_t dst, const void* from, uint32_t n, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(from), "r"(n), "r"(bar)
                 : "memory");
}

// An arrival of this thread, one of those that the barrier counts, once its own copies have landed.
__device__ __forceinline__ void arrive_with_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}

// floor(log2 s) of a scale; -127 for zero and what is subnormal, at most 127.
__device__ __forceinline__ float exponent(float s) { return (float)min(127, (int)((__float_as_uint(s) >> 23) & 0xFF) - 127); }

// 2^e of a whole e in [-126, 127].
__device__ __forceinline__ float power(float e) { return __uint_as_float((uint32_t)(127 + (int)e) << 23); }

// Walks over the tiles of a CTA's share, tiles of TOKENS each.
template <int TOKENS>
struct Walk {
    int b, j;            // sequence, item of it: chunk `chunk` of the cache's head `head`
    int head, chunk;
    int tile, tiles;     // of the item; none where the sequence is empty
    int lo, n;           // tokens [lo, n) are not masked
    int start;           // first token of the first tile

    __device__ __forceinline__ void enter(const AttendArgs& a, int seq, int length) {
        b = seq;
        n = min(max(length, 0), a.limit);
        lo = a.window > 0 && n > a.window ? n - a.window : 0;
        start = lo / TOKENS * TOKENS;
        tiles = (int)(((uint32_t)(n - start) + TOKENS - 1) / TOKENS);
    }
};

// An item's result: sums of columns rel. to the reference m (log2), and their total. A sink beside which the tokens weigh nothing is lse as it
// is, at the ends of 32 bits too, where its base-2 logarithm would be infinite.
__device__ __forceinline__ void finish(const AttendArgs& a, int b, int head, float m, float l, float& inv, float& lse) {
    constexpr float kLog2e = 1.44269504088896340736f;
    if (a.sinks) {
        const float sink = a.sinks[head], log = sink * kLog2e, s = log > -kNone ? -kNone : log < kNone ? kNone : log;
        const float M = fmaxf(m, s), f = ex2_approx(m - M), tokens = l * f;
        l = tokens + ex2_approx(s - M);
        inv = tokens == 0.0f ? 0.0f : f / l;
        lse = tokens == 0.0f ? sink : (M + log2f(l)) * kLn2;
        return;
    }
    inv = l == 0.0f ? 0.0f : 1.0f / l;
    lse = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The results of an empty sequence, whose items are in no CTA's share.
__device__ __forceinline__ void empty(const AttendArgs& a, int b) {
    uint2* const out = reinterpret_cast<uint2*>(a.out + (int64_t)b * a.q.n * a.c.D);
    for (int i = threadIdx.x; i < a.q.n * a.c.D / 4; i += blockDim.x) out[i] = make_uint2(0, 0);
    if (a.lse)
        for (int h = threadIdx.x; h < a.q.n; h += blockDim.x) {
            float inv;
            finish(a, b, h, kNone, 0.0f, inv, a.lse[(int64_t)b * a.q.n + h]);
        }
    if (a.joined == kByItem)
        for (int j = threadIdx.x; j < a.items; j += blockDim.x) reinterpret_cast<Shared*>(a.ws)[b * a.items + j].first = -1;
}

// Four values, times f, to 16 bits.
template <int DT>
__device__ __forceinline__ void store4(uint16_t* to, float4 y, float f) {
    *reinterpret_cast<uint2*>(to) = DT == DT_BF16 ? make_uint2(f32x2_to_bf16x2(y.x * f, y.y * f), f32x2_to_bf16x2(y.z * f, y.w * f))
                                                  : make_uint2(f32x2_to_f16x2(y.x * f, y.y * f), f32x2_to_f16x2(y.z * f, y.w * f));
}

static __device__ uint32_t gave_up;   // CTAs in which a wait ran out of time

// Stores of one CTA of a cluster, read by another.
__device__ __forceinline__ uint32_t in_cta(uint32_t at, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 ld_cluster16(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float ld_cluster4(uint32_t at) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// DIRECT: a cluster of a.split CTAs takes one item, each an equal run of its tiles. Else CTAs take shares of all tiles.
template <int KIND, int DP, int CG, int NT, bool DIRECT>
__global__ void __launch_bounds__(Shape<KIND, DP, CG, NT, DIRECT>::threads, Shape<KIND, DP, CG, NT, DIRECT>::ctas) attend_kernel(const __grid_constant__ AttendArgs a) {
    using S = Shape<KIND, DP, CG, NT, DIRECT>;
    constexpr bool kF8 = S::fp8, kBf = KIND == BF16;
    // A move of the reference leaves the largest w near 2^kRoom (rows' scales counted by their powers of two), and one above kMost is what moves
    // it. fp16 ends at 2^-24, in both parts of p, and at 65504: with 6 weights down to 2^-30 of the largest are in the product (with 0
    // those below 2^-25 were lost: 32768 tokens 17.5 nats under one that the same warps took came to 0), and moves are as rare as
    // with 0 and 512; with 10 and 32768 they cost 61.9 us for 54.1 (32 sequences of 8192, groups of 16, E4M3). bf16 ends where 32 bits do.
    constexpr float kRoom = kBf ? 0.0f : 6.0f, kMost = kBf ? 512.0f : 65504.0f;
    constexpr int kDt = KIND == BF16 || KIND == FP8_BF16 ? DT_BF16 : DT_F16;
    constexpr int kSteps = DP / 16, kCols = CG * NT * 8, kThreads = S::threads;
    extern __shared__ uint8_t raw[];
    uint8_t* const tiles = raw + ((1024 - (tc::smem_addr(raw) & 1023)) & 1023);      // the swizzle goes by 1024 bytes
    __shared__ uint64_t s_bar[kParts][kStages];                  // a tile's copies have landed
    __shared__ uint32_t s_stop;                                  // a wait ran out of time
    volatile uint32_t* const stop = &s_stop;
    __shared__ int sum_part[S::warps];
    __shared__ int share_b, share_n, share_off;
    __shared__ float s_m[kParts][kCols], s_l[kParts][kCols];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int part = warp % kParts, cg = warp / kParts;          // of the tile's tokens, of the columns
    // the warps of a part of the tokens, who share its copies
    auto group_sync = [&]() {
        if (CG == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + part), "n"(CG * 32) : "memory");
    };

    if (threadIdx.x < kParts * kStages) {
        if (threadIdx.x == 0) s_stop = 0;
        // the copy engine's, and where lanes copy each lane's own
        tc::bar_init(tc::smem_addr(&s_bar[0][0] + threadIdx.x), a.boxes ? 1 : 33);
        tc::fence_barrier_init();
    }
    if (a.boxes && threadIdx.x == 0) {
        tc::prefetch_map(&a.km);
        tc::prefetch_map(&a.vm);
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    using W = Walk<S::tokens>;
    W ld;
    int total = 0, G = 1, each = 0, more = 0, from = 0, count = 0, next_n = 0;       // counted in tiles, an item's end as kEnd of them
    const int me = (int)blockIdx.x;
    if (DIRECT) {
        const int rank = a.split > 1 ? (int)cluster_rank() : 0, item = me / a.split, b = item / a.items;
        ld.enter(a, b, a.lengths[b]);
        ld.j = item - b * a.items;
        from = ld.tile = ld.tiles * rank / a.split;
        count = ld.tiles * (rank + 1) / a.split - from;
    } else {
        // The CTA's share of all tiles, and where it begins: each thread sums the tiles of a run of sequences.
        auto tiles_of = [&](int length) {
            W w;
            w.enter(a, 0, length);
            return w.tiles > 0 ? (w.tiles + kEnd) * a.items : 0;
        };
        const int run = (a.B + kThreads - 1) / kThreads, b_from = min((int)threadIdx.x * run, a.B), b_to = min(b_from + run, a.B);
        int mine = 0;
        for (int b = b_from; b < b_to; ++b) mine += tiles_of(a.lengths[b]);
        int before = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, before, d);
            if (lane >= d) before += o;
        }
        if (lane == 31) sum_part[warp] = before;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < S::warps; ++w) {
            if (w < warp) before += sum_part[w];
            total += sum_part[w];
        }
        before -= mine;
        // With fewer tiles than CTAs the last ones have none: no CTA between two that share an item is without a tile.
        G = max(1, min((int)gridDim.x, total));
        each = total / G;
        more = total - each * G;         // the first `more` CTAs take one tile more
        from = me * each + min(me, more);
        count = me >= G ? 0 : each + (me < more ? 1 : 0);
        if (count > 0 && from >= before && from < before + mine) {
            int at = before;
            for (int b = b_from; b < b_to; ++b) {
                const int n = a.lengths[b], next = at + tiles_of(n);
                if (from < next) {
                    share_b = b;
                    share_n = n;
                    share_off = from - at;
                    break;
                }
                at = next;
            }
        }
        __syncthreads();
        for (int b = me; b < a.B; b += (int)gridDim.x)
            if (a.lengths[b] <= 0) empty(a, b);
        if (count == 0) {
            if (a.joined == kByCta && threadIdx.x == 0) reinterpret_cast<Shared*>(a.ws)[blockIdx.x].first = -1;
            return;
        }
        ld.enter(a, share_b, share_n);
        ld.j = share_off / (ld.tiles + kEnd);
        ld.tile = share_off - ld.j * (ld.tiles + kEnd);
        next_n = ld.b + 1 < a.B ? a.lengths[ld.b + 1] : 0;
    }
    ld.head = a.chunks > 1 ? ld.j / a.chunks : ld.j;
    ld.chunk = ld.j - ld.head * a.chunks;

    // The next tile of the share.
    auto advance = [&](W& w, bool ahead) {
        if (++w.tile < w.tiles || DIRECT) return;
        w.tile = 0;
        if (++w.chunk == a.chunks) {
            w.chunk = 0;
            ++w.head;
        }
        if (++w.j < a.items) return;
        w.j = w.head = 0;
        while (w.b + 1 < a.B) {                                  // behind the last: not used
            w.enter(a, w.b + 1, ahead ? next_n : a.lengths[w.b + 1]);
            if (ahead) next_n = w.b + 1 < a.B ? a.lengths[w.b + 1] : 0;
            if (w.tiles > 0) return;
        }
    };
    if (!DIRECT && ld.tile >= ld.tiles) {                        // the share begins in an item's end
        const int rest = ld.tiles + kEnd - ld.tile;
        from += rest;
        count -= rest;
        advance(ld, true);
        if (count <= 0) {
            if (a.joined == kByCta && threadIdx.x == 0) reinterpret_cast<Shared*>(a.ws)[blockIdx.x].first = -1;
            return;
        }
    }
    W cu = ld;
    int left = count;                                            // to copy

    // Copying, by the first warp of each group, in one of two ways. a.boxes, where pages are whole multiples of 16 tokens: boxes of 16
    // tokens, or of all that the warp takes, by 128 bytes, and their scales, which the copy engine brings while the warp computes (their issue by
    // one lane takes 300 to 700 cycles a tile; scales by the lanes 100 more: 8 sequences of 65536, D 64, E4M3: 100 us, so 95). Else 16 bytes a lane and instruction, each lane with the rows of
    // its own token's page: their issue keeps the warp from computing, 700 cycles a tile and more the more of them are under way, but
    // boxes as small as odd pages allow take longer. (8 sequences of 65536, bf16: 271 us by boxes, 288 by lanes; 32 of 8192,
    // pages of one token: 248 by boxes of one, 136 by lanes.)
    const uint32_t base = tc::smem_addr(tiles) + part * S::slot;
    __shared__ uint32_t s_mask[kParts][kStages];
    auto scales_at = [&](int slot) { return tc::smem_addr(tiles) + a.stages * S::step + (slot * kParts + part) * S::scales; };
    auto bar_at = [&](int slot) { return tc::smem_addr(&s_bar[part][slot]); };
    const int64_t v_from_k = a.c.v - a.c.k;
    constexpr int kRowsAt = 32 / S::pieces > 0 ? 32 / S::pieces : 1;              // rows that 32 lanes copy at once
    const int lane_row = kRowsAt > 1 ? lane / S::pieces : 0, piece = lane % S::pieces;
    const bool used = piece * 16 < a.c.D * S::elem;              // columns from D on are filled with zeros
    const int lane_piece = S::piece_at(lane_row, piece);
    // the lane's token of w's tile (of 16 tokens both halves of a warp have the same); behind the last that an int counts: negative, masked
    auto token_of = [&](const W& w) { return w.start + w.tile * S::tokens + part * S::rows + (lane & (S::rows - 1)); };
    auto page_of = [&](const W& w, int on = 0) {                 // of the lane's token, `on` tiles on; -1 where it is masked
        const int t = token_of(w) + on * S::tokens;
        if (t < w.lo || t >= w.n) return -1;
        return a.table[w.b * a.width + quotient(t, a.c.page)];
    };
    // Copies w's tile into a slot; pid: page_of(w), asked for a tile before. Masked rows of a box come with it.
    auto copy = [&](const W& w, int slot, int pid) {
        if (!SGQ_ATTEND_COPIES(w.b * a.items + w.j, part, w.tile)) return;
        const uint32_t at = base + slot * S::step, bar = bar_at(slot);
        const int t = token_of(w);
        const bool there = pid >= 0 && pid < a.c.pages;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there) & S::full;
        const int place = t - (int)(quotient(t, a.c.page) * a.c.page.d);
        if (a.boxes) {
            // each box's tokens lie in one page: that of any that is there, from the place of the first on
            const int n = a.boxes / 16, boxes = S::halves / n;
            int page[S::halves], y[S::halves];
            uint32_t some[S::halves];
#pragma unroll
            for (int h = 0; h < S::halves; ++h) {
                some[h] = boxes == 1 ? (h == 0 ? mask : 0) : (mask >> (16 * h)) & 0xFFFFu;
                page[h] = __shfl_sync(0xFFFFFFFFu, pid, 16 * h + (some[h] ? __ffs(some[h]) - 1 : 0));
                y[h] = __shfl_sync(0xFFFFFFFFu, place, 16 * h);
            }
            if (tc::elect()) {
                s_mask[part][slot] = mask;
                int count = 0;
#pragma unroll
                for (int h = 0; h < S::halves; ++h) count += some[h] ? a.boxes : 0;
                tc::bar_arrive_expect(bar, count * 2 * (DP * S::elem + (kF8 ? 4 : 0)));
#pragma unroll
                for (int h = 0; h < S::halves; ++h) {
                    if (!some[h]) continue;
#pragma unroll
                    for (int b = 0; b < S::blocks; ++b) {
                        const uint32_t to = at + b * S::rows * S::block + h * 16 * S::block;
                        load_4d(to, &a.km, bar, b * S::block, y[h], w.head, page[h]);
                        load_4d(to + S::half, &a.vm, bar, b * S::block, y[h], w.head, page[h]);
                    }
                    if (kF8) {
                        const int64_t row = ((int64_t)page[h] * a.c.heads + w.head) * a.c.page.d + y[h];
                        const uint32_t to = scales_at(slot) + h * 64;
                        load_bytes(to, a.c.ks + row, a.boxes * 4, bar);
                        load_bytes(to + S::rows * 4, a.c.vs + row, a.boxes * 4, bar);
                    }
                }
            }
            __syncwarp();
            return;
        }
        if (lane == 0) {
            s_mask[part][slot] = mask;
            tc::bar_arrive(bar);
        }
        __syncwarp();
        const int64_t off = there ? (int64_t)pid * a.c.ps + (int64_t)w.head * a.c.hs + (int64_t)place * a.c.ts : 0;
#pragma unroll
        for (int i = 0; i < S::rows / kRowsAt; ++i) {
            const int row = i * kRowsAt + lane_row;
            const bool ok = used && ((mask >> row) & 1);
            const uint8_t* k = a.c.k + __shfl_sync(0xFFFFFFFFu, off, row) + piece * 16;
            const uint32_t to = at + i * kRowsAt * S::block + (lane_piece ^ S::turn(i * kRowsAt));
            copy16(to, ok ? k : a.c.k, ok);
            copy16(to + S::half, ok ? k + v_from_k : a.c.k, ok);
        }
        if (kF8 && lane < S::rows) {
            const int64_t row = there ? ((int64_t)pid * a.c.heads + w.head) * a.c.page.d + place : 0;
            const uint32_t to = scales_at(slot) + lane * 4;
            copy4(to, a.c.ks + row, there);
            copy4(to + S::rows * 4, a.c.vs + row, there);
        }
        arrive_with_copies(bar);
    };

    // q of the current item as the right operand of S, and the factors of its columns: asked for, then made ready.
    uint32_t qf[kSteps][NT][2];
    float factor[NT][2];
    auto ask_q = [&](const W& w) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = w.chunk * kCols + (cg * NT + nt) * 8 + g;
            const bool there = col < a.group;
            const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q.p + (int64_t)w.b * a.q.ts + (int64_t)(there ? w.head * a.group + col : 0) * a.q.hs);
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
                // the columns that this lane's pieces of k meet
                const int d0 = kF8 ? (kk >> 2) * 64 + c * 16 + (kk & 3) * 4 : kk * 16 + c * 2, d1 = kF8 ? d0 + 2 : d0 + 8;
                qf[kk][nt][0] = there && d0 < a.c.D ? q[d0 >> 1] : 0u;
                qf[kk][nt][1] = there && d1 < a.c.D ? q[d1 >> 1] : 0u;
            }
        }
    };
    auto ready_q = [&]() {
        constexpr float kLog2e = 1.44269504088896340736f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float up = 1.0f;
            if (KIND == FP8_BF16) {      // bf16 -> fp16 by a power of two a head, its largest value in [1, 2)
                float top = 0.0f;
#pragma unroll
                for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[kk][nt][i] << 16)), fabsf(__uint_as_float(qf[kk][nt][i] & 0xFFFF0000u))));
                top = group_max<4>(top);
                const int e = max(-120, min(120, (int)(__float_as_uint(top) >> 23) - 127));
                const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t v = qf[kk][nt][i];
                        qf[kk][nt][i] = f32x2_to_f16x2(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xFFFF0000u) * down);
                    }
            }
            // column 2c (+ 1)'s factor is held by the lanes of row 2c (+ 1)
            factor[nt][0] = __shfl_sync(0xFFFFFFFFu, up, c * 8) * (a.scale * kLog2e);
            factor[nt][1] = __shfl_sync(0xFFFFFFFFu, up, c * 8 + 4) * (a.scale * kLog2e);
        }
    };

    // sums of w v, and of p. down (E4M3 rows): w = p times the row's scale times down, so the sums of w v are 1 / down of what they stand for
    float o[kSteps][NT][4], ref[NT][2], sum[NT][2], down[NT][2];
    auto clear = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            ref[nt][0] = ref[nt][1] = kNone;
            sum[nt][0] = sum[nt][1] = 0.0f;
            down[nt][0] = down[nt][1] = 1.0f;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.0f;
        }
    };

    auto tile = [&](int slot) {
        constexpr int H = S::halves;
        const uint32_t at = base + slot * S::step, vt = at + S::half, sc = kF8 ? scales_at(slot) : 0;
        const uint32_t mask = s_mask[part][slot];
        // What masked rows of v hold, and their scales, is multiplied by 0: it has to be a number. Each warp of the part writes the zeros that it
        // reads, so that no barrier hangs on the mask: where a wait ran out, the part's warps may have seen unlike ones.
        if (mask != S::full) {
            if (kF8 && lane < S::rows && !((mask >> lane) & 1)) sts_f32(sc + (S::rows + lane) * 4, 0.0f);
            for (int i = lane; i < S::half / 16; i += 32) {
                const int r = i * 16 / S::block % S::rows;
                if (!((mask >> r) & 1)) sts16(vt + i * 16, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
            }
            tc::fence_async_smem();                  // before the copies that come here next
            __syncwarp();
        }
        // S, in two chains of products a tile of 16 by 8
        float x[H][NT][4];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float x2[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[h][nt][i] = x2[nt][i] = 0.0f;
            if (!kF8) {
#pragma unroll
                for (int kk = 0; kk < kSteps; ++kk) {
                    uint32_t k[4];
                    ldmatrix4(k, at + S::piece_at(lane & 15, kk * 2 + (lane >> 4)));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma<kBf>(kk & 1 ? x2[nt] : x[h][nt], k, qf[kk][nt][0], qf[kk][nt][1]);
                }
            } else {
#pragma unroll
                for (int blk = 0; blk < DP / 64; ++blk) {
                    const uint32_t from = at + S::piece_at(h * 16 + g, blk * 4 + c);
                    const uint4 p = lds16(from), q = lds16(from + 8 * S::block);
                    const uint32_t up[4] = {p.x, p.y, p.z, p.w}, dn[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t k[4];
                        widen(up[i], k[0], k[2]);
                        widen(dn[i], k[1], k[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma<false>(i & 1 ? x2[nt] : x[h][nt], k, qf[blk * 4 + i][nt][0], qf[blk * 4 + i][nt][1]);
                    }
                }
            }
            const float k0 = kF8 ? lds_f32(sc + (h * 16 + g) * 4) : 1.0f, k1 = kF8 ? lds_f32(sc + (h * 16 + g + 8) * 4) : 1.0f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[h][nt][i] = (x[h][nt][i] + x2[nt][i]) * (kF8 ? factor[nt][i & 1] * (i < 2 ? k0 : k1) : factor[nt][i & 1]);
        }
        if (mask != S::full) {
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!((mask >> (h * 16 + g + 8 * (i >> 1))) & 1)) x[h][nt][i] = -INFINITY;
        }
        // p, and w = p times the row's v scale, times the column's power of two. Where one is out of bounds (or no number) the reference moves to
        // the largest logit, so that p is 1 at most (16-bit rows: 2^room), and the power to where the largest w is 2^room: they are two, since the scales may be
        // as far apart as 32 bits allow, and the total counts every row the same whatever its scale.
        float vs[H][2], w[H][NT][4], s0[NT], s1[NT];
        bool over = false;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            vs[h][0] = kF8 ? lds_f32(sc + (S::rows + h * 16 + g) * 4) : 1.0f;
            vs[h][1] = kF8 ? lds_f32(sc + (S::rows + h * 16 + g + 8) * 4) : 1.0f;
        }
        auto weigh = [&]() {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                s0[nt] = s1[nt] = 0.0f;
#pragma unroll
                for (int h = 0; h < H; ++h) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[h][nt][i] = ex2_approx(x[h][nt][i] - ref[nt][i & 1]);
                    s0[nt] += w[h][nt][0] + w[h][nt][2];
                    s1[nt] += w[h][nt][1] + w[h][nt][3];
                    if (kF8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[h][nt][i] = w[h][nt][i] * vs[h][i >> 1] * down[nt][i & 1];
                    }
                }
            }
        };
        weigh();
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) over |= !(w[h][nt][i] <= kMost);
        if (kF8) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) over |= !(fmaxf(s0[nt], s1[nt]) <= kMostSum);
        }
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int col = 0; col < 2; ++col) {
                    float top = kF8 ? ref[nt][col] : ref[nt][col] + kRoom;
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int r = 0; r < 2; ++r) top = fmaxf(top, x[h][nt][2 * r + col]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                    if (!kF8) top -= kRoom;
                    const float moved = ref[nt][col] - top;
                    ref[nt][col] = top;
                    sum[nt][col] *= ex2_approx(moved);
                    float f = moved;                             // of the sums of w v, log2
                    if (kF8) {
                        const float old = -exponent(down[nt][col]);              // log2 of what w is divided by
                        float most = old + moved + kRoom;
#pragma unroll
                        for (int h = 0; h < H; ++h)
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                if (vs[h][r] != 0.0f) most = fmaxf(most, x[h][nt][2 * r + col] - top + exponent(vs[h][r]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
                        most = fminf(fmaxf(ceilf(most) - kRoom, kLeastExp), kMostExp);
                        down[nt][col] = power(-most);
                        f += old - most;
                    }
                    f = ex2_approx(f);
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        o[i][nt][col] *= f;
                        o[i][nt][2 + col] *= f;
                    }
                }
            weigh();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            sum[nt][0] += s0[nt];
            sum[nt][1] += s1[nt];
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            uint32_t p[S::parts][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float w0 = w[h][nt][2 * r], w1 = w[h][nt][2 * r + 1];
                    const uint32_t hi = kBf ? f32x2_to_bf16x2(w0, w1) : f32x2_to_f16x2(w0, w1);
                    p[0][nt][r] = transposed(hi);
                    if (S::parts == 2) {
                        const float2 back = kBf ? make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)) : f16x2_to_f32x2(hi);
                        p[S::parts - 1][nt][r] = transposed(kBf ? f32x2_to_bf16x2(w0 - back.x, w1 - back.y) : f32x2_to_f16x2(w0 - back.x, w1 - back.y));
                    }
                }
            if (!kF8) {
                // 8 x 8 pieces of V^T: tokens 0-7 by columns 0-7, columns 8-15, then tokens 8-15
                const int row = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t v[4];
                    ldmatrix4t(v, vt + S::piece_at(row, i * 2 + ((lane >> 3) & 1)));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < S::parts; ++e) mma<kBf>(o[i][nt], v, p[e][nt][0], p[e][nt][1]);
                }
            } else {
                constexpr int kWords = DP >= 128 ? 4 : 2;        // 4 codes of a token each
#pragma unroll
                for (int blk = 0; blk < (DP + 127) / 128; ++blk) {
                    uint32_t v[4][4];                            // tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int row = h * 16 + 2 * c + (t & 1) + (t >> 1) * 8;
                        const uint32_t from = vt + (kWords == 4 ? S::piece_at(row, blk * 8 + g) : S::piece_at(row, g >> 1) + (g & 1) * 8);
                        if (kWords == 4) {
                            const uint4 q = lds16(from);
                            v[t][0] = q.x, v[t][1] = q.y, v[t][2] = q.z, v[t][3] = q.w;
                        } else {
                            const uint2 q = lds8(from);
                            v[t][0] = q.x, v[t][1] = q.y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kWords; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {            // columns 4 i + 2 e, + 1 of the lane's
                            uint32_t m[4];
                            widen(__byte_perm(v[0][i], v[1][i], e ? 0x7362 : 0x5140), m[0], m[1]);
                            widen(__byte_perm(v[2][i], v[3][i], e ? 0x7362 : 0x5140), m[2], m[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int n = 0; n < S::parts; ++n) mma<false>(o[blk * 8 + 2 * i + e][nt], m, p[n][nt][0], p[n][nt][1]);
                        }
                }
            }
        }
    };

    // Where a CTA of a cluster leaves its sums of a column.
    __shared__ float s_M[kCols], s_L[kCols];
    auto part_at = [&](int col, int slot) {
        return (uint32_t)__cvta_generic_to_shared(tiles) + (uint32_t)(slot * S::step + (col >> 3) * S::slot + (col & 7) * S::line);
    };
    // Adds up what the warps have of the item at w and writes it: the result, or this CTA's part of it.
    auto flush = [&](const W& w, int slot, bool begun_here, bool ends_here) {
        const bool whole = DIRECT ? a.split == 1 : begun_here && ends_here;
        float* to_part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + attend_header_bytes()) +
                         (size_t)(2 * blockIdx.x + (begun_here ? 1 : 0)) * attend_part(kCols, DP);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                float l = sum[nt][col];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
                float m = ref[nt][col];
                if (kF8) {
                    // One reference again, the one at which the total is between 1 and 2 (0 where there is no token): the values' means
                    // stay as far inside 32 bits as the rows are, and sums of some thousands of warps too.
                    const float e = l > 0.0f ? exponent(l) : 0.0f, less = power(-e), up = power(-exponent(down[nt][col]));
                    m += e;
                    l *= less;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        o[i][nt][col] = o[i][nt][col] * less * up;
                        o[i][nt][2 + col] = o[i][nt][2 + col] * less * up;
                    }
                }
                if (g == 0) {
                    s_m[part][(cg * NT + nt) * 8 + 2 * c + col] = m;
                    s_l[part][(cg * NT + nt) * 8 + 2 * c + col] = l;
                }
            }
        group_sync();
        constexpr int kEach = kThreads / (8 * S::at_once);       // threads a column, 4 values at a time
#pragma unroll
        for (int turn = 0; turn < NT * CG / S::at_once; ++turn) {
            const int nt = turn % NT, round = turn / NT;
            if (cg / S::at_once == round) {
                const uint32_t own = base + slot * S::step + (cg % S::at_once) * 8 * S::line;
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int col = 2 * c + (e & 1), r = e >> 1;
                        constexpr int kSide = DP >= 128 ? 16 : 8;                // columns of V side by side in a lane (FP8)
                        const int d = kF8 ? (i >> 3) * 128 + g * kSide + 2 * (i & 7) + r : i * 16 + g + 8 * r;
                        sts_f32(own + col * S::line + d * 4, o[i][nt][e]);
                    }
                tc::fence_async_smem();                          // before the copies that come here next
            }
            __syncthreads();
            const int at = threadIdx.x / kEach, col = ((round * S::at_once + (at >> 3)) * NT + nt) * 8 + (at & 7), q = w.chunk * kCols + col;
            if (q < a.group) {
                float M = kNone, f[kParts], L = 0.0f;
#pragma unroll
                for (int v = 0; v < kParts; ++v) M = fmaxf(M, s_m[v][col]);
#pragma unroll
                for (int v = 0; v < kParts; ++v) {
                    f[v] = ex2_approx(s_m[v][col] - M);
                    L += s_l[v][col] * f[v];
                }
                const int qh = w.head * a.group + q;
                float inv = 1.0f, lse = 0.0f;
                if (whole) finish(a, w.b, qh, M, L, inv, lse);
                const uint32_t all = (uint32_t)__cvta_generic_to_shared(tiles) + slot * S::step + at * S::line;
#pragma unroll
                for (int d = (threadIdx.x % kEach) * 4; d < DP; d += kEach * 4) {
                    float4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int v = 0; v < kParts; ++v) {
                        const uint4 u = lds16(all + v * S::slot + d * 4);
                        y.x += __uint_as_float(u.x) * f[v];
                        y.y += __uint_as_float(u.y) * f[v];
                        y.z += __uint_as_float(u.z) * f[v];
                        y.w += __uint_as_float(u.w) * f[v];
                    }
                    if (!whole && DIRECT) {
                        sts16(part_at(col, slot ^ 1) + d * 4, y);
                    } else if (!whole) {
                        *reinterpret_cast<float4*>(to_part + col * DP + d) = y;
                    } else if (d < a.c.D) {
                        store4<kDt>(a.out + ((int64_t)w.b * a.q.n + qh) * a.c.D + d, y, inv);
                    }
                }
                if (threadIdx.x % kEach == 0) {
                    if (!whole && DIRECT) {
                        s_M[col] = M;
                        s_L[col] = L;
                    } else if (!whole) {
                        to_part[kCols * DP + col] = M;
                        to_part[kCols * DP + kCols + col] = L;
                    } else if (a.lse) {
                        a.lse[(int64_t)w.b * a.q.n + qh] = lse;
                    }
                }
            }
            __syncthreads();
        }
    };

    // Turn i copies tile i and computes tile i - a.stages, whose slot that is. One loop, so that the copying's code is there once.
    ask_q(cu);
    const bool copies = cg == 0;
    uint32_t parity = 1;                                         // of the slots' barriers: 0 the first time round
    // a tile's pages are asked for a tile before its copy; where all tiles are one item's, two
    int pid = copies && left > 0 ? page_of(ld) : -1, pid2 = DIRECT && copies && left > 1 ? page_of(ld, 1) : -1, todo = count, slot = 0, issued = 0;
    bool fresh = true, begun_here = cu.tile == 0;                // the item's first tile here; whether it is the item's first
    for (int turn = 0; todo > 0; ++turn) {
        if (turn >= a.stages) {
            // (once one has run out the others do not begin)
            if (!tc::bar_test(bar_at(slot), parity) && !*stop) tc::bar_wait(bar_at(slot), parity, stop, SGQ_ATTEND_WAIT);
            __syncwarp();
            if (fresh) {
                ready_q();
                clear();
                fresh = false;
            }
            tile(slot);
            const bool ends = cu.tile + 1 == cu.tiles;
            const int at = from + count - todo;
            todo -= !DIRECT && ends ? 1 + kEnd : 1;
            if (!DIRECT && (ends || todo <= 0)) {
                const W done = cu;
                if (todo > 0) {
                    advance(cu, false);
                    ask_q(cu);
                }
                flush(done, slot, begun_here, ends);
                // who joins: the entry of the item, by the CTA that begins it, or of this CTA
                if (threadIdx.x == 0 && (a.joined == kByItem ? begun_here : todo <= 0)) {
                    Shared sh = {done.b, done.j, -1, -1};
                    if (begun_here && !ends) {
                        // the item goes on in the next CTAs, to the one that has its last tile
                        const int last = at + (done.tiles - done.tile - 1);
                        sh.first = me;
                        sh.last = last < more * (each + 1) ? last / (each + 1) : more + (last - more * (each + 1)) / each;
                    }
                    reinterpret_cast<Shared*>(a.ws)[a.joined == kByItem ? done.b * a.items + done.j : me] = sh;
                }
                fresh = begun_here = true;
            } else {
                advance(cu, false);
            }
            group_sync();
        }
        if (copies && left > 0 && !__any_sync(0xFFFFFFFFu, *stop)) {
            copy(ld, slot, pid);
            ++issued;
            left -= !DIRECT && ld.tile + 1 == ld.tiles ? 1 + kEnd : 1;
            if (left > 0) {
                advance(ld, true);
                if (!DIRECT) pid = page_of(ld);
            }
            if (DIRECT) {
                pid = pid2;
                pid2 = left > 1 ? page_of(ld, 1) : -1;
            }
        }
        if (++slot == a.stages) {
            slot = 0;
            parity ^= 1;
        }
    }
    // All warps have made their last wait here, and take one way: a CTA in which one of them ran out of time, and another was done
    // before, would else part at the barriers behind.
    if (__syncthreads_or((int)*stop)) {
        // Out of time: what was computed since is no result. The last copies get as long again, so that none lands behind this CTA's
        // end: the i-th went to slot i % stages, in that slot's phase i / stages. (Other phases may never end.)
        uint32_t none = 0;
        if (copies)
            for (int i = max(0, issued - a.stages); i < issued; ++i) tc::bar_wait(bar_at(i % a.stages), (i / a.stages) & 1, &none, SGQ_ATTEND_WAIT);
        __syncthreads();
        if (threadIdx.x == 0) atomicAdd(&gave_up, 1);
    }
    if (fresh) clear();                                          // a CTA of a cluster that had no tile
    if (!DIRECT) return;
    __syncthreads();
    flush(cu, 0, true, true);
    if (a.split == 1) return;
    // The cluster's CTAs each join some of the columns' values.
    cluster_arrive();
    cluster_wait();
    constexpr int kEach = DP / 4;                                // of a column, 4 values each
    for (int u = (int)cluster_rank() * kThreads + (int)threadIdx.x; u < kCols * kEach; u += a.split * kThreads) {
        const int col = u / kEach, d = (u - col * kEach) * 4, q = cu.chunk * kCols + col;
        if (q >= a.group) continue;
        float M = kNone, L = 0.0f;
        float4 y = {0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t at_m = (uint32_t)__cvta_generic_to_shared(&s_M[col]), at_l = (uint32_t)__cvta_generic_to_shared(&s_L[col]), at = part_at(col, 1) + d * 4;
        for (int r = 0; r < a.split; ++r) M = fmaxf(M, ld_cluster4(in_cta(at_m, r)));
#pragma unroll 4
        for (int r = 0; r < a.split; ++r) {
            const float f = ex2_approx(ld_cluster4(in_cta(at_m, r)) - M);
            const float4 v = ld_cluster16(in_cta(at, r));
            L += f * ld_cluster4(in_cta(at_l, r));
            y.x += f * v.x;
            y.y += f * v.y;
            y.z += f * v.z;
            y.w += f * v.w;
        }
        const int qh = cu.head * a.group + q;
        float inv, lse;
        finish(a, cu.b, qh, M, L, inv, lse);
        if (d < a.c.D) store4<kDt>(a.out + ((int64_t)cu.b * a.q.n + qh) * a.c.D + d, y, inv);
        if (d == 0 && a.lse) a.lse[(int64_t)cu.b * a.q.n + qh] = lse;
    }
    cluster_arrive();                                            // no CTA leaves while another reads its sums
    cluster_wait();
}

// Joins the parts of the items that several CTAs share: CTA (x, column) those of the item of entry x. Each warp takes
// every WARPS-th part, four at a time, with a maximum of its own; the warps meet in shared memory. One round of
// reads, bound by its latency, where an item has few parts; 16 warps where it may have many.
template <int DT, int DP, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) attend_join_kernel(const AttendArgs a, int cols) {
    pdl_wait();
    pdl_trigger();
    const Shared sh = reinterpret_cast<const Shared*>(a.ws)[blockIdx.x];
    if (sh.first < 0) return;
    const int col = blockIdx.y, head = sh.j / a.chunks, q = (sh.j - head * a.chunks) * cols + col;
    if (q >= a.group) return;
    __shared__ float s_o[WARPS][DP + 2];                         // sums, then the total and the maximum
    const float* parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + attend_header_bytes());
    const int n = sh.last - sh.first + 1, size = attend_part(cols, DP), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kEach = DP / 32, kAhead = 4;
    float y[kEach] = {}, L = 0.0f, M = kNone;
    for (int i0 = warp; i0 < n; i0 += WARPS * kAhead) {
        float m[kAhead], l[kAhead], v[kAhead][kEach];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * WARPS;
            // the first CTA's part is its second, the others' their first
            const float* p = parts + (size_t)(2 * (sh.first + min(i, n - 1)) + (i == 0 ? 1 : 0)) * size;
            m[k] = i < n ? p[cols * DP + col] : kNone;
            l[k] = i < n ? p[cols * DP + cols + col] : 0.0f;
#pragma unroll
            for (int e = 0; e < kEach; ++e) v[k][e] = i < n ? p[col * DP + e * 32 + lane] : 0.0f;
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) top = fmaxf(top, m[k]);
        const float old = ex2_approx(M - top);
        M = top;
        L *= old;
#pragma unroll
        for (int e = 0; e < kEach; ++e) y[e] *= old;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float f = ex2_approx(m[k] - top);
            L += f * l[k];
#pragma unroll
            for (int e = 0; e < kEach; ++e) y[e] += f * v[k][e];
        }
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) s_o[warp][e * 32 + lane] = y[e];
    if (lane == 0) {
        s_o[warp][DP] = L;
        s_o[warp][DP + 1] = M;
    }
    __syncthreads();
    float f[WARPS];
    M = kNone;
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_o[w][DP + 1]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        f[w] = ex2_approx(s_o[w][DP + 1] - M);
        L += f[w] * s_o[w][DP];
    }
    const int qh = head * a.group + q;
    float inv, lse;
    finish(a, sh.b, qh, M, L, inv, lse);
    for (int d = threadIdx.x; d < a.c.D; d += WARPS * 32) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += f[w] * s_o[w][d];
        const uint32_t r = DT == DT_BF16 ? f32x2_to_bf16x2(v * inv, 0.0f) : f32x2_to_f16x2(v * inv, 0.0f);
        a.out[((int64_t)sh.b * a.q.n + qh) * a.c.D + d] = (uint16_t)r;
    }
    if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)sh.b * a.q.n + qh] = lse;
}

template <int KIND, int DP, int CG, int NT>
cudaError_t launch(const Device& dev, const AttendArgs& args, cudaStream_t stream) {
    constexpr int kDt = KIND == BF16 || KIND == FP8_BF16 ? DT_BF16 : DT_F16;
    AttendArgs a = args;
    using Any = Shape<KIND, DP, CG, NT, true>;
    // Boxes of as many tokens as a warp takes, or 16, whose rows and scales lie in one page.
    a.boxes = a.c.page.d % 16 != 0 || ((uintptr_t)a.c.ks | (uintptr_t)a.c.vs) % 16 != 0 ? 0 : a.c.page.d % Any::rows == 0 ? Any::rows : 16;
    if (a.boxes && (!encode_cache(&a.km, a.c, a.c.k, a.boxes, Any::block, Any::elem) || !encode_cache(&a.vm, a.c, a.c.v, a.boxes, Any::block, Any::elem)))
        return cudaErrorInvalidValue;
    const int64_t sms = dev.sms > 0 ? dev.sms : 152;
    if (a.split > 0) {
        using S = Shape<KIND, DP, CG, NT, true>;
        // Few CTAs have the room to copy many tiles at once; as many as the device holds do better with two tiles of
        // wide rows, eight of narrow ones (200 sequences up to 900, D 64: 11.3 us, with two 12.3).
        const int64_t ctas = (int64_t)a.B * a.items * a.split;
        const int each = ctas <= attend_room(sms, 1, a.split) ? 1 : S::ctas > 2 && ctas <= attend_room(sms, 2, a.split) ? 2 : S::ctas, most = each < S::ctas || DP == 64 ? kStages : 2;
        const int need = (a.tiles + a.split - 1) / a.split;
        a.stages = S::fit(each) < most ? S::fit(each) : most;
        if (a.stages > need) a.stages = need < 2 ? 2 : need;
        return launch_grid(attend_kernel<KIND, DP, CG, NT, true>, dim3((unsigned)ctas), S::threads, S::bytes(a.stages), a.split, dev.id, a, stream);
    }
    using S = Shape<KIND, DP, CG, NT, false>;
    // Two tiles ahead, three where one CTA fills a multiprocessor: three are worse (64 sequences up to 4096, bf16: 84 us and 78; 8 up to 131072, E4M3: 284 and 281).
    a.stages = S::ctas == 1 && S::fit(1) > 2 ? 3 : 2;
    int64_t ctas = sms * S::ctas;
    if (ctas > kAttendCtas) ctas = kAttendCtas;
    const int64_t most = (int64_t)a.B * a.items * a.tiles;
    if (ctas > most) ctas = most;
    const int64_t items = (int64_t)a.B * a.items;
    a.joined = items <= 64 ? kByItem : kByCta;
    const cudaError_t e = launch_grid(attend_kernel<KIND, DP, CG, NT, false>, dim3((unsigned)ctas), S::threads, S::bytes(a.stages), 1, dev.id, a, stream);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.joined == kByItem ? items : ctas), (unsigned)(a.group < CG * NT * 8 ? a.group : CG * NT * 8));
    cfg.blockDim = dim3(a.joined == kByItem ? 512 : 128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.joined == kByItem ? attend_join_kernel<kDt, DP, 16> : attend_join_kernel<kDt, DP, 4>, a, CG * NT * 8);
}

template <int KIND>
cudaError_t launch_kind(const Device& dev, const AttendArgs& a, cudaStream_t stream) {
    const int DP = a.DP, cols = attend_columns(a.group, DP);
    // 16 columns: two tiles of 8 a warp, so that each row is read from shared memory and widened once (8 sequences of 65536, 4 heads, E4M3: 89 us,
    // by two warps side by side 118); heads of 256 have no registers for that.
    if (DP == 64) return cols == 8 ? launch<KIND, 64, 1, 1>(dev, a, stream) : cols == 16 ? launch<KIND, 64, 1, 2>(dev, a, stream) : launch<KIND, 64, 2, 2>(dev, a, stream);
    if (DP == 128) return cols == 8 ? launch<KIND, 128, 1, 1>(dev, a, stream) : cols == 16 ? launch<KIND, 128, 1, 2>(dev, a, stream) : launch<KIND, 128, 2, 2>(dev, a, stream);
    return cols == 8 ? launch<KIND, 256, 1, 1>(dev, a, stream) : launch<KIND, 256, 2, 1>(dev, a, stream);
}

inline cudaError_t read_gave_up(uint32_t* n) { return cudaMemcpyFromSymbol(n, gave_up, sizeof *n); }

cudaError_t launch_bf16(const Device& dev, const AttendArgs& a, cudaStream_t stream);
cudaError_t gave_up_bf16(uint32_t* n);
cudaError_t launch_f16(const Device& dev, const AttendArgs& a, cudaStream_t stream);
cudaError_t gave_up_f16(uint32_t* n);
cudaError_t launch_fp8_bf16(const Device& dev, const AttendArgs& a, cudaStream_t stream);
cudaError_t gave_up_fp8_bf16(uint32_t* n);
cudaError_t launch_fp8_f16(const Device& dev, const AttendArgs& a, cudaStream_t stream);
cudaError_t gave_up_fp8_f16(uint32_t* n);

}  // namespace attend
}  // namespace sgq
