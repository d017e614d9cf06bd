// sgq_attend.cuh -- attention of one new token a sequence over a paged cache
// (include/sgq_cache.h, paged_attention).
//
// Reading the cache bounds it: every key and value row is used by `group` heads
// of q, 4 to 16 operations a byte. One launch gives all CTAs equal shares of the
// cache's tiles, whatever the sequences' lengths; a second joins what several CTAs
// have computed of one sequence.
//
// Shares. An item is a sequence and a head of the cache (a chunk of its group of
// q heads, where there are more than a CTA's columns); its tiles are 64 tokens
// each. All items' tiles stand in one row, and CTA c of G takes those from
// total c / G to total (c + 1) / G. The lengths are summed on the device, so a
// captured graph follows them.
//
// Inside a CTA each of four warps takes 16 tokens of every tile and runs by itself:
// its own asynchronous copies, several tiles ahead and across the items' borders, its own
// running maximum and sums. The warps meet where an item ends, to add up.
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
// The running maximum is a reference that is moved only when a value exceeds it
// by 2^8, so most tiles need no reduction over lanes and no rescaling.
#pragma once

#include "sgq_cache.cuh"

namespace sgq {
namespace attend {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;                        // tokens a warp takes at a time
constexpr float kNone = -3.0e38f;                // below every logit
constexpr float kRoom = 8.0f;                    // log2 of what p may exceed 1 by

// Kinds of rows and queries.
enum Kind : int { BF16 = 0, F16 = 1, FP8_BF16 = 2, FP8_F16 = 3 };

template <int KIND, int DP, int NT>
struct Shape {
    static constexpr bool fp8 = KIND >= FP8_BF16;
    static constexpr int elem = fp8 ? 1 : 2;
    static constexpr int pieces = DP * elem / 16;                // 16-byte pieces of a row
    static constexpr int stride = DP * elem + 16;                // of rows in shared memory: 8 rows' pieces meet no bank twice
    static constexpr int slot = 2 * kRows * stride + (fp8 ? 2 * kRows * 4 : 0);
    static constexpr int budget = 104 * 1024;                    // two CTAs a multiprocessor
    static constexpr int fit = budget / (slot * kWarps);
    static constexpr int stages = fit < 2 ? 2 : fit > 8 ? 8 : fit;
    static constexpr int smem = stages * slot * kWarps;
    static constexpr int parts = KIND == FP8_BF16 ? 1 : 2;       // 16-bit parts of p
    static constexpr int ctas = smem <= 110 * 1024 ? 2 : 1;      // a multiprocessor
    static_assert(8 * (DP + 4) * 4 <= slot, "an item's sums of 8 columns pass through a slot");
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

__device__ __forceinline__ void sts_f32(uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }

// Four E4M3 codes -> two fp16 pairs, exactly.
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}

// floor(log2 s) of a scale, held inside +-100; zero and what is not finite included.
__device__ __forceinline__ float scale_log(float s) {
    const int e = (int)((__float_as_uint(s) >> 23) & 0xFF) - 127;
    return (float)max(-100, min(100, e));
}

// Walks over the tiles of a CTA's share.
struct Walk {
    int b, j;            // sequence, item of it
    int tile, tiles;     // of the item
    int lo, n;           // tokens [lo, n) are not masked
    int start;           // first token of the first tile

    __device__ __forceinline__ void enter(const AttendArgs& a, int seq, int length) {
        b = seq;
        n = min(max(length, 0), a.limit);
        lo = a.window > 0 && n > a.window ? n - a.window : 0;
        start = lo / kAttendTile * kAttendTile;
        tiles = max(1, (n - start + kAttendTile - 1) / kAttendTile);
    }
};

__device__ __forceinline__ int tiles_of(const AttendArgs& a, int length) {
    Walk w;
    w.enter(a, 0, length);
    return w.tiles;
}

// An item's result: sums of columns rel. to the reference m (log2), and their total.
__device__ __forceinline__ void finish(const AttendArgs& a, int b, int head, float m, float l, float& inv, float& lse) {
    constexpr float kLog2e = 1.44269504088896340736f;
    if (a.sinks) {
        const float s = a.sinks[head] * kLog2e, M = fmaxf(m, s), f = ex2_approx(m - M);
        l = l * f + ex2_approx(s - M);
        inv = l > 0.0f ? f / l : 0.0f;
        m = M;
    } else {
        inv = l == 0.0f ? 0.0f : 1.0f / l;
    }
    lse = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int KIND, int DP, int NT>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendArgs a) {
    using S = Shape<KIND, DP, NT>;
    constexpr bool kF8 = S::fp8, kBf = KIND == BF16;
    constexpr int kDt = KIND == BF16 || KIND == FP8_BF16 ? DT_BF16 : DT_F16;
    constexpr int kSteps = DP / 16, kCols = NT * 8;
    extern __shared__ __align__(16) uint8_t stages[];
    __shared__ long long sum_part[kWarps];
    __shared__ long long share_at;
    __shared__ int share_b;
    __shared__ float s_m[kWarps][kCols], s_l[kWarps][kCols];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

    pdl_wait();
    pdl_trigger();

    // The CTA's share of all tiles, and where it begins: each thread sums the tiles of a run of sequences.
    const int run = (a.B + kThreads - 1) / kThreads, b_from = min((int)threadIdx.x * run, a.B), b_to = min(b_from + run, a.B);
    long long mine = 0;
    for (int b = b_from; b < b_to; ++b) mine += tiles_of(a, a.lengths[b]);
    long long before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d) before += o;
    }
    if (lane == 31) sum_part[warp] = before;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sum_part[w];
        total += sum_part[w];
    }
    before -= mine;
    total *= a.items;
    // no CTA between two that share an item is without a tile: with fewer tiles than CTAs the last ones have none
    const long long G = min((long long)gridDim.x, total), me = min((long long)blockIdx.x, G);
    const long long from = total * me / G, to = total * min(me + 1, G) / G;
    if (from >= before * a.items && from < (before + mine) * a.items) {
        long long at = before * a.items;
        for (int b = b_from; b < b_to; ++b) {
            const long long next = at + (long long)tiles_of(a, a.lengths[b]) * a.items;
            if (from < next) {
                share_b = b;
                share_at = at;
                break;
            }
            at = next;
        }
    }
    __syncthreads();
    if (from >= to) {
        if (a.joined && threadIdx.x == 0) reinterpret_cast<Shared*>(a.ws)[blockIdx.x].first = -1;
        return;
    }

    Walk ld;
    ld.enter(a, share_b, a.lengths[share_b]);
    {
        const long long off = from - share_at;
        ld.j = (int)(off / ld.tiles);
        ld.tile = (int)(off - (long long)ld.j * ld.tiles);
    }
    Walk cu = ld;
    long long left = to - from;                                  // tiles to copy
    int next_n = ld.b + 1 < a.B ? a.lengths[ld.b + 1] : 0;

    auto advance = [&](Walk& w, bool ahead) {
        if (++w.tile < w.tiles) return;
        w.tile = 0;
        if (++w.j < a.items) return;
        w.j = 0;
        if (w.b + 1 >= a.B) return;                              // behind the last: not used
        w.enter(a, w.b + 1, ahead ? next_n : a.lengths[w.b + 1]);
        if (ahead) next_n = w.b + 1 < a.B ? a.lengths[w.b + 1] : 0;
    };

    const uint32_t base = (uint32_t)__cvta_generic_to_shared(stages) + warp * S::stages * S::slot;
    __shared__ uint32_t s_mask[kWarps][S::stages];
    auto page_of = [&](const Walk& w) {                          // of the lane's token of w's tile; -1 where it is masked
        const int t = w.start + w.tile * kAttendTile + warp * kRows + (lane & 15);
        if (t < w.lo || t >= w.n) return -1;
        return a.table[w.b * a.width + quotient(t, a.c.page)];
    };
    // Copies w's tile into a slot; pid: page_of(w), asked for a tile before.
    auto copy = [&](const Walk& w, int slot, int pid) {
        const uint32_t at = base + slot * S::slot;
        const int t = w.start + w.tile * kAttendTile + warp * kRows + (lane & 15);
        const int head = w.j / a.chunks;
        const bool there = pid >= 0 && pid < a.c.pages;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there) & 0xFFFFu;
        const int place = there ? t - (int)(quotient(t, a.c.page) * a.c.page.d) : 0;
        const int64_t page = there ? pid : 0;
        const int64_t off = page * a.c.ps + (int64_t)head * a.c.hs + place * a.c.ts;
        if (lane == 0) s_mask[warp][slot] = mask;
        constexpr int kRowsAt = 32 / S::pieces > 0 ? 32 / S::pieces : 1;      // rows that 32 lanes copy at once
        const int used = a.c.D * S::elem / 16;
#pragma unroll
        for (int i = 0; i < kRows * S::pieces / 32; ++i) {
            const int row = i * 32 / S::pieces + (kRowsAt > 1 ? lane / S::pieces : 0);
            const int piece = lane % S::pieces;
            const uint32_t lo = __shfl_sync(0xFFFFFFFFu, (uint32_t)off, row), hi = __shfl_sync(0xFFFFFFFFu, (uint32_t)(off >> 32), row);
            const int64_t o = (int64_t)(((uint64_t)hi << 32) | lo) + piece * 16;
            const bool ok = ((mask >> row) & 1) && piece < used;
            const uint32_t to_k = at + row * S::stride + piece * 16;
            copy16(to_k, a.c.k + (ok ? o : 0), ok);
            copy16(to_k + kRows * S::stride, a.c.v + (ok ? o : 0), ok);
        }
        if (kF8) {
            const int64_t row = (page * a.c.heads + head) * a.c.page.d + place;
            copy4(at + 2 * kRows * S::stride + lane * 4, (lane < 16 ? a.c.ks : a.c.vs) + row, there);
        }
    };

    // q of the current item as the right operand of S, and the factors of its columns.
    uint32_t qf[kSteps][NT][2];
    float factor[NT][2];
    auto load_q = [&](const Walk& w) {
        constexpr float kLog2e = 1.44269504088896340736f;
        const int head = w.j / a.chunks, first = (w.j - head * a.chunks) * kCols;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = first + nt * 8 + g;
            const bool there = col < a.group;
            const uint16_t* q = a.q.p + (int64_t)w.b * a.q.ts + (int64_t)(there ? head * a.group + col : 0) * a.q.hs;
            float top = 0.0f;
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
                // the columns that this lane's pieces of k meet
                const int d0 = kF8 ? (kk >> 2) * 64 + c * 16 + (kk & 3) * 4 : kk * 16 + c * 2, d1 = kF8 ? d0 + 2 : d0 + 8;
                const uint32_t* p = reinterpret_cast<const uint32_t*>(q);
                qf[kk][nt][0] = there && d0 < a.c.D ? p[d0 >> 1] : 0u;
                qf[kk][nt][1] = there && d1 < a.c.D ? p[d1 >> 1] : 0u;
                if (KIND == FP8_BF16) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[kk][nt][i] << 16)), fabsf(__uint_as_float(qf[kk][nt][i] & 0xFFFF0000u))));
                }
            }
            float up = 1.0f;
            if (KIND == FP8_BF16) {      // bf16 -> fp16 by a power of two a head, its largest value in [1, 2)
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

    float o[kSteps][NT][4], ref[NT][2], sum[NT][2];
    auto clear = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            ref[nt][0] = ref[nt][1] = kNone;
            sum[nt][0] = sum[nt][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.0f;
        }
    };

    auto tile = [&](int slot) {
        const uint32_t at = base + slot * S::slot, vt = at + kRows * S::stride, sc = vt + kRows * S::stride;
        const uint32_t mask = s_mask[warp][slot];
        float x[NT][4] = {}, x2[NT][4] = {};         // two chains of products
        if (!kF8) {
            const uint32_t from = at + (lane & 15) * S::stride + (lane >> 4) * 16;
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
                uint32_t k[4];
                ldmatrix4(k, from + kk * 32);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<kBf>(kk & 1 ? x2[nt] : x[nt], k, qf[kk][nt][0], qf[kk][nt][1]);
            }
        } else {
#pragma unroll
            for (int blk = 0; blk < DP / 64; ++blk) {
                const uint4 p = lds16(at + g * S::stride + blk * 64 + c * 16), q = lds16(at + (g + 8) * S::stride + blk * 64 + c * 16);
                const uint32_t up[4] = {p.x, p.y, p.z, p.w}, dn[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t k[4];
                    widen(up[i], k[0], k[2]);
                    widen(dn[i], k[1], k[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma<false>(i & 1 ? x2[nt] : x[nt], k, qf[blk * 4 + i][nt][0], qf[blk * 4 + i][nt][1]);
                }
            }
        }
        float ks[2] = {1.0f, 1.0f}, vs[2] = {1.0f, 1.0f}, lg[2] = {0.0f, 0.0f};
        if (kF8) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                ks[r] = lds_f32(sc + (g + 8 * r) * 4);
                vs[r] = lds_f32(sc + (kRows + g + 8 * r) * 4);
                lg[r] = scale_log(vs[r]);
            }
        }
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = i & 1, r = i >> 1;
                float v = (x[nt][i] + x2[nt][i]) * factor[nt][col];
                if (kF8) v *= ks[r];
                if (!((mask >> (g + 8 * r)) & 1)) v = -INFINITY;
                x[nt][i] = v;
                over |= (kF8 ? v + lg[r] : v) > ref[nt][col] + kRoom;
            }
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int col = 0; col < 2; ++col) {
                    float top = fmaxf(x[nt][col] + lg[0], x[nt][2 + col] + lg[1]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                    top = fmaxf(top, ref[nt][col]);
                    const float f = ex2_approx(ref[nt][col] - top);
                    ref[nt][col] = top;
                    sum[nt][col] *= f;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        o[i][nt][col] *= f;
                        o[i][nt][2 + col] *= f;
                    }
                }
        }
        uint32_t p[S::parts][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float w0 = ex2_approx(x[nt][2 * r] - ref[nt][0]), w1 = ex2_approx(x[nt][2 * r + 1] - ref[nt][1]);
                sum[nt][0] += w0;
                sum[nt][1] += w1;
                if (kF8) {
                    w0 *= vs[r];
                    w1 *= vs[r];
                }
                const uint32_t hi = kBf ? f32x2_to_bf16x2(w0, w1) : f32x2_to_f16x2(w0, w1);
                p[0][nt][r] = transposed(hi);
                if (S::parts == 2) {
                    const float2 back = kBf ? make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)) : f16x2_to_f32x2(hi);
                    p[S::parts - 1][nt][r] = transposed(kBf ? f32x2_to_bf16x2(w0 - back.x, w1 - back.y) : f32x2_to_f16x2(w0 - back.x, w1 - back.y));
                }
            }
        if (!kF8) {
            // 8 x 8 pieces of V^T: tokens 0-7 by columns 0-7, columns 8-15, then tokens 8-15
            const uint32_t from = vt + ((lane & 7) + (lane >> 4) * 8) * S::stride + ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                uint32_t v[4];
                ldmatrix4t(v, from + i * 32);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < S::parts; ++e) mma<kBf>(o[i][nt], v, p[e][nt][0], p[e][nt][1]);
            }
        } else {
            constexpr int kWords = DP >= 128 ? 4 : 2;            // 4 codes of a token each
#pragma unroll
            for (int blk = 0; blk < (DP + 127) / 128; ++blk) {
                uint32_t v[4][4];                                // tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t from = vt + (2 * c + (t & 1) + (t >> 1) * 8) * S::stride + blk * 128 + g * kWords * 4;
                    if (kWords == 4) {
                        const uint4 q = lds16(from);
                        v[t][0] = q.x, v[t][1] = q.y, v[t][2] = q.z, v[t][3] = q.w;
                    } else {
                        const uint2 q = lds8(from);
                        v[t][0] = q.x, v[t][1] = q.y;
                    }
                }
#pragma unroll
                for (int w = 0; w < kWords; ++w)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {                // columns 4 w + 2 e, + 1 of the lane's
                        uint32_t m[4];
                        widen(__byte_perm(v[0][w], v[1][w], e ? 0x7362 : 0x5140), m[0], m[1]);
                        widen(__byte_perm(v[2][w], v[3][w], e ? 0x7362 : 0x5140), m[2], m[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int part = 0; part < S::parts; ++part)
                                mma<false>(o[blk * 8 + 2 * w + e][nt], m, p[part][nt][0], p[part][nt][1]);
                    }
            }
        }
    };

    // Adds up what the warps have of the item at w and writes it: the result, or this CTA's part of it.
    auto flush = [&](const Walk& w, int slot, bool begun_here, bool ends_here) {
        const int head = w.j / a.chunks, first = (w.j - head * a.chunks) * kCols;
        const bool whole = begun_here && ends_here;
        float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + attend_header_bytes()) +
                      (size_t)(2 * blockIdx.x + (begun_here ? 1 : 0)) * attend_part(kCols, DP);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                float l = sum[nt][col];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
                if (g == 0) {
                    s_m[warp][nt * 8 + 2 * c + col] = ref[nt][col];
                    s_l[warp][nt * 8 + 2 * c + col] = l;
                }
            }
        const uint32_t own = base + slot * S::slot;
        constexpr int kLine = (DP + 4) * 4;                      // bytes of a column: 4 lanes' columns meet no bank twice
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = 2 * c + (e & 1), r = e >> 1;
                    constexpr int kEach = DP >= 128 ? 16 : 8;    // columns of V side by side in a lane (FP8)
                    const int d = kF8 ? (i >> 3) * 128 + g * kEach + 2 * (i & 7) + r : i * 16 + g + 8 * r;
                    sts_f32(own + col * kLine + d * 4, o[i][nt][e]);
                }
            __syncthreads();
            // 16 threads a column, 4 values at a time
            const int col = threadIdx.x >> 4, q = first + nt * 8 + col;
            if (q < a.group) {
                float M = kNone, f[kWarps], L = 0.0f;
#pragma unroll
                for (int v = 0; v < kWarps; ++v) M = fmaxf(M, s_m[v][nt * 8 + col]);
#pragma unroll
                for (int v = 0; v < kWarps; ++v) {
                    f[v] = ex2_approx(s_m[v][nt * 8 + col] - M);
                    L += s_l[v][nt * 8 + col] * f[v];
                }
                const int qh = head * a.group + q;
                float inv = 1.0f, lse = 0.0f;
                if (whole) finish(a, w.b, qh, M, L, inv, lse);
                const uint32_t all = (uint32_t)__cvta_generic_to_shared(stages) + slot * S::slot + col * kLine;
#pragma unroll
                for (int d = (threadIdx.x & 15) * 4; d < DP; d += 64) {
                    float4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int v = 0; v < kWarps; ++v) {
                        const uint4 u = lds16(all + v * S::stages * S::slot + d * 4);
                        y.x += __uint_as_float(u.x) * f[v];
                        y.y += __uint_as_float(u.y) * f[v];
                        y.z += __uint_as_float(u.z) * f[v];
                        y.w += __uint_as_float(u.w) * f[v];
                    }
                    if (!whole) {
                        *reinterpret_cast<float4*>(part + (nt * 8 + col) * DP + d) = y;
                    } else if (d < a.c.D) {
                        uint16_t* to = a.out + ((int64_t)w.b * a.q.n + qh) * a.c.D + d;
                        const uint2 v = kDt == DT_BF16 ? make_uint2(f32x2_to_bf16x2(y.x * inv, y.y * inv), f32x2_to_bf16x2(y.z * inv, y.w * inv))
                                                       : make_uint2(f32x2_to_f16x2(y.x * inv, y.y * inv), f32x2_to_f16x2(y.z * inv, y.w * inv));
                        *reinterpret_cast<uint2*>(to) = v;
                    }
                }
                if ((threadIdx.x & 15) == 0) {
                    if (!whole) {
                        part[kCols * DP + nt * 8 + col] = M;
                        part[kCols * DP + kCols + nt * 8 + col] = L;
                    } else if (a.lse) {
                        a.lse[(int64_t)w.b * a.q.n + qh] = lse;
                    }
                }
            }
            __syncthreads();
        }
    };

    // Copies run S::stages tiles ahead, a commit group each (empty behind the last).
    int pid = page_of(ld);
#pragma unroll 1
    for (int s = 0; s < S::stages; ++s) {
        if (left > 0) {
            copy(ld, s, pid);
            if (--left > 0) {
                advance(ld, true);
                pid = page_of(ld);
            }
        }
        cp_async_commit();
    }
    load_q(cu);
    clear();
    bool begun_here = cu.tile == 0;
    long long todo = to - from;
    for (int slot = 0; todo > 0; slot = slot + 1 == S::stages ? 0 : slot + 1) {
        cp_async_wait<S::stages - 1>();
        __syncwarp();
        tile(slot);
        --todo;
        const bool ends = cu.tile + 1 == cu.tiles;
        if (ends || todo == 0) {
            const Walk done = cu;
            if (todo > 0) {
                advance(cu, false);
                load_q(cu);
            }
            flush(done, slot, begun_here, ends);
            if (a.joined && todo == 0 && threadIdx.x == 0) {
                // The item goes on in the next CTAs: the last of them holds its last tile.
                Shared sh = {done.b, done.j, -1, -1};
                if (begun_here && !ends) {
                    const long long last = to + (done.tiles - done.tile - 1) - 1;
                    long long k = last * G / total;
                    while (total * (k + 1) / G <= last) ++k;
                    while (total * k / G > last) --k;
                    sh.first = blockIdx.x;
                    sh.last = (int)k;
                }
                reinterpret_cast<Shared*>(a.ws)[blockIdx.x] = sh;
            }
            clear();
            begun_here = true;
        } else {
            advance(cu, false);
        }
        __syncwarp();
        if (left > 0) {
            copy(ld, slot, pid);
            if (--left > 0) {
                advance(ld, true);
                pid = page_of(ld);
            }
        }
        cp_async_commit();
    }
}

// Joins the parts of the items that several CTAs share: CTA (c, column) those of the item that CTA c of the first launch has begun.
template <int DT, int DP>
__global__ void __launch_bounds__(kThreads) attend_join_kernel(const AttendArgs a, int cols) {
    pdl_wait();
    pdl_trigger();
    const Shared sh = reinterpret_cast<const Shared*>(a.ws)[blockIdx.x];
    if (sh.first < 0) return;
    const int col = blockIdx.y, head = sh.j / a.chunks, q = (sh.j - head * a.chunks) * cols + col;
    if (q >= a.group) return;
    __shared__ float s_m[kThreads], s_o[kWarps][DP + 1];
    const float* parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + attend_header_bytes());
    const int n = sh.last - sh.first + 1, size = attend_part(cols, DP), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the first CTA's part is its second, the others' their first
    auto part = [&](int i) { return parts + (size_t)(2 * (sh.first + i) + (i == 0 ? 1 : 0)) * size; };
    float M = kNone;
    for (int i = threadIdx.x; i < n; i += kThreads) M = fmaxf(M, part(i)[cols * DP + col]);
    s_m[threadIdx.x] = M;
    __syncthreads();
    M = kNone;
    for (int i = 0; i < min(n, kThreads); ++i) M = fmaxf(M, s_m[i]);
    constexpr int kEach = DP / 32;
    float y[kEach] = {}, L = 0.0f;
#pragma unroll 4
    for (int i = warp; i < n; i += kWarps) {
        const float* p = part(i);
        const float f = ex2_approx(p[cols * DP + col] - M);
        L += f * p[cols * DP + cols + col];
#pragma unroll
        for (int e = 0; e < kEach; ++e) y[e] += f * p[col * DP + e * 32 + lane];
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) s_o[warp][e * 32 + lane] = y[e];
    if (lane == 0) s_o[warp][DP] = L;
    __syncthreads();
    L = s_o[0][DP] + s_o[1][DP] + s_o[2][DP] + s_o[3][DP];
    const int qh = head * a.group + q;
    float inv, lse;
    finish(a, sh.b, qh, M, L, inv, lse);
    for (int d = threadIdx.x; d < a.c.D; d += kThreads) {
        const float v = (s_o[0][d] + s_o[1][d] + s_o[2][d] + s_o[3][d]) * inv;
        const uint32_t r = DT == DT_BF16 ? f32x2_to_bf16x2(v, 0.0f) : f32x2_to_f16x2(v, 0.0f);
        a.out[((int64_t)sh.b * a.q.n + qh) * a.c.D + d] = (uint16_t)r;
    }
    if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)sh.b * a.q.n + qh] = lse;
}

template <int KIND, int DP, int NT>
cudaError_t launch(const Device& dev, const AttendArgs& args, cudaStream_t stream) {
    using S = Shape<KIND, DP, NT>;
    AttendArgs a = args;
    const int sms = dev.sms > 0 ? dev.sms : 152;
    // a window may begin anywhere in its first tile
    int64_t tiles = a.limit;
    if (a.window > 0 && tiles > (int64_t)a.window + kAttendTile - 1) tiles = (int64_t)a.window + kAttendTile - 1;
    tiles = tiles <= kAttendTile ? 1 : (tiles + kAttendTile - 1) / kAttendTile;
    int64_t ctas = (int64_t)sms * S::ctas;
    if (ctas > kAttendCtas) ctas = kAttendCtas;
    if (ctas > (int64_t)a.B * a.items * tiles) ctas = (int64_t)a.B * a.items * tiles;
    // where no item has two tiles no two CTAs share one
    a.joined = tiles > 1;
    cudaError_t e = launch_grid(attend_kernel<KIND, DP, NT>, dim3((unsigned)ctas), kThreads, S::smem, 1, dev.id, a, stream);
    if (e != cudaSuccess || !a.joined) return e;
    constexpr int kDt = KIND == BF16 || KIND == FP8_BF16 ? DT_BF16 : DT_F16;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)(a.group < NT * 8 ? a.group : NT * 8));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_join_kernel<kDt, DP>, a, NT * 8);
}

template <int KIND>
cudaError_t launch_kind(const Device& dev, const AttendArgs& a, cudaStream_t stream) {
    const int DP = attend_padded(a.c.D);
    const bool one = attend_columns(a.group) == 8;
    if (DP == 64) return one ? launch<KIND, 64, 1>(dev, a, stream) : launch<KIND, 64, 2>(dev, a, stream);
    if (DP == 128) return one ? launch<KIND, 128, 1>(dev, a, stream) : launch<KIND, 128, 2>(dev, a, stream);
    return one ? launch<KIND, 256, 1>(dev, a, stream) : launch<KIND, 256, 2>(dev, a, stream);
}

cudaError_t launch_bf16(const Device& dev, const AttendArgs& a, cudaStream_t stream);
cudaError_t launch_f16(const Device& dev, const AttendArgs& a, cudaStream_t stream);
cudaError_t launch_fp8_bf16(const Device& dev, const AttendArgs& a, cudaStream_t stream);
cudaError_t launch_fp8_f16(const Device& dev, const AttendArgs& a, cudaStream_t stream);

}  // namespace attend
}  // namespace sgq
