// sgq_lora.cu -- low-rank adapters of many requests, added to a shared
// projection's output (include/sgq_group.h, lora_add).
//
// One launch in plain fp32 for few slots an adapter (below). Else two launches,
// both on the tensor cores (tcgen05) with the slots as the M side, so that a
// thread owns one slot's row of the result:
//
//   shrink   v = x . a^T, tiles of 128 slots x the whole rank. Bound by the
//            reading of x (prefill) or of a (decode), so the length of x is
//            split over the CTAs of a cluster while the tiles are too few to
//            fill the device; the parts are summed through distributed shared
//            memory in the order of the CTAs.
//   expand   y += c (v . b^T), tiles of 128 slots x 128 columns. Bound
//            by reading and writing y.
//
// 8192 rows of 8 adapters, rank 64, K = 4096, N = 8192: 77 us, 20 and 57 (347 MB,
// 51 us at the copy bandwidth); rank 128: 97 us.
//
// v is fp32 between them, in rows of the workspace. The tensor cores multiply
// 16-bit values, so expand splits each v into three, h = round(v), m = round(v -
// h) and l = round(v - h - m), and its product runs over all of them: three
// parts of 8 bits and a sign each hold the 24 bits of v, three of 11 more than
// them. (Two parts of bf16 lose up to 2^-18 of v; made by shrink, they took 73.5 us.)
// fp16 rows are scaled by a power of two first, so that their largest |v| lies in
// [2^14, 2^15): what is left behind l is then at most 2^-39 of it, nothing for the |v|
// from 2^-16 of it up. The row's factor stands behind it.
#include "sgq_group.cuh"
#include "sgq_ragged.cuh"
#include "sgq_tc.cuh"

namespace sgq {

namespace {

constexpr int kM = 128;              // slots a tile
constexpr int kMaxStages = 8;
constexpr int kShrinkThreads = 256;  // warp 0 copies of a, 1 products, 4-7 rows of x, then the result
constexpr int kGather = 128;
constexpr int kLoaders = 128;
constexpr int kSplitters = 256;
constexpr int kExpandThreads = 288 + kLoaders + kSplitters;   // warps 0-7 the sums, 8 copies and products, 9-12 loads of y, 13-20 v
constexpr int kParts = 3;            // 16-bit parts of v

__device__ uint32_t g_gave_up;       // launches in which a wait ran out of time

struct alignas(128) ShrinkParams {
    CUtensorMap ma;                  // a as bytes [groups][R][K], box 128 x R rows
    LoraArgs l;
    int chunks, kbytes, stages, stage_bytes, split;
};

struct alignas(128) ExpandParams {
    CUtensorMap mb;                  // b as bytes [groups][N][R], box 128 x 128 rows
    LoraArgs l;
    int n_tiles;
};

// The token of slot s, or -1 where it is outside or its own slot is another.
__device__ __forceinline__ int64_t token_of(const LoraArgs& l, int s) {
    if (!l.rows) return s;
    const int64_t t = l.rows[s];
    return t >= 0 && t < l.T && l.slots[t] == s ? t : -1;
}

// Barrier `id` of THREADS threads of the block; true when `ok` is in all of them.
template <int THREADS>
__device__ __forceinline__ bool all_agree(int id, bool ok) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)ok), "r"(id), "n"(THREADS)
                 : "memory");
    return r != 0;
}

// fp32 sums over kind::f16 operands: M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_f16(int dt, int n) {
    return (1u << 4) | (dt == DT_BF16 ? (1u << 7) | (1u << 10) : 0) | ((uint32_t)(n >> 3) << 17) | ((kM >> 4) << 24);
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return DT == DT_BF16 ? f32x2_to_bf16x2(lo, hi) : f32x2_to_f16x2(lo, hi);
}

// Shared memory: stages of (x 16 KB, a R x 128 bytes), the parts of v that
// this CTA sums [split][128 / split][R + 4] floats, offsets, barriers.
template <int DT, int BEHIND>
__global__ void __launch_bounds__(kShrinkThreads, 2) lora_shrink_kernel(const __grid_constant__ ShrinkParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    const LoraArgs& l = p.l;
    const int R = l.R, stages = p.stages, ld = R + 4;
    float* parts = reinterpret_cast<float*>(smem + stages * p.stage_bytes);
    int* tokens = reinterpret_cast<int*>(parts + kM * ld);       // of the tile's slots
    float* factors = reinterpret_cast<float*>(tokens + kM);      // of the slots that this CTA sums
    int* lo = reinterpret_cast<int*>(factors + kM);
    int* first = lo + table_ints(l.groups);
    uint64_t* bars = reinterpret_cast<uint64_t*>(first + table_ints(l.groups));
    uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 2);
    int* part = reinterpret_cast<int*>(misc + 4);
    volatile uint32_t* stop = misc + 1;
    const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kMaxStages, acc = empty + 8 * kMaxStages, done = acc + 8;
    const uint32_t stages_at = tc::smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int split = p.split, rank = blockIdx.x % split;
    const int cols = R <= 32 ? 32 : R <= 64 ? 64 : 128;

    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            tc::bar_init(full + 8 * i, 1 + kGather / 32);
            tc::bar_init(empty + 8 * i, 1);
        }
        tc::bar_init(acc, 1);
        tc::bar_init(done, 1);
        tc::fence_barrier_init();
        *stop = 0;
        tc::prefetch_map(&p.ma);
    }
    if (warp == 2) tc::tmem_alloc(tc::smem_addr(misc), cols);
    cluster_arrive_relaxed();
    pdl_wait();
    scan_groups(l.offsets, l.groups, l.S, kM, lo, first, part);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    // the next launch, which holds tensor memory while it waits for this one,
    // may start only now that this CTA has its own
    pdl_trigger();
    cluster_wait();                  // every CTA of the cluster runs: its shared memory may be written
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, misc[0], 0);
    int g, s0, m;
    const bool any = find_tile(lo, first, l.groups, kM, blockIdx.x / split, g, s0, m);   // the same in the whole cluster
    if (any && tid < kM) tokens[tid] = tid < m ? (int)token_of(l, s0 + tid) : -1;
    __syncthreads();
    const int per = (p.chunks + split - 1) / split;
    const int k_from = rank * per, k_to = min(p.chunks, k_from + per);
    const int active = (p.chunks + per - 1) / per;                                   // CTAs that have chunks

    if (any && k_from < k_to) {
        if (warp == 0) {
            int st = 0;
            uint32_t ph = 0;
            int issued = 0;
            bool ok = true;
            for (int kc = k_from; kc < k_to; ++kc) {
                ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(empty + 8 * st, ph ^ 1, stop));
                if (!ok) break;
                if (tc::elect()) {
                    tc::bar_arrive_expect(full + 8 * st, (uint32_t)R * kChunk);
                    tc::load_3d(stages_at + st * p.stage_bytes + kM * kChunk, &p.ma, full + 8 * st, kc * kChunk, 0, g);
                }
                __syncwarp();
                ++issued;
                if (++st == stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!ok) {
                // gave up: wait (a while) for the copies in flight
                for (int i = 0; i < stages && i < issued; ++i) {
                    uint32_t never = 0;
                    if (--st < 0) {
                        st = stages - 1;
                        ph ^= 1;
                    }
                    tc::bar_wait(full + 8 * st, ph, &never, 1 << 27);
                }
            }
        } else if (warp == 1) {
            const uint32_t idesc = idesc_f16(DT, (R + 15) & ~15);
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int kc = k_from; kc < k_to; ++kc) {
                ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(full + 8 * st, ph, stop));
                if (!ok) break;
                tc::fence_after();
                if (tc::elect()) {
                    const uint64_t dx = tc::desc_sw128(stages_at + st * p.stage_bytes);
                    const uint64_t da = tc::desc_sw128(stages_at + st * p.stage_bytes + kM * kChunk);
                    const int left = p.kbytes - kc * kChunk, steps = left >= kChunk ? 4 : (left + 31) / 32;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k >= steps) break;
                        tc::mma_f16(tmem, dx + 2 * k, da + 2 * k, idesc, kc > k_from || k > 0);
                    }
                    tc::commit(empty + 8 * st);
                    if (kc == k_to - 1) tc::commit(acc);
                }
                __syncwarp();
                if (++st == stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!ok) {
                uint32_t never = 0;
                if (tc::elect()) tc::commit(done);
                __syncwarp();
                tc::bar_wait(done, 0, &never, 1 << 27);
            }
        } else if (warp >= 4) {
            // thread u copies 16-byte piece u % 8 of rows u / 8 + 16 i
            const int u = tid - 128, piece = u & 7;
            const uint8_t* src[kM / 16];
#pragma unroll
            for (int i = 0; i < kM / 16; ++i) {
                const int c = (u >> 3) + 16 * i;
                const int64_t t = tokens[c];
                src[i] = t >= 0 ? reinterpret_cast<const uint8_t*>(l.x) + t * p.kbytes + piece * 16 : nullptr;
            }
            int st = 0, lag_st = 0, behind = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto hand_over = [&]() {
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::bar_arrive(full + 8 * lag_st);
                if (++lag_st == stages) lag_st = 0;
                --behind;
            };
            for (int kc = k_from; kc < k_to; ++kc) {
                ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(empty + 8 * st, ph ^ 1, stop));
                if (!ok) break;
                uint8_t* dst = smem + st * p.stage_bytes + (u >> 3) * kChunk + ((piece ^ ((u >> 3) & 7)) << 4);
                const int k = kc * kChunk;
                const bool in = k + piece * 16 < p.kbytes;               // zeros behind the row's end
#pragma unroll
                for (int i = 0; i < kM / 16; ++i)
                    if (src[i]) cp_async16(dst + i * 16 * kChunk, in ? src[i] + k : src[i], in ? 16 : 0);
                cp_async_commit();
                if (++behind > BEHIND) {
                    cp_async_wait<BEHIND>();
                    hand_over();
                }
                if (++st == stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            cp_async_wait<0>();
            while (ok && behind > 0) hand_over();
            ok = __all_sync(0xFFFFFFFFu, ok && tc::bar_wait(acc, 0, stop));
            if (ok) {
                // this thread's slot: its part of v to the CTA that sums the slot
                const int quarter = warp & 3, c = quarter * 32 + lane, share = kM / split;
                tc::fence_after();
                float* to = parts + ((size_t)rank * share + c % share) * ld;
                for (int r0 = 0; r0 < R; r0 += 32) {
                    uint32_t v[32];
                    tc::tmem_load32(tmem + ((uint32_t)quarter << 21) + r0, v);
                    tc::tmem_load_wait(v);
                    if (c < m) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            if (r0 + i < R)
                                st_cluster16(to + r0 + i, (uint32_t)(c / share),
                                             make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                                         __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])));
                    }
                }
                tc::fence_before();
            }
        }
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (any) {
        const int share = kM / split, mine = min(share, m - rank * share);       // slots that this CTA sums
        auto sum4 = [&](int c, int r) {                  // v[r .. r + 3] of slot c, the parts in the order of the CTAs
            const float* from = parts + (size_t)c * ld + r;
            float4 f = *reinterpret_cast<const float4*>(from);
            for (int q = 1; q < active; ++q) {
                const float4 o = *reinterpret_cast<const float4*>(from + (size_t)q * share * ld);
                f.x += o.x, f.y += o.y, f.z += o.z, f.w += o.w;
            }
            return f;
        };
        if (DT == DT_F16) {
            if (tid < mine) {
                float top = 0.0f;
                for (int r = 0; r < R; r += 4) {
                    const float4 f = sum4(tid, r);
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w))));
                }
                // 2^e with top / 2^e in [2^14, 2^15), e held to where both powers are normal
                const int e = min(max((int)(__float_as_uint(top) >> 23) - 14, 27), 227);
                factors[tid] = __uint_as_float((uint32_t)e << 23);
            }
            __syncthreads();
        }
        const int pieces = R / 8;
        for (int i = tid; i < mine * pieces; i += kShrinkThreads) {
            const int c = i / pieces, r = (i - c * pieces) * 8;
            uint8_t* row = static_cast<uint8_t*>(l.v) + (int64_t)(s0 + rank * share + c) * lora_row_bytes(R);
            *reinterpret_cast<float4*>(row + 4 * r) = sum4(c, r);
            *reinterpret_cast<float4*>(row + 4 * r + 16) = sum4(c, r + 4);
            if (DT == DT_F16 && r == 0) *reinterpret_cast<float*>(row + 4 * R) = factors[c];
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 2) tc::tmem_free(tmem, cols);
    if (tid == 0 && *stop) atomicAdd(&g_gave_up, 1);
}

// A tile of y: 128 slots x 128 columns, in shared memory in rows of 272 bytes
// (the 16 over let a warp read 32 rows' same columns without bank conflicts).
// VC chunks of 128 bytes hold R values.
template <int VC>
struct ExpandCfg {
    static constexpr int kNT = 128, kPitch = 2 * kNT + 16;
    static constexpr int kB = kNT * kChunk, kV = kM * kChunk, kY = kM * kPitch;
    static constexpr int kBufs = VC == 1 ? 2 : 1;                    // of b: the next tile's under this one's
    static constexpr int kYBufs = VC == 1 ? 4 : 2;                   // of y: loads one or three tiles ahead
    static constexpr int kVAt = kBufs * VC * kB;                     // [kParts][VC]
    static constexpr int kYAt = kVAt + kParts * VC * kV;
    static constexpr int kTokensAt = kYAt + kYBufs * kY;
    static constexpr int kTablesAt = kTokensAt + kYBufs * 4 * kM;
    static int smem(int groups) { return kTablesAt + 2 * 4 * table_ints(groups) + 256; }
    static_assert(kTablesAt + 2 * 4 * table_ints(kMaxGroups) + 256 <= kMaxDynamicSmem, "tile too large");
};

// The tiles of one CTA: a piece of their list, in which the columns' tiles of
// one set of slots follow one another, so that a CTA mostly keeps its slots
// (their tokens and v) from tile to tile.
struct ExpandWalk {
    const int* lo;
    const int* first;
    int G, n_tiles, nt;
    int64_t tile, end;
    int q, g, s0, m, n0;
    bool fresh;                      // other slots than the tile before
    __device__ ExpandWalk(const int* lo_, const int* first_, int G_, int n_tiles_, int nt_)
        : lo(lo_), first(first_), G(G_), n_tiles(n_tiles_), nt(nt_), q(-1) {
        const int64_t all = (int64_t)first_[G_] * n_tiles_;
        tile = all * blockIdx.x / gridDim.x;
        end = all * (blockIdx.x + 1) / gridDim.x;
    }
    __device__ bool next() {
        if (tile >= end) return false;
        const int at = (int)(tile / n_tiles);
        n0 = (int)(tile - (int64_t)at * n_tiles) * nt;
        fresh = at != q;
        if (fresh) find_tile(lo, first, G, kM, at, g, s0, m);
        q = at;
        ++tile;
        return true;
    }
};

template <int DT, int VC>
__global__ void __launch_bounds__(kExpandThreads, 1) lora_expand_kernel(const __grid_constant__ ExpandParams p) {
    using C = ExpandCfg<VC>;
    constexpr int NT = C::kNT;
    extern __shared__ __align__(1024) uint8_t smem[];        // the swizzle counts in pieces of 1024
    const LoraArgs& l = p.l;
    int* tokens = reinterpret_cast<int*>(smem + C::kTokensAt);           // [kYBufs][128]
    int* lo = reinterpret_cast<int*>(smem + C::kTablesAt);
    int* first = lo + table_ints(l.groups);
    uint64_t* bars = reinterpret_cast<uint64_t*>(first + table_ints(l.groups));
    uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 16);
    int* part = reinterpret_cast<int*>(misc + 4);
    volatile uint32_t* stop = misc + 1;
    const uint32_t full_b = tc::smem_addr(bars), full_v = full_b + 16, acc = full_v + 8, acc_empty = acc + 16;
    const uint32_t y_full = acc_empty + 16, y_empty = y_full + 32, v_empty = y_empty + 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), R = l.R;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(full_b + 8 * i, 1);
            tc::bar_init(acc + 8 * i, 1);
            tc::bar_init(acc_empty + 8 * i, 4);
        }
        tc::bar_init(full_v, kSplitters / 32);
        tc::bar_init(v_empty, 1);
        for (int i = 0; i < C::kYBufs; ++i) {
            tc::bar_init(y_full + 8 * i, kLoaders + kLoaders / 32);
            tc::bar_init(y_empty + 8 * i, 4);
        }
        tc::fence_barrier_init();
        *stop = 0;
        tc::prefetch_map(&p.mb);
    }
    // The shrink launch before this one lets it start after it has waited for
    // everything before itself, and writes the workspace alone: all but the
    // workspace may be read before the wait.
    if (warp == 8) tc::tmem_alloc(tc::smem_addr(misc), 2 * NT);
    scan_groups(l.offsets, l.groups, l.S, kM, lo, first, part);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, misc[0], 0);
    ExpandWalk walk(lo, first, l.groups, p.n_tiles, NT);
    if (warp >= 9 + kLoaders / 32) {
        // ------------------------------------- v: fp32 rows -> three 16-bit parts
        // thread u takes pieces u, u + 256, ... of 8 values of the tile's rows; an odd
        // last piece is filled up with zeros (a product takes 16 values). Eight warps,
        // so that at rank 64 all of it is read before the parts are free (four: 78.4 us
        // for 77.1, 8192 rows of 8 adapters, K = 4096, N = 8192; rank 128 100 for 97).
        const int u = tid - 288 - kLoaders, pieces = (R / 8 + 1) & ~1, all = kM * pieces;
        bool ok = true;
        uint32_t vs = 0;                                                 // sets of slots so far
        pdl_wait();
        pdl_trigger();
        while (ok && walk.next()) {
            if (!walk.fresh) continue;
            bool free = vs == 0;
            for (int j0 = 0; j0 < all; j0 += 4 * kSplitters) {
                float v[4][8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int j = j0 + q * kSplitters + u, c = j / pieces, r = (j - c * pieces) * 8;
                    const bool in = j < all && c < walk.m && r < R;
                    const uint8_t* row = static_cast<const uint8_t*>(l.v) + (int64_t)(walk.s0 + (in ? c : 0)) * lora_row_bytes(R);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 f = in ? __ldcg(reinterpret_cast<const float4*>(row + 4 * r) + h) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        v[q][4 * h] = f.x, v[q][4 * h + 1] = f.y, v[q][4 * h + 2] = f.z, v[q][4 * h + 3] = f.w;
                    }
                    if (DT == DT_F16) {
                        const float factor = in ? __ldcg(reinterpret_cast<const float*>(row + 4 * R)) : 1.0f;
                        const float down = __uint_as_float((254u << 23) - __float_as_uint(factor));       // 1 / factor
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[q][k] *= down;
                    }
                }
                if (!free) {         // the products are done with the parts of the set before
                    ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(v_empty, (vs - 1) & 1, stop));
                    if (!ok) break;
                    free = true;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int j = j0 + q * kSplitters + u, c = j / pieces, piece = j - c * pieces;
                    if (j >= all) break;
                    uint8_t* to = smem + C::kVAt + (piece >> 3) * C::kV + c * kChunk + (((piece ^ c) & 7) << 4);
#pragma unroll
                    for (int h = 0; h < kParts; ++h) {
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 8; k += 2) {
                            const float a0 = round_io<DT>(v[q][k]), a1 = round_io<DT>(v[q][k + 1]);
                            o[k / 2] = pack2<DT>(a0, a1);
                            v[q][k] -= a0;
                            v[q][k + 1] -= a1;
                        }
                        *reinterpret_cast<uint4*>(to + h * VC * C::kV) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            tc::fence_async_smem();
            __syncwarp();
            if (ok && lane == 0) tc::bar_arrive(full_v);
            ++vs;
        }
    } else if (warp > 8) {
        // ------------------------------------------------------- loads of y
        const int u = tid - 288, piece = u & 15;
        bool ok = true;
        int t = -1;
        for (uint32_t i = 0; walk.next(); ++i) {
            const uint32_t buf = i % C::kYBufs;
            if (walk.fresh) t = u < walk.m ? (int)token_of(l, walk.s0 + u) : -1;
            ok = tc::bar_wait(y_empty + 8 * buf, ((i / C::kYBufs) & 1) ^ 1, stop);
            int* tk = tokens + buf * kM;
            if (ok) tk[u] = t;
            if (!all_agree<kLoaders>(1, ok)) break;
            if (lane == 0) tc::bar_arrive(y_full + 8 * buf);             // the tokens; the copies arrive by themselves
            uint8_t* to = smem + C::kYAt + buf * C::kY + piece * 16;
            const int n = walk.n0 + piece * 8;
#pragma unroll
            for (int j = 0; j < kM / 8; ++j) {
                const int c = (u >> 4) + 8 * j, row = tk[c];
                if (row >= 0 && n < l.N) cp_async16(to + c * C::kPitch, l.y + (int64_t)row * l.N + n, 16);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(y_full + 8 * buf) : "memory");
        }
        cp_async_wait<0>();
        pdl_wait();
        pdl_trigger();
    } else if (warp == 8) {
        // ------------------------------------------------ copies of b, products
        const uint32_t at = tc::smem_addr(smem), v_at = at + C::kVAt;
        auto load_b = [&](const ExpandWalk& w, uint32_t i) {             // tile i's rows of b into buffer i % kBufs
            if (tc::elect()) {
                const uint32_t bar = full_b + 8 * (i % C::kBufs), to = at + (i % C::kBufs) * VC * C::kB;
                tc::bar_arrive_expect(bar, VC * C::kB);
#pragma unroll
                for (int c = 0; c < VC; ++c) tc::load_3d(to + c * C::kB, &p.mb, bar, c * kChunk, w.n0, w.g);
            }
            __syncwarp();
        };
        ExpandWalk ahead = walk;
        bool more = ahead.next();
        if (more) load_b(ahead, 0);
        pdl_wait();
        pdl_trigger();
        bool ok = true;
        uint32_t vs = 0;                                                 // sets of slots so far
        for (uint32_t i = 0; ok && walk.next(); ++i) {
            const uint32_t buf = i & 1;
            // the product before is done with the other buffer of b
            if (i > 0) ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(acc + 8 * (buf ^ 1), ((i - 1) >> 1) & 1, stop));
            if (!ok) break;
            if (walk.fresh) {
                if (i > 0 && tc::elect()) tc::bar_arrive(v_empty);       // and with the other slots' v
                __syncwarp();
                ++vs;
            }
            if (C::kBufs == 1) {
                if (i > 0) load_b(walk, i);
                more = false;
            } else {
                more = ahead.next();
                if (more) load_b(ahead, i + 1);
            }
            ok = tc::bar_wait(full_v, (vs - 1) & 1, stop) &&
                 tc::bar_wait(full_b + 8 * (i % C::kBufs), (i / C::kBufs) & 1, stop) &&
                 tc::bar_wait(acc_empty + 8 * buf, ((i >> 1) & 1) ^ 1, stop);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) {
                // gave up: wait (a while) for the copies in flight
                uint32_t never = 0;
                tc::bar_wait(full_b + 8 * (i % C::kBufs), (i / C::kBufs) & 1, &never, 1 << 27);
                never = 0;
                if (more) tc::bar_wait(full_b + 8 * ((i + 1) % C::kBufs), ((i + 1) / C::kBufs) & 1, &never, 1 << 27);
                break;
            }
            tc::fence_after();
            if (tc::elect()) {
                const uint32_t idesc = idesc_f16(DT, NT), b_at = at + (i % C::kBufs) * VC * C::kB;
                const int steps = (R + 15) / 16;                         // of 16 values
#pragma unroll
                for (int h = 0; h < kParts; ++h)
#pragma unroll
                    for (int k = 0; k < 4 * VC; ++k) {
                        if (k >= steps) break;
                        tc::mma_f16(tmem + buf * NT, tc::desc_sw128(v_at + (h * VC + k / 4) * C::kV) + 2 * (k % 4),
                                    tc::desc_sw128(b_at + (k / 4) * C::kB) + 2 * (k % 4), idesc, h > 0 || k > 0);
                    }
                tc::commit(acc + 8 * buf);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------- sums: the 128 columns of slot c a thread.
        // Warps 0-3 take the even tiles and 4-7 the odd ones, so that the waits
        // and barriers of one overlap the other's work (all eight on each tile:
        // 54 us for 8192 rows of 8192 and rank 64).
        const int quarter = warp & 3, group = warp >> 2, u = tid & 127, c = u, piece = u & 15;
        float f = 0.0f;
        int seen = -1;
        pdl_wait();
        for (uint32_t i = 0; walk.next(); ++i) {
            if ((i & 1) != (uint32_t)group) continue;
            const uint32_t buf = i & 1, y_buf = i % C::kYBufs;
            uint8_t* y = smem + C::kYAt + y_buf * C::kY;
            const int* tk = tokens + y_buf * kM;
            if (walk.q != seen) {
                seen = walk.q;
                f = l.scaling ? l.scaling[walk.g] : 1.0f;
                if (DT == DT_F16 && c < walk.m)
                    f *= *reinterpret_cast<const float*>(static_cast<const uint8_t*>(l.v) +
                                                         (int64_t)(walk.s0 + c) * lora_row_bytes(R) + 4 * R);
            }
            const bool ok = tc::bar_wait(y_full + 8 * y_buf, (i / C::kYBufs) & 1, stop) && tc::bar_wait(acc + 8 * buf, (i >> 1) & 1, stop);
            if (!all_agree<128>(2 + group, ok)) break;
            tc::fence_after();
            uint4* row = reinterpret_cast<uint4*>(y + c * C::kPitch);
#pragma unroll
            for (int h = 0; h < NT / 32; ++h) {
                uint32_t v[32];
                tc::tmem_load32(tmem + ((uint32_t)quarter << 21) + buf * NT + 32 * h, v);
                tc::tmem_load_wait(v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 was = row[4 * h + j];
                    float o[8];
                    load8<DT>(was, o);
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = fmaf(f, __uint_as_float(v[8 * j + k]), o[k]);
                    row[4 * h + j] = pack8<DT>(o);
                }
            }
            tc::fence_before();
            asm volatile("bar.sync %0, 128;" ::"r"(2 + group) : "memory");     // the tile's rows are done
            if (lane == 0) tc::bar_arrive(acc_empty + 8 * buf);
            const int n = walk.n0 + piece * 8;
#pragma unroll
            for (int j = 0; j < kM / 8; ++j) {
                const int r = (u >> 4) + 8 * j, t = tk[r];
                if (t >= 0 && n < l.N)
                    st16_if(l.y + (int64_t)t * l.N + n, *reinterpret_cast<const uint4*>(y + r * C::kPitch + piece * 16), true);
            }
            __syncwarp();
            if (lane == 0) tc::bar_arrive(y_empty + 8 * y_buf);
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 8) tc::tmem_free(tmem, 2 * NT);
    if (tid == 0 && *stop) atomicAdd(&g_gave_up, 1);
}

// ------------------------------------------------ few slots an adapter
//
// A decode batch: one or a few slots an adapter, so that the tensor cores'
// tiles of 128 slots would be empty and their latency most of the time. Plain
// fp32 arithmetic instead, in one launch: a cluster of 8 CTAs takes up to 8
// slots of one adapter, each CTA an eighth of the ranks (every value of a is read
// once for all slots), then, v having gone round through distributed shared
// memory, an eighth of the columns of y. As two launches with v in the
// workspace, 64 rows of 32 adapters (rank 16, K = N = 4096) took 8.0 us in a
// graph, against 9.4, but 19.8 as a call from Python, against 9.9.

constexpr int kFew = 8;              // slots a tile
constexpr int kFewCtas = 8;          // of a cluster
constexpr int kFewThreads = 256;

template <int DT>
__global__ void __launch_bounds__(kFewThreads) lora_few_kernel(const LoraArgs l) {
    extern __shared__ int few_smem[];
    int* lo = few_smem;
    int* first = lo + table_ints(l.groups);
    __shared__ __align__(16) float v[kFew][kMaxRank];
    __shared__ float sums[kFewThreads / 32][kFew];
    __shared__ int part[kFewThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster_rank();
    cluster_arrive_relaxed();
    pdl_wait();
    pdl_trigger();
    scan_groups(l.offsets, l.groups, l.S, kFew, lo, first, part);
    cluster_wait();                  // every CTA of the cluster runs: its shared memory may be written
    int g, s0, m;
    if (!find_tile(lo, first, l.groups, kFew, blockIdx.x / kFewCtas, g, s0, m)) return;     // the whole cluster
    const int64_t mine = lane < m ? token_of(l, s0 + lane) : -1;
    int64_t t[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i) t[i] = __shfl_sync(0xFFFFFFFFu, mine, i);

    // this CTA's columns, two a thread at a time; the first ones' values are read ahead
    const int columns = (l.N / 2 + kFewCtas - 1) / kFewCtas * 2, n_to = min(l.N, (rank + 1) * columns);
    int n = rank * columns + 2 * tid;
    uint32_t old[kFew];
    uint4 b0 = {}, b1 = {};
    auto read = [&]() {
        if (n >= n_to) return;
#pragma unroll
        for (int i = 0; i < kFew; ++i)
            if (t[i] >= 0) old[i] = *reinterpret_cast<const uint32_t*>(l.y + t[i] * l.N + n);
        const uint16_t* b = l.b + ((int64_t)g * l.N + n) * l.R;
        b0 = *reinterpret_cast<const uint4*>(b);
        b1 = *reinterpret_cast<const uint4*>(b + l.R);
    };
    read();

    // v of two ranks at a time, four warps each, a quarter of K a warp
    for (int r0 = 2 * rank; r0 < l.R; r0 += 2 * kFewCtas) {
        const uint16_t* a = l.a + ((int64_t)g * l.R + r0 + warp / 4) * l.K;
        float sum[kFew] = {};
        const int chunks = l.K / 8, per = (chunks + 3) / 4, from = (warp & 3) * per, to = min(chunks, from + per);
#pragma unroll 4
        for (int c = from + lane; c < to; c += 32) {
            float fa[8];
            load8<DT>(*reinterpret_cast<const uint4*>(a + 8 * c), fa);
#pragma unroll
            for (int i = 0; i < kFew; ++i) {
                if (t[i] >= 0) {
                    float fx[8];
                    load8<DT>(*reinterpret_cast<const uint4*>(l.x + t[i] * l.K + 8 * c), fx);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[i] = fmaf(fa[j], fx[j], sum[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
#pragma unroll
            for (int d = 16; d; d >>= 1) sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], d);
            if (lane == 0) sums[warp][i] = sum[i];
        }
        __syncthreads();
        if (tid < 2 * kFew * kFewCtas) {
            const int i = tid % kFew, k = tid / kFew % 2;
            st_cluster4(&v[i][r0 + k], (uint32_t)(tid / (2 * kFew)),
                        (sums[4 * k][i] + sums[4 * k + 1][i]) + (sums[4 * k + 2][i] + sums[4 * k + 3][i]));
        }
        __syncthreads();
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();

    const float scale = l.scaling ? l.scaling[g] : 1.0f;
    while (n < n_to) {
        const uint16_t* b = l.b + ((int64_t)g * l.N + n) * l.R;
        float acc[kFew][2] = {};
        for (int r = 0; r < l.R; r += 8) {
            float f0[8], f1[8];
            load8<DT>(b0, f0);
            load8<DT>(b1, f1);
            if (r + 8 < l.R) {
                b0 = *reinterpret_cast<const uint4*>(b + r + 8);
                b1 = *reinterpret_cast<const uint4*>(b + l.R + r + 8);
            }
#pragma unroll
            for (int i = 0; i < kFew; ++i)
                if (i < m) {
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(&v[i][r + j]);
                        acc[i][0] = fmaf(w.x, f0[j], fmaf(w.y, f0[j + 1], fmaf(w.z, f0[j + 2], fmaf(w.w, f0[j + 3], acc[i][0]))));
                        acc[i][1] = fmaf(w.x, f1[j], fmaf(w.y, f1[j + 1], fmaf(w.z, f1[j + 2], fmaf(w.w, f1[j + 3], acc[i][1]))));
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < kFew; ++i)
            if (t[i] >= 0) {
                const float2 was = DT == DT_BF16 ? make_float2(__uint_as_float(old[i] << 16), __uint_as_float(old[i] & 0xFFFF0000u))
                                                 : f16x2_to_f32x2(old[i]);
                *reinterpret_cast<uint32_t*>(l.y + t[i] * l.N + n) =
                    pack2<DT>(fmaf(scale, acc[i][0], was.x), fmaf(scale, acc[i][1], was.y));
            }
        n += 2 * kFewThreads;
        read();
    }
}

template <int DT>
cudaError_t run_few(const Device& dev, const LoraArgs& l, cudaStream_t stream) {
    const int64_t tiles = (int64_t)l.S / kFew + (l.S < l.groups ? l.S : l.groups);   // at most
    if (tiles > 0x7FFFFFFF / kFewCtas) return cudaErrorInvalidConfiguration;
    return launch_grid(lora_few_kernel<DT>, dim3((unsigned)(tiles * kFewCtas)), kFewThreads, 2 * 4 * table_ints(l.groups),
                       kFewCtas, dev.id, l, stream);
}

template <int DT, int BEHIND>
cudaError_t shrink(const Device& dev, ShrinkParams& p, int64_t tiles, int smem, cudaStream_t stream) {
    const int64_t ctas = tiles * p.split;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_grid(lora_shrink_kernel<DT, BEHIND>, dim3((unsigned)ctas), kShrinkThreads, smem, p.split, dev.id, p, stream);
}

template <int DT, int VC>
cudaError_t expand(const Device& dev, ExpandParams& p, int64_t tiles, cudaStream_t stream) {
    using C = ExpandCfg<VC>;
    const LoraArgs& l = p.l;
    const cuuint64_t bd[3] = {(cuuint64_t)(2 * l.R), (cuuint64_t)l.N, (cuuint64_t)l.groups};
    if (!encode_rows(&p.mb, l.b, 3, bd, C::kNT)) return cudaErrorInvalidValue;
    p.n_tiles = (l.N + C::kNT - 1) / C::kNT;
    const int64_t most = tiles * p.n_tiles, room = dev.sms > 0 ? dev.sms : 1;
    return launch_grid(lora_expand_kernel<DT, VC>, dim3((unsigned)(most < room ? most : room)), kExpandThreads,
                       C::smem(l.groups), 1, dev.id, p, stream);
}

template <int DT>
cudaError_t run(const Device& dev, const LoraArgs& l, cudaStream_t stream) {
    if (lora_few(l.S, l.groups, l.R)) return run_few<DT>(dev, l, stream);
    ShrinkParams p;
    p.l = l;
    p.kbytes = 2 * l.K;
    p.chunks = (p.kbytes + kChunk - 1) / kChunk;
    p.stage_bytes = (kM + l.R) * kChunk;
    const cuuint64_t ad[3] = {(cuuint64_t)p.kbytes, (cuuint64_t)l.R, (cuuint64_t)l.groups};
    if (!encode_rows(&p.ma, l.a, 3, ad, l.R)) return cudaErrorInvalidValue;
    const int64_t tiles = (int64_t)l.S / kM + (l.S < l.groups ? l.S : l.groups);     // at most
    const int fixed = 1024 + 4 * kM * (l.R + 4) + 2 * 4 * kM + 2 * 4 * table_ints(l.groups) + 512;
    // two CTAs a multiprocessor where at least 5 stages of each fit
    const bool two = (kMaxDynamicSmem - 2048) / 2 - fixed >= 5 * p.stage_bytes;
    p.stages = ((two ? (kMaxDynamicSmem - 2048) / 2 : kMaxDynamicSmem) - fixed) / p.stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    // the length of x over a cluster while all the tiles' parts are resident
    // at once and a CTA keeps at least 4 chunks
    p.split = 1;
    while (p.split < kMaxCluster && tiles * p.split * 2 <= (two ? 2 : 1) * dev.sms && p.chunks >= 8 * p.split) p.split *= 2;
    const int smem = fixed + p.stages * p.stage_bytes;
    cudaError_t e = p.stages >= 7 ? shrink<DT, 5>(dev, p, tiles, smem, stream) : shrink<DT, 3>(dev, p, tiles, smem, stream);
    if (e != cudaSuccess) return e;
    ExpandParams q;
    q.l = l;
    return l.R <= 64 ? expand<DT, 1>(dev, q, tiles, stream) : expand<DT, 2>(dev, q, tiles, stream);
}

}  // namespace

cudaError_t lora_gave_up(uint32_t* n) { return cudaMemcpyFromSymbol(n, g_gave_up, sizeof *n); }

cudaError_t launch_lora(int dt, const Device& dev, const LoraArgs& a, cudaStream_t stream) {
    return dt == DT_F16 ? run<DT_F16>(dev, a, stream) : run<DT_BF16>(dev, a, stream);
}

}  // namespace sgq
