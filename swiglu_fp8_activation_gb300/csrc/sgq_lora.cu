// sgq_lora.cu -- low-rank adapters of many requests, added to a shared
// projection's output (include/sgq_group.h, lora_add).
//
// Two launches, both on the tensor cores (tcgen05) with the slots as the M
// side, so that a thread owns one slot's row of the result:
//
//   shrink   v = x . a^T, tiles of 128 slots x the whole rank. Bound by the
//            reading of x (prefill) or of a (decode), so the length of x is
//            split over the CTAs of a cluster while the tiles are too few to
//            fill the device; the parts are summed through distributed shared
//            memory in the order of the CTAs.
//   expand   y += c (v . b^T), tiles of 128 slots x 128 or 256 columns. Bound
//            by reading and writing y.
//
// v is kept to about 16 bits and more between them: a row of the workspace
// holds v as two 16-bit parts, hi = round(v) and lo = round(v - hi), and the
// expand product runs over both, so that rounding v costs 2^-17 of it and not
// 2^-9. fp16 rows are first scaled by a power of two to below 2 (the row's
// factor stands behind them), so that no v leaves the type's range.
#include "sgq_group.cuh"
#include "sgq_ragged.cuh"
#include "sgq_tc.cuh"

namespace sgq {

namespace {

constexpr int kM = 128;              // slots a tile
constexpr int kMaxStages = 8;
constexpr int kShrinkThreads = 256;  // warp 0 copies of a, 1 products, 4-7 rows of x, then the result
constexpr int kGather = 128;
constexpr int kExpandThreads = 288;  // warps 0-7 the result, warp 8 copies and products

__device__ uint32_t g_gave_up;       // launches in which a wait ran out of time

struct alignas(128) ShrinkParams {
    CUtensorMap ma;                  // a as bytes [groups][R][K], box 128 x R rows
    LoraArgs l;
    int chunks, kbytes, stages, stage_bytes, split;
};

struct alignas(128) ExpandParams {
    CUtensorMap mb;                  // b as bytes [groups][N][R], box 128 x NT rows
    CUtensorMap mv;                  // workspace rows, box 128 x 128 rows
    LoraArgs l;
    int n_tiles;
    int wide;                        // rows of y are 32-byte aligned
};

// The token of slot s, or -1 where it is outside or its own slot is another.
__device__ __forceinline__ int64_t token_of(const LoraArgs& l, int s) {
    if (!l.rows) return s;
    const int64_t t = l.rows[s];
    return t >= 0 && t < l.T && l.slots[t] == s ? t : -1;
}

// The group and slots [s0, s0 + m) of tile q; false behind the last. Binary
// search in the scanned offsets.
__device__ __forceinline__ bool find_tile(const int* lo, const int* first, int G, int q, int& g, int& s0, int& m) {
    if (q >= first[G]) return false;
    int a = 0, b = G;                // first[a] <= q < first[b]
    while (b - a > 1) {
        const int c = (a + b) >> 1;
        if (first[c] <= q) a = c;
        else b = c;
    }
    g = a;
    s0 = lo[a] + (q - first[a]) * kM;
    m = min(kM, lo[a + 1] - s0);
    return true;
}

// fp32 sums over kind::f16 operands: M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_f16(int dt, int n) {
    return (1u << 4) | (dt == DT_BF16 ? (1u << 7) | (1u << 10) : 0) | ((uint32_t)(n >> 3) << 17) | ((kM >> 4) << 24);
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return DT == DT_BF16 ? f32x2_to_bf16x2(lo, hi) : f32x2_to_f16x2(lo, hi);
}

__device__ __forceinline__ void st_cluster16(const void* p, uint32_t rank, float4 v) {
    const uint32_t local = (uint32_t)__cvta_generic_to_shared(p);
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(remote), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// Shared memory: stages of (x 16 KB, a R x 128 bytes), the parts of v that
// this CTA sums [split][128 / split][R + 4] floats, offsets, barriers.
template <int DT, int BEHIND>
__global__ void __launch_bounds__(kShrinkThreads, 1) lora_shrink_kernel(const __grid_constant__ ShrinkParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    const LoraArgs& l = p.l;
    const int R = l.R, stages = p.stages, ld = R + 4;
    float* parts = reinterpret_cast<float*>(smem + stages * p.stage_bytes);
    int* lo = reinterpret_cast<int*>(parts + kM * ld);
    int* first = lo + kMaxGroups + 8;
    uint64_t* bars = reinterpret_cast<uint64_t*>(first + kMaxGroups + 8);
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
    const bool any = find_tile(lo, first, l.groups, blockIdx.x / split, g, s0, m);   // the same in the whole cluster
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
                const int64_t t = c < m ? token_of(l, s0 + c) : -1;
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
    if (any && warp >= 4) {
        const int share = kM / split, c = rank * share + tid - 128;
        if (tid - 128 < share && c < m) {
            const float* from = parts + (size_t)(tid - 128) * ld;
            auto sum4 = [&](int r) {                     // v[r .. r + 3], the parts in the order of the CTAs
                float4 f = *reinterpret_cast<const float4*>(from + r);
                for (int q = 1; q < active; ++q) {
                    const float4 o = *reinterpret_cast<const float4*>(from + (size_t)q * share * ld + r);
                    f.x += o.x, f.y += o.y, f.z += o.z, f.w += o.w;
                }
                return f;
            };
            float factor = 1.0f, down = 1.0f;
            if (DT == DT_F16) {
                float top = 0.0f;
                for (int r = 0; r < R; r += 4) {
                    const float4 f = sum4(r);
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w))));
                }
                // 2^e with top / 2^e in [1, 2), e held to where both powers are normal
                const int e = min(max((int)(__float_as_uint(top) >> 23), 27), 227);
                factor = __uint_as_float((uint32_t)e << 23);
                down = __uint_as_float((uint32_t)(254 - e) << 23);
            }
            uint8_t* row = reinterpret_cast<uint8_t*>(l.v) + (int64_t)(s0 + c) * lora_row_bytes(R);
            for (int r = 0; r < R; r += 8) {
                uint32_t hi[4], low[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 f = sum4(r + 4 * h);
                    const float v[4] = {f.x * down, f.y * down, f.z * down, f.w * down};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float a0 = round_io<DT>(v[2 * i]), a1 = round_io<DT>(v[2 * i + 1]);
                        hi[2 * h + i] = pack2<DT>(a0, a1);
                        low[2 * h + i] = pack2<DT>(v[2 * i] - a0, v[2 * i + 1] - a1);
                    }
                }
                *reinterpret_cast<uint4*>(row + 2 * r) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(row + 2 * R + 2 * r) = make_uint4(low[0], low[1], low[2], low[3]);
            }
            *reinterpret_cast<float4*>(row + 4 * R) = make_float4(factor, 0.0f, 0.0f, 0.0f);
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 2) tc::tmem_free(tmem, cols);
    if (tid == 0 && *stop) atomicAdd(&g_gave_up, 1);
}

// 16 values of y from p on (8 where the row ends there), in 32- or 16-byte accesses.
__device__ __forceinline__ void load_y(const uint16_t* p, int n, int N, bool wide, uint32_t (&v)[8]) {
    if (wide && n + 16 <= N) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(p)
                     : "memory");
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (n + 8 * h < N) {
            const uint4 t = *reinterpret_cast<const uint4*>(p + 8 * h);
            v[4 * h] = t.x, v[4 * h + 1] = t.y, v[4 * h + 2] = t.z, v[4 * h + 3] = t.w;
        }
}

__device__ __forceinline__ void store_y(uint16_t* p, int n, int N, bool wide, const uint32_t (&v)[8]) {
    if (wide && n + 16 <= N) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                     "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (n + 8 * h < N) *reinterpret_cast<uint4*>(p + 8 * h) = make_uint4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
}

// y rows of one tile: 128 slots x NT columns. VC chunks of 128 bytes hold R values.
template <int DT, int NT, int VC>
struct ExpandCfg {
    static constexpr int kB = NT * kChunk, kV = kM * kChunk;
    static constexpr int kSmem = 1024 + VC * kB + 2 * VC * kV + 2 * 4 * (kMaxGroups + 8) + 256;
};

template <int DT, int NT, int VC>
__global__ void __launch_bounds__(kExpandThreads, 2) lora_expand_kernel(const __grid_constant__ ExpandParams p) {
    using C = ExpandCfg<DT, NT, VC>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    int* lo = reinterpret_cast<int*>(smem + VC * C::kB + 2 * VC * C::kV);
    int* first = lo + kMaxGroups + 8;
    uint64_t* bars = reinterpret_cast<uint64_t*>(first + kMaxGroups + 8);
    uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 3);
    int* part = reinterpret_cast<int*>(misc + 4);
    volatile uint32_t* stop = misc + 1;
    const uint32_t full = tc::smem_addr(bars), acc = full + 8;
    const LoraArgs& l = p.l;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), R = l.R;
    if (tid == 0) {
        tc::bar_init(full, 1);
        tc::bar_init(acc, 1);
        tc::fence_barrier_init();
        *stop = 0;
        tc::prefetch_map(&p.mb);
        tc::prefetch_map(&p.mv);
    }
    // The shrink launch before this one lets it start after it has waited for
    // everything before itself, and writes the workspace alone: all but the
    // workspace may be read before the wait.
    if (warp == 8) tc::tmem_alloc(tc::smem_addr(misc), NT);
    scan_groups(l.offsets, l.groups, l.S, kM, lo, first, part);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, misc[0], 0);
    int g, s0, m;
    const bool any = find_tile(lo, first, l.groups, blockIdx.x / (uint32_t)p.n_tiles, g, s0, m);
    const int n0 = (int)(blockIdx.x % (uint32_t)p.n_tiles) * NT;
    if (!any) {
        pdl_wait();
        pdl_trigger();
    } else if (warp == 8) {
        const uint32_t at = tc::smem_addr(smem), v_at = at + VC * C::kB;
        if (tc::elect()) {
            tc::bar_arrive_expect(full, VC * C::kB + 2 * VC * C::kV);
#pragma unroll
            for (int c = 0; c < VC; ++c) tc::load_3d(at + c * C::kB, &p.mb, full, c * kChunk, n0, g);
        }
        __syncwarp();
        pdl_wait();
        pdl_trigger();
        if (tc::elect()) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < VC; ++c)
                    tc::load_2d(v_at + (h * VC + c) * C::kV, &p.mv, full, h * 2 * R + c * kChunk, s0);
        }
        __syncwarp();
        if (__all_sync(0xFFFFFFFFu, tc::bar_wait(full, 0, stop))) {
            tc::fence_after();
            if (tc::elect()) {
                const uint32_t idesc = idesc_f16(DT, NT);
                const int steps = (R + 15) / 16;                         // of 16 values
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 4 * VC; ++k) {
                        if (k >= steps) break;
                        tc::mma_f16(tmem, tc::desc_sw128(v_at + (h * VC + k / 4) * C::kV) + 2 * (k % 4),
                                    tc::desc_sw128(at + (k / 4) * C::kB) + 2 * (k % 4), idesc, h > 0 || k > 0);
                    }
                tc::commit(acc);
            }
        } else {
            uint32_t never = 0;
            tc::bar_wait(full, 0, &never, 1 << 27);
        }
        __syncwarp();
    } else {
        // this thread: slot s0 + c, columns n0 + first_n ..
        const int quarter = warp & 3, c = quarter * 32 + lane;
        const int first_n = (warp >> 2) * (NT / 2);
        const int64_t t = c < m ? token_of(l, s0 + c) : -1;
        const float scale = l.scaling ? l.scaling[g] : 1.0f;
        uint16_t* y = l.y + (t >= 0 ? t : 0) * l.N + n0 + first_n;
        const int n = n0 + first_n;
        constexpr int kBlocks = NT / 2 / 32;
        uint32_t next[2][8];
        if (t >= 0)
#pragma unroll
            for (int h = 0; h < 2; ++h) load_y(y + 16 * h, n + 16 * h, l.N, p.wide, next[h]);
        pdl_wait();
        float f = scale;
        if (DT == DT_F16 && t >= 0)
            f *= *reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(l.v) + (int64_t)(s0 + c) * lora_row_bytes(R) + 4 * R);
        const bool ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(acc, 0, stop));
        if (ok) {
            tc::fence_after();
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                uint32_t v[32], cur[2][8];
                tc::tmem_load32(tmem + ((uint32_t)quarter << 21) + first_n + 32 * b, v);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 8; ++i) cur[h][i] = next[h][i];
                if (b + 1 < kBlocks && t >= 0)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        load_y(y + 32 * (b + 1) + 16 * h, n + 32 * (b + 1) + 16 * h, l.N, p.wide, next[h]);
                tc::tmem_load_wait(v);
                if (t >= 0)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t w = cur[h][i];
                            const float2 old = DT == DT_BF16
                                                   ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u))
                                                   : f16x2_to_f32x2(w);
                            o[i] = pack2<DT>(fmaf(f, __uint_as_float(v[16 * h + 2 * i]), old.x),
                                             fmaf(f, __uint_as_float(v[16 * h + 2 * i + 1]), old.y));
                        }
                        store_y(y + 32 * b + 16 * h, n + 32 * b + 16 * h, l.N, p.wide, o);
                    }
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 8) tc::tmem_free(tmem, NT);
    if (tid == 0 && *stop) atomicAdd(&g_gave_up, 1);
}

template <int DT, int BEHIND>
cudaError_t shrink(const Device& dev, ShrinkParams& p, int64_t tiles, int smem, cudaStream_t stream) {
    const int64_t ctas = tiles * p.split;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_grid(lora_shrink_kernel<DT, BEHIND>, dim3((unsigned)ctas), kShrinkThreads, smem, p.split, dev.id, p, stream);
}

template <int DT, int NT, int VC>
cudaError_t expand(const Device& dev, ExpandParams& p, int64_t tiles, cudaStream_t stream) {
    const LoraArgs& l = p.l;
    const cuuint64_t bd[3] = {(cuuint64_t)(2 * l.R), (cuuint64_t)l.N, (cuuint64_t)l.groups};
    const cuuint64_t vd[2] = {(cuuint64_t)lora_row_bytes(l.R), (cuuint64_t)l.S};
    if (!encode_rows(&p.mb, l.b, 3, bd, NT) || !encode_rows(&p.mv, l.v, 2, vd, kM)) return cudaErrorInvalidValue;
    p.n_tiles = (l.N + NT - 1) / NT;
    const int64_t ctas = tiles * p.n_tiles;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_grid(lora_expand_kernel<DT, NT, VC>, dim3((unsigned)ctas), kExpandThreads, ExpandCfg<DT, NT, VC>::kSmem, 1,
                       dev.id, p, stream);
}

template <int DT>
cudaError_t run(const Device& dev, const LoraArgs& l, cudaStream_t stream) {
    ShrinkParams p;
    p.l = l;
    p.kbytes = 2 * l.K;
    p.chunks = (p.kbytes + kChunk - 1) / kChunk;
    p.stage_bytes = (kM + l.R) * kChunk;
    const int fixed = 1024 + 4 * kM * (l.R + 4) + 2 * 4 * (kMaxGroups + 8) + 512;
    p.stages = (kMaxDynamicSmem - fixed) / p.stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    const cuuint64_t ad[3] = {(cuuint64_t)p.kbytes, (cuuint64_t)l.R, (cuuint64_t)l.groups};
    if (!encode_rows(&p.ma, l.a, 3, ad, l.R)) return cudaErrorInvalidValue;
    const int64_t tiles = (int64_t)l.S / kM + (l.S < l.groups ? l.S : l.groups);     // at most
    // the length of x over a cluster while the tiles leave multiprocessors
    // idle and a CTA keeps at least 4 chunks
    p.split = 1;
    while (p.split < kMaxCluster && tiles * p.split * 2 <= dev.sms && p.chunks >= 8 * p.split) p.split *= 2;
    const int smem = fixed + p.stages * p.stage_bytes;
    cudaError_t e = p.stages >= 7 ? shrink<DT, 5>(dev, p, tiles, smem, stream) : shrink<DT, 3>(dev, p, tiles, smem, stream);
    if (e != cudaSuccess) return e;
    ExpandParams q;
    q.l = l;
    q.wide = reinterpret_cast<uintptr_t>(l.y) % 32 == 0 && l.N % 16 == 0;
    return l.R <= 64 ? expand<DT, 256, 1>(dev, q, tiles, stream) : expand<DT, 128, 2>(dev, q, tiles, stream);
}

}  // namespace

cudaError_t launch_lora(int dt, const Device& dev, const LoraArgs& a, cudaStream_t stream) {
    return dt == DT_F16 ? run<DT_F16>(dev, a, stream) : run<DT_BF16>(dev, a, stream);
}

}  // namespace sgq
