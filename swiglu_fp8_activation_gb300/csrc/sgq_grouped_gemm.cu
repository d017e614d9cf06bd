// sgq_grouped_gemm.cu -- matrix products grouped by ragged sets of rows
// (include/sgq_group.h, grouped_gemm), on the fifth-generation tensor cores.
//
// One tile is 128 channels (rows of w[g]) by up to BN slots of group g; the
// weights are the M side of the product and the slots its N side, so that a
// group of one row costs an N of 16 and not an M of 128, and the weights,
// which bound a decode step, stream through the same 16 KB tiles at every
// size. out^T = w . x^T: a lane of the accumulator is a channel, a column a
// slot. Both operands are K-major rows of 128 bytes (128 FP8 or 64 16-bit
// values, one "chunk" of K) in 128-byte swizzle.
//
// A CTA keeps its tensor memory and walks over tiles (persistent, one CTA a
// multiprocessor). The tiles follow from the offsets on the device: every CTA
// scans them once (running maximum, which holds them in order, then the sum
// of tiles). Warps:
//   0     copies: the weights' tile by TMA, their scales as 512-byte tiles
//         (MXFP8), the slots' rows as a box where they follow one another
//   1     the products (one thread), four instructions of 32 bytes of K a chunk
//         (with 1x128 scales warp 3 issues half of them)
//   2, 3  the slots' scales (MXFP8, and 1x128 in warp 2): row-major in memory,
//         written into the operand's layout in shared memory
//   4-7   the epilogue, one quarter of the channels each (with 1x128 scales
//         4-11, one quarter of the slots and half of the channels each)
//   last 4  with row indices: the slots' rows, gathered in 16-byte
//         asynchronous copies into the swizzled layout. (TMA's four-row gather
//         took 76 cycles an instruction of 512 bytes: 32768 MXFP8 rows of N =
//         4096, K = 6144 ran in 3687 us with it.)
// Large groups run on pairs of CTAs (cta_group::2): 256 channels by 224 or 256
// slots, each CTA holding its 128 channels and half of the slots' rows, which
// halves what it fetches and reads of them. Where tiles are very few, the CTAs of
// a cluster share the K of one and sum the parts through distributed shared
// memory. pick() below has the rule, with both sides measured.
//
// What bounds it: the weights' bytes for small groups (64 x 8 MXFP8 rows, 54 of 64
// experts in use, N = K = 4096: 935 MB in 143 us, 6.5 TB/s), the tensor cores for large ones (32768
// rows, N = 4096, K = 6144, in order: MXFP8 529 us, 3115 TFLOP/s, per-token 496; 8192
// bf16 rows, N = K = 8192: 586 us, 1876 TFLOP/s), the epilogue's sums with 1x128
// scales (711 us for those 32768 rows).
//
// Two accumulators in tensor memory let the epilogue of one tile run under
// the products of the next. With 1x128 scales, which fp32 holds and no block
// scale of the tensor core can, every chunk is its own accumulator (two pairs)
// and the epilogue warps sum the chunks in registers, scaled. There the slots
// are the M side: a lane is a slot, whose scale (times the weights', one for
// all 128 channels) is one register. With the channels as lanes every thread
// had to read every slot's scale from shared memory for each chunk, 512 cycles
// a chunk by itself (32768 rows, N = 4096, K = 6144: 1381 us).
#include <stddef.h>

#include "sgq_group.cuh"
#include "sgq_ragged.cuh"
#include "sgq_tc.cuh"

namespace sgq {

namespace {

constexpr int kGatherThreads = 128;
constexpr int kM = 128;              // channels a tile
constexpr int kTurn = 32 * 64;       // bytes in which an epilogue warp turns 32 slots x 32 channels
constexpr int kTurnPitch = 80;       // ... with 1x128 scales in rows of 64 + 16 bytes, free of bank conflicts
constexpr int kScaleBufs = 4;        // chunks whose scales tensor memory holds: copies and products of one
                                     // thread run in order, and a place is written again 4 chunks later

struct alignas(128) GemmParams {
    CUtensorMap mw;                // w as bytes [groups][N][K], box 128 x 128 rows
    CUtensorMap mx;                // x as bytes [x_rows][K], box 128 x a CTA's slots (not used with row indices)
    CUtensorMap ms;                // MXFP8: w_scale as tiles of 512 bytes
    GroupGemmArgs a;
    int n_tiles;                   // tiles of 128 channels
    int chunks;                    // chunks of K
    int kbytes;                    // bytes of a row
    int f16;                       // out (and 16-bit operands) are fp16
    int split;                     // CTAs of a cluster that share a tile's K (1: none)
    int across;                    // tiles of channels (a pair's: 256) beside one another
    int step_q, step_r;            // from one of a CTA's tiles to its next: tiles of slots, and of channels
    int xs_align;                  // 16, 4 or 1: alignment of every 4-byte (4 chunks: 16-byte) piece of x_scale
};

template <int FMT, int BN, bool PAIR, bool SPLIT = false>
struct Cfg {
    static constexpr bool kMx = FMT == FMT_MX, kB128 = FMT == FMT_B128;
    static constexpr int kXRows = PAIR ? BN / 2 : BN;             // slots whose rows a CTA holds
    static constexpr int kW = kM * kChunk, kX = kXRows * kChunk;
    static constexpr int kHalves = (BN + 127) / 128;              // 128-slot pieces of the slots' scales
    static constexpr int kSw = kMx ? 512 : 0;                     // weights' scales of a chunk
    static constexpr int kSx = kMx ? 512 * kHalves : 0;           // slots' scales of a chunk
    static constexpr int kStage = kW + kX + kSw + kSx;
    static constexpr int kEpiWarps = kB128 ? 8 : 4;
    static constexpr int kScaleThreads = kB128 ? 32 : 64;         // warp 2, and 3 where it issues no products
    // fp32 scales of the slots: for each quarter of the channels, or for each accumulator
    static constexpr int kXbuf = FMT == FMT_PT || kB128 ? 4 * 4 * BN : 0;
    static constexpr int kTurnBytes = kB128 ? 32 * kTurnPitch : kTurn;
    static constexpr int kParts = SPLIT ? 4 * BN * kM : 0;       // the tile's parts that this CTA sums
    static constexpr int kFixed =
        1024 /* alignment */ + 2 * 4 * (kMaxGroups + 8) + kXbuf + kEpiWarps * kTurnBytes + kParts + (kB128 && BN < kM ? (kM - BN) * kChunk : 0) + 1024;
    static constexpr int kFit = (kMaxDynamicSmem - kFixed) / kStage;
    static constexpr int kStages = kFit < 12 ? kFit : 12;
    static constexpr int kAccs = 2;                               // accumulators
    static constexpr int kAccWidth = kB128 ? 2 * kM : BN;         // columns of one: two chunks' channels, or slots
    static constexpr int kAccCols = kAccs * kAccWidth;
    static constexpr int kScaleCols = kMx ? kScaleBufs * 4 * (1 + kHalves) : 0;
    static constexpr int kNeed = kAccCols + kScaleCols;
    static constexpr int kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    static constexpr int kGatherWarp = 4 + kEpiWarps;             // first of the four
    static constexpr int kThreads = 32 * kGatherWarp;             // without the gather's
    static constexpr int kBehind = 2;                             // chunks of a gather's copies in flight
    static constexpr int kSmem = kFixed + kStages * kStage;
    static_assert(kNeed <= 512 && kStages >= 3, "tile too large");
};

// The tiles of one CTA in order: slots [s0, s0 + m) of group g, channels from
// n0 on. The q-th tile of slots and the r-th of the channels' are stepped
// without divisions, which every role of the CTA would wait for at every tile
// (1x128, 16384 rows, N = 4096, K = 1536: 156 us with 64-bit divisions, 141 without).
struct Walk {
    const int* lo;
    const int* first;
    const GemmParams& p;
    int bn, ctas, rank;              // tiles of `ctas` x 128 channels, this CTA's being the rank-th 128
    int q, r, end;
    int g, s0, m, n0;

    __device__ Walk(const int* lo_, const int* first_, const GemmParams& p_, int bn_, int ctas_, uint32_t from)
        : lo(lo_), first(first_), p(p_), bn(bn_), ctas(ctas_), rank((int)(blockIdx.x % ctas_)), q((int)(from / (uint32_t)p_.across)),
          r((int)(from % (uint32_t)p_.across)), end(first_[p_.a.groups]), g(0) {}
    __device__ bool next() {
        if (q >= end) return false;
        while (first[g + 1] <= q) ++g;
        s0 = lo[g] + (q - first[g]) * bn;
        m = min(bn, lo[g + 1] - s0);
        n0 = (r * ctas + rank) * kM;
        q += p.step_q;
        r += p.step_r;
        if (r >= p.across) {
            r -= p.across;
            ++q;
        }
        return true;
    }
    __device__ void stop() { end = 0; }
};

// a0 += v0 f, a1 += v1 f, in one instruction (32768 rows, N = 4096, K = 6144 with
// 1x128 scales: 761 us, 827 in two).
__device__ __forceinline__ void fma2(float& a0, float& a1, uint32_t v0, uint32_t v1, float f) {
    asm("{\n\t.reg .b64 a, v, f;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 f, {%4, %4};\n\t"
        "fma.rn.f32x2 a, v, f, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "r"(v0), "r"(v1), "f"(f));
}

__device__ uint32_t g_gave_up;     // launches in which a wait ran out of time

template <int FMT, int BN, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(Cfg<FMT, BN, PAIR, SPLIT>::kThreads + kGatherThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ GemmParams p) {
    using C = Cfg<FMT, BN, PAIR, SPLIT>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (tc::smem_addr(smem_raw) & 1023)) & 1023);
    uint8_t* tiles = smem;
    uint8_t* scales = smem + kStages * (C::kW + C::kX);
    int* lo = reinterpret_cast<int*>(scales + kStages * (C::kSw + C::kSx));
    int* first = lo + kMaxGroups + 8;
    float* xbuf = reinterpret_cast<float*>(first + kMaxGroups + 8);      // [4][BN]
    uint8_t* turns = reinterpret_cast<uint8_t*>(xbuf) + C::kXbuf;         // [epilogue warps][32 slots][32 channels]
    float* parts = reinterpret_cast<float*>(turns + C::kEpiWarps * C::kTurnBytes);   // [split][BN / split][128 channels]
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(parts) + C::kParts);
    uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 6);
    int* part = reinterpret_cast<int*>(misc + 4);                        // 24 ints
    volatile uint32_t* stop = misc + 1;
    const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kStages;
    const uint32_t acc_full = empty + 8 * kStages, acc_empty = acc_full + 16, done = acc_empty + 16;
    const uint32_t tiles_at = tc::smem_addr(tiles), scales_at = tc::smem_addr(scales);

    const GroupGemmArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int chunks = p.chunks;
    const bool gather = a.rows != nullptr;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            // the copies' thread and the warps that write scales or rows (in a pair, of both CTAs)
            const int writers = (C::kMx ? C::kScaleThreads / 32 : 0) + (gather ? kGatherThreads / 32 : 0);
            tc::bar_init(full + 8 * i, 1 + (PAIR ? 2 : 1) * writers);
            tc::bar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < C::kAccs; ++i) {
            tc::bar_init(acc_full + 8 * i, 1 + (C::kB128 ? C::kScaleThreads / 32 : 0));
            tc::bar_init(acc_empty + 8 * i, (PAIR ? 2 : 1) * C::kEpiWarps);
        }
        tc::bar_init(done, 1);
        tc::bar_init(done + 8, 1);
        tc::fence_barrier_init();
        *stop = 0;
        tc::prefetch_map(&p.mw);
        tc::prefetch_map(&p.mx);
        if (C::kMx) tc::prefetch_map(&p.ms);
    }
    if (warp == 2) tc::tmem_alloc<PAIR>(tc::smem_addr(misc), C::kCols);
    if (SPLIT) cluster_arrive_relaxed();
    pdl_wait();
    scan_groups(a.offsets, a.groups, a.S, BN, lo, first, part);
    tc::fence_before();
    __syncthreads();
    if (PAIR) {                      // the other's barriers and tensor memory are there
        cluster_arrive();
        cluster_wait();
    }
    if (SPLIT) cluster_wait();       // every CTA of the cluster runs: its shared memory may be written
    tc::fence_after();
    // a next launch that holds tensor memory while it waits for this one may
    // start only now that this CTA has its own
    pdl_trigger();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, misc[0], 0);
    Walk walk(lo, first, p, BN, PAIR ? 2 : 1, blockIdx.x / (SPLIT ? (uint32_t)p.split : PAIR ? 2 : 1));
    // Where few tiles would leave multiprocessors idle, the CTAs of a cluster
    // share one: each takes a piece of K (a multiple of 4 chunks), and each sums
    // the pieces, in order, for some of the slots.
    int k_from = 0, k_to = chunks, share = 0, part_no = 0;
    if (SPLIT) {
        part_no = (int)(blockIdx.x % (uint32_t)p.split);
        share = BN / p.split;
        const int per = ((chunks + p.split - 1) / p.split + 3) & ~3;
        k_from = min(chunks, part_no * per);
        k_to = min(chunks, k_from + per);
        if (k_from == k_to) walk.stop();
    }
    // In a pair the first CTA issues the products: what makes a stage full, and
    // an accumulator free, arrives at its barriers, and the products' ends at both CTAs'.
    const bool leader = !PAIR || walk.rank == 0;
    const uint32_t full_at = PAIR ? tc::at_rank(full, 0) : full, acc_empty_at = PAIR ? tc::at_rank(acc_empty, 0) : acc_empty;
    auto arrive = [&](uint32_t bar) {
        if (PAIR) tc::bar_arrive_cluster(bar);
        else tc::bar_arrive(bar);
    };
    // the product's N, a multiple of 16 a CTA, half each in a pair
    auto columns = [](int m) { return PAIR ? (m + 31) & ~31 : (m + 15) & ~15; };

    if (warp == 0) {
        // ---------------------------------------------------------- copies
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        int64_t issued = 0;
        while (ok && walk.next()) {
            const int scale_row = (walk.g * p.n_tiles + min(walk.n0 / kM, p.n_tiles - 1)) * chunks;
            const uint32_t bytes = (PAIR ? 2 : 1) * (C::kW + C::kSw + (gather ? 0 : C::kX));
            const int s0 = walk.s0 + walk.rank * (columns(walk.m) / 2);
            for (int kc = k_from; kc < k_to; ++kc) {
                ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(empty + 8 * st, ph ^ 1, stop));
                if (!ok) break;
                const uint32_t w_at = tiles_at + st * (C::kW + C::kX), x_at = w_at + C::kW;
                const uint32_t bar = full_at + 8 * st;
                if (tc::elect()) {
                    if (leader) tc::bar_arrive_expect(full + 8 * st, bytes);
                    tc::load_3d<PAIR>(w_at, &p.mw, bar, kc * kChunk, walk.n0, walk.g);
                    if (C::kMx) tc::load_2d<PAIR>(scales_at + st * (C::kSw + C::kSx), &p.ms, bar, 0, scale_row + kc);
                    if (!gather) tc::load_2d<PAIR>(x_at, &p.mx, bar, kc * kChunk, s0);
                }
                ++issued;
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok && lane == 0 && leader) {
            // gave up: wait (a while) for the copies in flight before the block's memory goes
            uint32_t never = 0;
            for (int i = 0; i < kStages && i < issued; ++i) {
                if (--st < 0) {
                    st = kStages - 1;
                    ph ^= 1;
                }
                tc::bar_wait(full + 8 * st, ph, &never, 1 << 27);
                never = 0;
            }
        }
    } else if (C::kB128 && (warp == 1 || warp == 3)) {
        // ------------------------------------- products with 1x128 scales
        // Two chunks fill a pair of accumulators. Warp 1 issues for the even pairs
        // and warp 3 for the odd ones: the issuing thread is held while its
        // products run, and what it does between (three waits, the votes, the
        // descriptors) runs under the other's products (32768 rows, N = 4096, K =
        // 6144: 972 us with warp 1 alone and a division a tile, 827 with both and none).
        const int mine = warp >> 1;
        const uint64_t base = tc::desc_sw128(tiles_at);
        const uint32_t idesc = (1u << 4) | ((kM >> 3) << 17) | ((kM >> 4) << 24);
        const uint32_t d = tmem + mine * C::kAccWidth, acc_bars = 8 * mine;
        int st = 0;
        uint32_t ph = 0, use = 0;
        bool ok = true;
        auto products = [&](uint32_t to) {                               // of the next stage
            ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(full + 8 * st, ph, stop));
            if (!ok) return;
            tc::fence_after();
            if (tc::elect()) {
                const uint64_t dw = base + (uint32_t)(st * ((C::kW + C::kX) >> 4)), dx = dw + (C::kW >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) tc::mma_f8(to, dx + 2 * k, dw + 2 * k, idesc, k > 0);
                tc::commit(empty + 8 * st);
            }
            __syncwarp();
        };
        auto step = [&]() {
            if (++st == kStages) {
                st = 0;
                ph ^= 1;
            }
        };
        while (ok && walk.next()) {
            for (int kc = k_from; kc < k_to; kc += 2, ++use) {
                const bool two = kc + 1 < k_to;
                if ((use & 1) == (uint32_t)mine) {
                    ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(acc_empty + acc_bars, ((use >> 1) & 1) ^ 1, stop));
                    if (ok) products(d);
                    step();
                    if (ok && two) {
                        products(d + kM);
                    }
                    if (two) step();
                    if (!ok) break;
                    if (tc::elect()) tc::commit(acc_full + acc_bars);
                    __syncwarp();
                } else {
                    step();
                    if (two) step();
                }
            }
        }
        if (!ok) {
            uint32_t never = 0;
            if (tc::elect()) tc::commit(done + 8 * mine);
            __syncwarp();
            tc::bar_wait(done + 8 * mine, 0, &never, 1 << 27);
        }
    } else if (warp == 1) {
        // -------------------------------------------------------- products
        int st = 0, use = 0;
        uint32_t ph = 0, chunk_no = 0;
        bool ok = true, ready = false;
        while (ok && leader && walk.next()) {
            const uint32_t n = (uint32_t)columns(walk.m);
            constexpr int kRows = PAIR ? 2 * kM : kM;
            uint32_t idesc;
            if (C::kMx) idesc = ((n >> 3) << 17) | (1u << 23) | ((kRows >> 7) << 27);
            else idesc = (1u << 4) | ((n >> 3) << 17) | ((kRows >> 4) << 24);
            if (FMT == FMT_16BIT && !p.f16) idesc |= (1u << 7) | (1u << 10);
            const int left = p.kbytes - (chunks - 1) * kChunk;
            const int last_steps = (left + 31) / 32;
            for (int kc = k_from; kc < k_to; ++kc, ++chunk_no) {
                const int buf = use % C::kAccs;
                if (!ready) {
                    ok = true;
                    if (kc == k_from) ok = tc::bar_wait<PAIR>(acc_empty + 8 * buf, ((use / C::kAccs) & 1) ^ 1, stop);
                    ok = __all_sync(0xFFFFFFFFu, ok && tc::bar_wait<PAIR>(full + 8 * st, ph, stop));
                    if (!ok) break;
                }
                tc::fence_after();
                const bool done_acc = kc == k_to - 1;
                const int next_st = st + 1 == kStages ? 0 : st + 1;
                const uint32_t next_ph = ph ^ (next_st == 0);
                // whether the next chunk can follow at once: asked for now, so that
                // the answer (90 cycles) is there when this chunk's products are issued
                bool next_ready = tc::bar_test<PAIR>(full + 8 * next_st, next_ph);
                if (done_acc)
                    next_ready &= tc::bar_test<PAIR>(acc_empty + 8 * ((use + 1) % C::kAccs), (((use + 1) / C::kAccs) & 1) ^ 1);
                if (tc::elect()) {
                    const uint32_t w_at = tiles_at + st * (C::kW + C::kX);
                    const uint64_t dw = tc::desc_sw128(w_at), dx = tc::desc_sw128(w_at + C::kW);
                    const uint32_t d = tmem + buf * C::kAccWidth;
                    const uint32_t sw = tmem + C::kAccCols + (chunk_no % kScaleBufs) * 4 * (1 + C::kHalves), sx = sw + 4;
                    if (C::kMx) {
                        const uint32_t s_at = scales_at + st * (C::kSw + C::kSx);
                        tc::copy_scales<PAIR>(sw, tc::desc_rows16(s_at));
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            tc::copy_scales<PAIR>(sx + 4 * h, tc::desc_rows16(s_at + 512 + 512 * h));
                    }
                    const int steps = kc == chunks - 1 ? last_steps : 4;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t add = k > 0 || kc > k_from;
                        if (k >= steps) break;
                        if (C::kMx) tc::mma_mx8<PAIR>(d, dw + 2 * k, dx + 2 * k, idesc | (k << 4) | (k << 29), sw, sx, add);
                        else if (FMT == FMT_16BIT) tc::mma_f16<PAIR>(d, dw + 2 * k, dx + 2 * k, idesc, add);
                        else tc::mma_f8<PAIR>(d, dw + 2 * k, dx + 2 * k, idesc, add);
                    }
                    tc::commit<PAIR>(empty + 8 * st);
                    if (done_acc) tc::commit<PAIR>(acc_full + 8 * buf);
                }
                ready = __all_sync(0xFFFFFFFFu, next_ready);
                use += done_acc;
                st = next_st;
                ph = next_ph;
            }
        }
        if (!ok) {
            uint32_t never = 0;
            if (tc::elect()) tc::commit<PAIR>(done);
            __syncwarp();
            tc::bar_wait(done, 0, &never, 1 << 27);
        }
    } else if (warp < 4) {
        // ------------------------------------------------- scales of the slots
        if (C::kMx || C::kB128) {
            constexpr int kScaleThreads = C::kScaleThreads, kRows = (BN + kScaleThreads - 1) / kScaleThreads;
            const int u = tid - 64;
            int st = 0, use = 0;
            uint32_t ph = 0;
            bool ok = true;
            const int64_t row_bytes = C::kMx ? p.kbytes / 32 : (int64_t)chunks * 4;
            // a tile's row indices are read during the tile before it, its first scales during that tile's last chunks
            Walk ahead = walk;
            int64_t row[kRows];
            const uint8_t* src[kRows];
            const float *ws = nullptr, *next_ws = nullptr;
            auto read_rows = [&]() {
                const bool more = ahead.next();
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int c = u + i * kScaleThreads;
                    row[i] = more && c < ahead.m ? (gather ? a.rows[ahead.s0 + c] : ahead.s0 + c) : -1;
                }
                next_ws = C::kB128 && more ? static_cast<const float*>(a.ws) +
                                                 ((int64_t)ahead.g * p.n_tiles + min(ahead.n0 / kM, p.n_tiles - 1)) * chunks
                                           : nullptr;
            };
            auto sources = [&]() {
                ws = next_ws;
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    src[i] = row[i] >= 0 && row[i] < a.x_rows ? static_cast<const uint8_t*>(a.xs) + row[i] * row_bytes : nullptr;
            };
            // four chunks' scales a row at a time, the next four in flight
            uint32_t cur[kRows][4], nxt[kRows][4];
            float cur_w[4], nxt_w[4];                                    // 1x128: the weights' scales of the same chunks
            auto fetch = [&](uint32_t (&v)[kRows][4], float (&w)[4], int kc) {
                if (C::kB128) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) w[q] = ws && kc + q < chunks ? ws[kc + q] : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[i][q] = 0;
                    if (!src[i]) continue;
                    const uint8_t* s = src[i] + (int64_t)kc * 4;
                    if (p.xs_align == 16) {
                        const uint4 t = *reinterpret_cast<const uint4*>(s);
                        v[i][0] = t.x, v[i][1] = t.y, v[i][2] = t.z, v[i][3] = t.w;
                    } else if (p.xs_align == 4) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (kc + q < chunks) v[i][q] = reinterpret_cast<const uint32_t*>(s)[q];
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            if (kc * 4 + q < row_bytes) v[i][q / 4] |= (uint32_t)s[q] << (8 * (q % 4));
                    }
                }
            };
            read_rows();
            sources();
            fetch(cur, cur_w, k_from);
            read_rows();
            while (ok && walk.next()) {
                for (int kc0 = k_from; ok && kc0 < k_to; kc0 += 4) {
                    if (kc0 + 4 < k_to) {
                        fetch(nxt, nxt_w, kc0 + 4);
                    } else {
                        sources();
                        fetch(nxt, nxt_w, 0);
                        read_rows();
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (kc0 + q >= k_to) break;
                        const int buf = use % C::kAccs;
                        if (C::kMx) ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(empty + 8 * st, ph ^ 1, stop));
                        else if (q % 2 == 0)
                            ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(acc_empty + 8 * buf, ((use / C::kAccs) & 1) ^ 1, stop));
                        if (!ok) break;
                        uint8_t* dst = C::kMx ? scales + st * (C::kSw + C::kSx) + C::kSw : reinterpret_cast<uint8_t*>(xbuf + (2 * buf + q % 2) * BN);
#pragma unroll
                        for (int i = 0; i < kRows; ++i) {
                            const int c = u + i * kScaleThreads;
                            if (c < BN) {
                                if (C::kMx)
                                    *reinterpret_cast<uint32_t*>(dst + (c >> 7) * 512 + (c & 31) * 16 + ((c >> 5) & 3) * 4) = cur[i][q];
                                else
                                    *reinterpret_cast<float*>(dst + 4 * c) = __uint_as_float(cur[i][q]) * cur_w[q];
                            }
                        }
                        if (C::kMx) tc::fence_async_smem();
                        __syncwarp();
                        if (C::kMx) {
                            if (lane == 0) arrive(full_at + 8 * st);
                        } else if (q % 2 == 1 || kc0 + q == k_to - 1) {
                            if (lane == 0) tc::bar_arrive(acc_full + 8 * buf);
                            ++use;
                        }
                        if (++st == kStages) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (C::kB128) cur_w[q] = nxt_w[q];
#pragma unroll
                        for (int i = 0; i < kRows; ++i) cur[i][q] = nxt[i][q];
                    }
                }
            }
        }
    } else if (warp >= C::kGatherWarp) {
        // ------------------------------------------- gathered rows of the slots
        // thread u copies 16-byte piece u % 8 of rows u / 8 + 16 i of the chunk
        constexpr int kRows = C::kXRows / 16;
        const int u = tid - 32 * C::kGatherWarp, piece = u & 7;
        int st = 0, lag_st = 0;
        uint32_t ph = 0;
        bool ok = true;
        int behind = 0;                                                  // chunks issued and not yet handed over
        auto hand_over = [&]() {
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(full_at + 8 * lag_st);
            if (++lag_st == kStages) lag_st = 0;
            --behind;
        };
        // a tile's row indices are read while the copies of the tile before it are issued
        Walk ahead = walk;
        int row[kRows];
        auto read_rows = [&]() {
            const bool more = ahead.next();
            const int n = more ? columns(ahead.m) : 0, from = PAIR ? ahead.rank * (n / 2) : 0, to = PAIR ? min(ahead.m, from + n / 2) : ahead.m;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int c = from + (u >> 3) + 16 * i;
                row[i] = more && c < to ? a.rows[ahead.s0 + c] : -1;
            }
        };
        read_rows();
        while (ok && walk.next()) {
            const uint8_t* src[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                src[i] = row[i] >= 0 && row[i] < a.x_rows
                             ? static_cast<const uint8_t*>(a.x) + (int64_t)row[i] * p.kbytes + piece * 16
                             : nullptr;
            read_rows();
            for (int kc = k_from; kc < k_to; ++kc) {
                ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(empty + 8 * st, ph ^ 1, stop));
                if (!ok) break;
                uint8_t* dst = tiles + st * (C::kW + C::kX) + C::kW + (u >> 3) * kChunk + ((piece ^ ((u >> 3) & 7)) << 4);
                const int k = kc * kChunk;
                const bool in = k + piece * 16 < p.kbytes;               // zeros behind the row's end
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (src[i]) cp_async16(dst + i * 16 * kChunk, in ? src[i] + k : src[i], in ? 16 : 0);
                cp_async_commit();
                if (++behind > C::kBehind) {
                    cp_async_wait<C::kBehind>();
                    hand_over();
                }
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        cp_async_wait<0>();
        while (ok && behind > 0) hand_over();
    } else {
        // -------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        const uint32_t lanes = (uint32_t)quarter << 21;                  // first lane of the quarter, in the address
        float* xrow = xbuf + quarter * BN;
        int use = 0;
        bool ok = true;
        while (ok && walk.next()) {
            const int n = walk.n0 + quarter * 32 + lane;                 // this thread's channel (not with 1x128 scales)
            const int m = walk.m;
            uint32_t there[BN / 32];
            float wn = 1.0f;
#pragma unroll
            for (int i = 0; i < BN / 32; ++i) {
                const int c = i * 32 + lane;
                int64_t r = c < m ? walk.s0 + c : -1;
                if (gather && c < m) r = a.rows[r];
                const bool valid = r >= 0 && r < a.x_rows;
                there[i] = __ballot_sync(0xFFFFFFFFu, valid);
                if (FMT == FMT_PT) xrow[c] = valid ? static_cast<const float*>(a.xs)[r] : 0.0f;
            }
            if (FMT == FMT_PT && n < a.N) wn = static_cast<const float*>(a.ws)[(int64_t)walk.g * a.N + n];
            __syncwarp();
            // columns c0 .. c0 + 31 of the tile: rounded once, turned in shared
            // memory from a channel a thread to rows of slots, stored in 16-byte
            // pieces (as 2-byte stores of a channel a thread, 192 slots took 4.4 us)
            uint8_t* turn = turns + (warp - 4) * C::kTurnBytes;
            auto store = [&](int c0, uint32_t valid, const float (&v)[32]) {
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float r = (valid >> c) & 1 ? v[c] : 0.0f;
                    *reinterpret_cast<uint16_t*>(turn + c * 64 + lane * 2) =
                        (uint16_t)(p.f16 ? f32x2_to_f16x2(r, 0.0f) : f32x2_to_bf16x2(r, 0.0f));
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 8 * i + (lane >> 2), ch = walk.n0 + quarter * 32 + (lane & 3) * 8;
                    if (c0 + c < m && ch < a.N)
                        st16_if(a.out + (int64_t)(walk.s0 + c0 + c) * a.N + ch,
                                *reinterpret_cast<const uint4*>(turn + c * 64 + (lane & 3) * 16), true);
                }
            };
            if (C::kB128) {
                // this thread's slot, 64 channels: the chunks' products scaled and
                // summed in registers, two chunks to a wait (one at a time, the
                // waits and arrivals were most of the loop's instructions)
                const int c = quarter * 32 + lane, first = ((warp - 4) >> 2) * 64;
                const bool busy = quarter * 32 < m;
                const float* scale = xbuf + (c < m ? c : 0);
                float acc[64];
#pragma unroll
                for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
                for (int kc = k_from; kc < k_to; kc += 2, ++use) {
                    const int buf = use & 1;
                    ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(acc_full + 8 * buf, (use >> 1) & 1, stop));
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t at = tmem + lanes + buf * C::kAccWidth + first;
                    // the pair is free once the last of it is in registers, before that is summed
                    // (arriving behind the sums: 135 us for 120, 16384 rows, N = 4096, K = 1536; 761 for 711, 32768 rows, K = 6144)
                    auto release = [&]() {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) tc::bar_arrive(acc_empty + 8 * buf);
                    };
                    if (busy) {
                        // 16 columns at a time, the next 16 on their way
                        uint32_t v[2][16];
                        tc::tmem_load16(at, v[0]);
                        const float f0 = scale[2 * buf * BN], f1 = scale[(2 * buf + 1) * BN];
                        const bool two = kc + 1 < k_to;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            uint32_t(&cur)[16] = v[j & 1];
                            uint32_t(&nxt)[16] = v[(j & 1) ^ 1];
                            if (j == 4 && !two) break;
                            tc::tmem_load_wait(cur);
                            if (j == (two ? 7 : 3)) release();
                            if (j < 7 && (j != 3 || two)) tc::tmem_load16(at + (j + 1) / 4 * kM + (j + 1) % 4 * 16, nxt);
#pragma unroll
                            for (int i = 0; i < 16; i += 2)
                                fma2(acc[j % 4 * 16 + i], acc[j % 4 * 16 + i + 1], cur[i], cur[i + 1], j < 4 ? f0 : f1);
                        }
                    } else {
                        release();
                    }
                }
                if (!ok) break;
                if (SPLIT) {
                    // this slot's 64 sums to the CTA that adds the parts up for it
                    if (c < m) {
                        const float* to = parts + (part_no * share + c % share) * kM + first;
#pragma unroll
                        for (int i = 0; i < 64; i += 4)
                            st_cluster16(to + i, (uint32_t)(c / share), make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]));
                    }
                    continue;
                }
                // half of the channels at a time through shared memory, so that four lanes store a slot's 64 bytes
                uint32_t valid = 0;
#pragma unroll
                for (int i = 0; i < BN / 32; ++i)
                    if (i == quarter) valid = there[i];
                const bool real = (valid >> lane) & 1;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!busy) break;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float o[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] = real ? acc[32 * h + 8 * i + j] : 0.0f;
                        *reinterpret_cast<uint4*>(turn + lane * kTurnPitch + 16 * i) = p.f16 ? pack8<DT_F16>(o) : pack8<DT_BF16>(o);
                    }
                    __syncwarp();
                    const int ch = walk.n0 + first + 32 * h + (lane & 3) * 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * i + (lane >> 2), slot = quarter * 32 + r;
                        if (slot < m && ch < a.N)
                            st16_if(a.out + (int64_t)(walk.s0 + slot) * a.N + ch,
                                    *reinterpret_cast<const uint4*>(turn + r * kTurnPitch + (lane & 3) * 16), true);
                    }
                }
            } else {
                const int buf = use % C::kAccs;
                ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(acc_full + 8 * buf, (use / C::kAccs) & 1, stop));
                if (!ok) break;
                ++use;
                tc::fence_after();
#pragma unroll
                for (int c0 = 0; c0 < BN; c0 += 32) {
                    if (c0 < m) {
                        uint32_t v[32];
                        float f[32];
                        tc::tmem_load32(tmem + lanes + buf * BN + c0, v);
                        tc::tmem_load_wait(v);
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            f[c] = __uint_as_float(v[c]);
                            if (FMT == FMT_PT) f[c] = f[c] * xrow[c0 + c] * wn;
                        }
                        if (SPLIT) {
                            // this channel's sums to the CTAs that add the parts up
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (c0 + c < m)
                                    st_cluster4(parts + (part_no * share + (c0 + c) % share) * kM + quarter * 32 + lane,
                                                (uint32_t)((c0 + c) / share), f[c]);
                        } else {
                            store(c0, there[c0 / 32], f);
                        }
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) arrive(acc_empty_at + 8 * buf);
            }
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        Walk one(lo, first, p, BN, 1, blockIdx.x / (uint32_t)p.split);
        if (one.next()) {
            const int per = ((chunks + p.split - 1) / p.split + 3) & ~3, active = (chunks + per - 1) / per;
            const int mine = min(share, one.m - part_no * share);
            for (int i = tid; i < mine * (kM / 8); i += blockDim.x) {
                const int c = i / (kM / 8), ch = i % (kM / 8) * 8, slot = one.s0 + part_no * share + c;
                float v[8] = {};
                const int64_t r = gather ? a.rows[slot] : slot;
                if (r >= 0 && r < a.x_rows)
                    for (int q = 0; q < active; ++q) {
                        const float* from = parts + (q * share + c) * kM + ch;
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += from[j];
                    }
                if (one.n0 + ch < a.N)
                    st16_if(a.out + (int64_t)slot * a.N + one.n0 + ch, p.f16 ? pack8<DT_F16>(v) : pack8<DT_BF16>(v), true);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (PAIR) {                      // the other may still arrive here, or read this CTA's operands
        cluster_arrive();
        cluster_wait();
    }
    tc::fence_after();
    if (warp == 2) tc::tmem_free<PAIR>(tmem, C::kCols);
    if (tid == 0 && *stop) atomicAdd(&g_gave_up, 1);
}

// --------------------------------------------------------------------- host

// Tiles of bn slots x one of n_tiles at most, whatever the offsets.
int64_t most_tiles(const GroupGemmArgs& a, int bn, int n_tiles) {
    return ((int64_t)a.S / bn + (a.S < a.groups ? a.S : a.groups)) * n_tiles;
}

template <int FMT, int BN, bool PAIR = false, bool SPLIT = false>
cudaError_t run(const Device& dev, GemmParams& p, cudaStream_t stream) {
    using C = Cfg<FMT, BN, PAIR, SPLIT>;
    const GroupGemmArgs& a = p.a;
    const cuuint64_t wd[3] = {(cuuint64_t)p.kbytes, (cuuint64_t)a.N, (cuuint64_t)a.groups};
    // with no row of x at all nothing of it is used: any memory serves as its map
    const cuuint64_t xd[2] = {(cuuint64_t)p.kbytes, (cuuint64_t)(a.x_rows ? a.x_rows : 1)};
    if (!encode_rows(&p.mw, a.w, 3, wd, kM) || !encode_rows(&p.mx, a.x_rows ? a.x : a.w, 2, xd, C::kXRows))
        return cudaErrorInvalidValue;
    if (C::kMx && !encode_tiles512(&p.ms, a.ws, (int64_t)a.groups * p.n_tiles * p.chunks)) return cudaErrorInvalidValue;
    constexpr int kCtas = PAIR ? 2 : 1;
    const int64_t most = most_tiles(a, BN, (p.n_tiles + kCtas - 1) / kCtas);
    const int64_t room = dev.sms >= kCtas ? dev.sms / kCtas : 1, tiles = SPLIT || most < room ? most : room;
    const int cluster = SPLIT ? p.split : kCtas;
    p.across = (p.n_tiles + kCtas - 1) / kCtas;
    p.step_q = (int)(tiles / p.across);              // with SPLIT all the tiles there may be: a cluster has one
    p.step_r = (int)(tiles % p.across);
    return launch_grid(grouped_gemm_kernel<FMT, BN, PAIR, SPLIT>, dim3((unsigned)(tiles * cluster)),
                       C::kThreads + (a.rows ? kGatherThreads : 0), C::kSmem, cluster, dev.id, p, stream);
}

template <int FMT>
cudaError_t pick(const Device& dev, GemmParams& p, cudaStream_t stream) {
    // Few tiles: a cluster a tile, from 24 chunks on, while that leaves
    // multiprocessors idle and a CTA keeps at least 8 chunks. One row, MXFP8, N =
    // 1536, K = 6144: 14.1 us whole, 8.5 in 4 pieces; 16 bf16 rows, N = 1024, K =
    // 4096: 15.0 and 7.2; 100 rows, per-token, N = 256, K = 2048: 7.3 whole, 9.2 in two.
    const int64_t few = most_tiles(p.a, 32, p.n_tiles);
    p.split = 1;
    while (p.split < kMaxCluster && few * p.split * 2 <= dev.sms && p.chunks >= (p.split == 1 ? 24 : 16 * p.split))
        p.split *= 2;
    if (p.split > 1) return run<FMT, 32, false, true>(dev, p, stream);
    // Else tiles about as wide as a group has slots on average, unless they are
    // fewer than three fifths of the multiprocessors: then narrower ones, which
    // read the weights more often but from more CTAs. 1000 MXFP8 rows of 4 groups,
    // N = 1024, K = 2048: pairs (64 CTAs) 12.2 us, 128 slots (64) 9.7, 64 (128) 8.3;
    // 4096 rows of 16 groups, N = K = 2048: pairs (512) 28.3, 128 slots (512) 31.1,
    // 64 (1024) 40.8; 999 per-token rows of 7 groups, N = 1544: pairs (98) 14.2, 128
    // slots (182) 14.7.
    constexpr int kPair = FMT == FMT_B128 ? 128 : FMT == FMT_MX ? 224 : 256;
    const int64_t groups = p.a.S < p.a.groups ? p.a.S : p.a.groups, mean = (p.a.S + groups - 1) / groups;
    auto ctas = [&](int level) {
        const int bn = level == 3 ? kPair : 32 << level;
        return groups * ((mean + bn - 1) / bn) * (level == 3 ? (p.n_tiles + 1) / 2 * 2 : p.n_tiles);
    };
    int level = mean <= 24 ? 0 : mean <= 64 ? 1 : FMT == FMT_B128 || mean <= 128 || p.n_tiles < 2 ? 2 : 3;
    while (level > 0 && 5 * ctas(level) < 3 * (int64_t)dev.sms) --level;
    switch (level) {
        case 0: return run<FMT, 32>(dev, p, stream);
        case 1: return run<FMT, 64>(dev, p, stream);
        case 2: return run<FMT, 128>(dev, p, stream);
        default: return run<FMT, kPair, FMT != FMT_B128>(dev, p, stream);
    }
}

}  // namespace

cudaError_t gemm_gave_up(uint32_t* n) { return cudaMemcpyFromSymbol(n, g_gave_up, sizeof *n); }

cudaError_t launch_grouped_gemm(int fmt, int dt, const Device& dev, const GroupGemmArgs& a, cudaStream_t stream) {
    GemmParams p;
    p.a = a;
    p.kbytes = fmt == FMT_16BIT ? 2 * a.K : a.K;
    p.chunks = (p.kbytes + kChunk - 1) / kChunk;
    p.n_tiles = (a.N + kM - 1) / kM;
    p.f16 = dt == DT_F16;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.xs);
    const int64_t row = fmt == FMT_MX ? a.K / 32 : (int64_t)p.chunks * 4;      // bytes of a row of x_scale
    p.xs_align = at % 16 == 0 && row % 16 == 0 ? 16 : at % 4 == 0 && row % 4 == 0 ? 4 : 1;
    switch (fmt) {
        case FMT_MX: return pick<FMT_MX>(dev, p, stream);
        case FMT_B128: return pick<FMT_B128>(dev, p, stream);
        case FMT_PT: return pick<FMT_PT>(dev, p, stream);
        default: return pick<FMT_16BIT>(dev, p, stream);
    }
}

}  // namespace sgq
