// sgq_cache_read.cu -- rows of a paged cache as 16-bit values
// (include/sgq_cache.h, cache_read).
//
// One pass, bound by memory: a thread reads 16 bytes of a row (8 values, or 16
// codes) of k and of v and writes them. Neighbouring threads take the pieces of a
// row, then the rows of a token's heads, so that the writes of a token are one run
// whatever the cache's order. 131072 tokens, 8 heads of 128, E4M3 to bf16 (814 MB): a
// piece a thread 127 us (6411 GB/s), two 135, four 143; past L2 (evict first) 136.
#include "sgq_cache.cuh"

namespace sgq {

namespace {

constexpr int kThreads = 256;
__device__ __forceinline__ uint4 load_piece(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Two E4M3 codes (low byte first) -> two floats, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(w));
    return f16x2_to_f32x2(h);
}

template <int FMT, int DT>
__device__ __forceinline__ void store_piece(uint16_t* to, uint4 v, float s) {
    if (FMT != FMT_PT) {
        st16_if(to, v, true);
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 c = e4m3x2_to_f32x2(w[2 * h + (i >> 1)] >> (16 * (i & 1)));
            f[2 * i] = c.x * s;
            f[2 * i + 1] = c.y * s;
        }
        st16_if(to + 8 * h, pack8<DT>(f), true);
    }
}

template <int FMT, int DT>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int kValues = FMT == FMT_PT ? 16 : 8;              // of 16 bytes
    const int64_t s0 = (int64_t)blockIdx.x * a.tpc;
    const int total = (int)min((int64_t)a.tpc, a.S - s0) * (int)a.pieces.d;
    for (int at = threadIdx.x; at < total; at += kThreads) {
        const int t = (int)quotient((uint32_t)at, a.pieces), rest = at - t * (int)a.pieces.d;
        const int head = (int)quotient((uint32_t)rest, a.row), c = rest - head * (int)a.row.d;
        const int64_t slot = load_index(a.slots, a.wide, s0 + t);
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        float ks = 0.0f, vs = 0.0f;
        if (slot >= 0 && slot < a.c.pages * a.c.page.d) {
            int place;
            const int64_t page = page_of_slot(slot, a.c.page, place);
            const int64_t off = page * a.c.ps + head * a.c.hs + place * a.c.ts + c * 16;
            if (a.k) k = load_piece(a.c.k + off);
            if (a.v) v = load_piece(a.c.v + off);
            if (FMT == FMT_PT) {
                const int64_t row = (page * a.c.heads + head) * a.c.page.d + place;
                if (a.k) ks = a.c.ks[row];
                if (a.v) vs = a.c.vs[row];
            }
        }
        const int64_t to = (s0 * a.pieces.d + at) * kValues;
        if (a.k) store_piece<FMT, DT>(a.k + to, k, ks);
        if (a.v) store_piece<FMT, DT>(a.v + to, v, vs);
    }
}

}  // namespace

cudaError_t launch_cache_read(int fmt, int dt, const Device& dev, const ReadArgs& r, cudaStream_t stream) {
    ReadArgs a = r;
    const int row = a.c.D / (fmt == FMT_PT ? 16 : 8), pieces = row * a.c.heads;
    a.pieces = make_div((uint32_t)pieces);
    a.row = make_div((uint32_t)row);
    // as many tokens a CTA as give each thread one piece
    a.tpc = pieces >= kThreads ? 1 : kThreads / pieces;
    const int64_t ctas = (a.S + a.tpc - 1) / a.tpc;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const auto k = fmt != FMT_PT ? cache_read_kernel<FMT_16BIT, DT_BF16>
                   : dt == DT_F16 ? cache_read_kernel<FMT_PT, DT_F16> : cache_read_kernel<FMT_PT, DT_BF16>;
    return launch_grid(k, dim3((unsigned)ctas), kThreads, 0, 1, dev.id, a, stream);
}

}  // namespace sgq
