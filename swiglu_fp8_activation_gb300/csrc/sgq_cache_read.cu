// sgq_cache_read.cu -- rows of a paged cache as 16-bit values
// (include/sgq_cache.h, cache_read).
//
// One pass, bound by memory: a thread reads 8 values of one row and writes
// them, k's and v's pieces issued together. Neighbouring threads take the pieces
// of a row, then the rows of a token's heads, so that the writes of a token are
// one run whatever the cache's order.
#include "sgq_cache.cuh"

namespace sgq {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;            // pieces a thread has in flight, of k and of v each

template <int FMT>
__device__ __forceinline__ uint4 load_piece(const uint8_t* p) {
    uint4 v = {0, 0, 0, 0};
    if (FMT == FMT_PT) asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    else
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
__device__ __forceinline__ uint4 piece_out(uint4 v, float s) {
    if (FMT != FMT_PT) return v;
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 c = e4m3x2_to_f32x2((i < 2 ? v.x : v.y) >> (16 * (i & 1)));
        f[2 * i] = c.x * s;
        f[2 * i + 1] = c.y * s;
    }
    return pack8<DT>(f);
}

template <int FMT, int DT>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int kPiece = FMT == FMT_PT ? 8 : 16;               // bytes of 8 values
    const int nch = a.c.D >> 3, per = nch * a.c.heads;           // pieces of a row, of a token
    const int64_t total = a.S * per;
    uint4 kv[kAhead], vv[kAhead];
    float ks[kAhead], vs[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int64_t at = ((int64_t)blockIdx.x * kAhead + i) * kThreads + threadIdx.x;
        kv[i] = vv[i] = make_uint4(0, 0, 0, 0);
        ks[i] = vs[i] = 0.0f;
        if (at >= total) continue;
        const int64_t s = at / per;
        const int rest = (int)(at - s * per), head = rest / nch, c = rest - head * nch;
        const int64_t slot = a.wide ? static_cast<const int64_t*>(a.slots)[s] : (int64_t) static_cast<const int32_t*>(a.slots)[s];
        if (slot < 0 || slot >= a.c.pages * a.c.page.d) continue;
        const int64_t page = slot / a.c.page.d, place = slot - page * a.c.page.d;
        const int64_t off = page * a.c.ps + head * a.c.hs + place * a.c.ts + c * kPiece;
        const int64_t row = (page * a.c.heads + head) * a.c.page.d + place;
        if (a.k) kv[i] = load_piece<FMT>(a.c.k + off);
        if (a.v) vv[i] = load_piece<FMT>(a.c.v + off);
        if (FMT == FMT_PT) {
            if (a.k) ks[i] = a.c.ks[row];
            if (a.v) vs[i] = a.c.vs[row];
        }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int64_t at = ((int64_t)blockIdx.x * kAhead + i) * kThreads + threadIdx.x;
        if (a.k) st16_if(a.k + at * 8, piece_out<FMT, DT>(kv[i], ks[i]), at < total);
        if (a.v) st16_if(a.v + at * 8, piece_out<FMT, DT>(vv[i], vs[i]), at < total);
    }
}

}  // namespace

cudaError_t launch_cache_read(int fmt, int dt, const Device& dev, const ReadArgs& a, cudaStream_t stream) {
    const int64_t pieces = a.S * (a.c.D / 8) * a.c.heads, ctas = (pieces + kAhead * kThreads - 1) / (kAhead * kThreads);
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const auto k = fmt != FMT_PT ? cache_read_kernel<FMT_16BIT, DT_BF16>
                   : dt == DT_F16 ? cache_read_kernel<FMT_PT, DT_F16> : cache_read_kernel<FMT_PT, DT_BF16>;
    return launch_grid(k, dim3((unsigned)ctas), kThreads, 0, 1, dev.id, a, stream);
}

}  // namespace sgq
