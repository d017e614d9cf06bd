// sgq_rope.cu -- rotary positions and the rows that go into a paged cache
// (include/sgq_cache.h: rope, cache_write).
//
// One pass: every row (a head of a token) is read once and written once, so
// memory bounds it. A row is cut into units of 16 values, two 16-byte pieces
// that hold whole pairs: pieces j and j + R/16 where pairs are (i, i + R/2),
// neighbours where they are (2i, 2i + 1). A lane owns a unit, 4 to 16 lanes a
// row, which find an FP8 row's largest value by shuffles, so a row never leaves
// its registers between being read and being written.
//
// The angles are a token's own, shared by all its heads: the CTA computes the
// R/2 cosines and sines of each of its tokens once, into shared memory. A
// frequency is a 64-bit fraction of a turn, so position * frequency wraps where
// the angle does and keeps 2^-64 of a turn for every 1 in position; its upper 32 bits
// are the angle.
#include "sgq_cache.cuh"

namespace sgq {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t load_index(const void* p, int wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(p)[i] : (int64_t) static_cast<const int32_t*>(p)[i];
}

__device__ __forceinline__ uint4 ld16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// LPR lanes a row, 16 values a lane.
template <int FMT, int DT, bool INTERLEAVED, int LPR>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteArgs a) {
    extern __shared__ float2 turn[];     // [tokens][pairs]: factor * (cos, sin)
    pdl_wait();
    pdl_trigger();
    const int64_t t0 = (int64_t)blockIdx.x * a.tpc;
    const int tokens = (int)min((int64_t)a.tpc, a.T - t0);
    const int half = a.rope.half;
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int t = i / half;
        const uint64_t phase = (uint64_t)load_index(a.rope.positions, a.rope.wide, t0 + t) * a.rope.freqs[i - t * half];
        // half a turn is 1: sincospi's argument in [-1, 1)
        float s, c;
        sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
        turn[i] = make_float2(a.rope.factor * c, a.rope.factor * (a.rope.inverse ? -s : s));
    }
    __syncthreads();

    const int D = a.D, nch = D >> 3, turned = half >> 2;         // 16-byte pieces of a row, of its rotated part
    const int rows = a.q.n + 2 * a.k.n;
    const int lane = threadIdx.x % LPR;
    constexpr int kRows = kThreads / LPR;
    const int total = tokens * rows;
    for (int r0 = (int)blockIdx.y * kRows; r0 < total; r0 += (int)gridDim.y * kRows) {
        const int at = r0 + (int)threadIdx.x / LPR;
        const int t = min(at, total - 1) / rows, h = min(at, total - 1) - t * rows;
        const bool is_q = h < a.q.n, is_k = !is_q && h < a.q.n + a.k.n;
        int64_t slot = -1;
        if (!is_q) slot = load_index(a.slots, a.wide, t0 + t);
        const bool there = at < total && (is_q || (slot >= 0 && slot < a.c.pages * a.c.page.d));
        const Heads& src = is_q ? a.q : is_k ? a.k : a.v;
        const int head = is_q ? h : is_k ? h - a.q.n : h - a.q.n - a.k.n;
        const uint16_t* x = src.p + (t0 + t) * src.ts + head * src.hs;
        const bool rot = (is_q || is_k) && lane * 2 < turned;
        const int c0 = INTERLEAVED || !rot ? 2 * lane : lane;
        const int c1 = INTERLEAVED || !rot ? c0 + 1 : lane + (turned >> 1);
        float u[8] = {}, w[8] = {};
        if (there && c0 < nch) load8<DT>(ld16(x + c0 * 8), u);
        if (there && c1 < nch) load8<DT>(ld16(x + c1 * 8), w);
        if (rot) {
            const float2* cs = turn + t * half + lane * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 e = cs[i];
                float& p = INTERLEAVED ? (i < 4 ? u[2 * (i & 3)] : w[2 * (i & 3)]) : u[i];
                float& o = INTERLEAVED ? (i < 4 ? u[2 * (i & 3) + 1] : w[2 * (i & 3) + 1]) : w[i];
                const float first = p * e.x - o * e.y, second = p * e.y + o * e.x;
                p = first;
                o = second;
            }
        }
        if (is_q) {
            uint16_t* y = a.qo.p + (t0 + t) * a.qo.ts + head * a.qo.hs;
            st16_if(y + c0 * 8, pack8<DT>(u), there && c0 < nch);
            st16_if(y + c1 * 8, pack8<DT>(w), there && c1 < nch);
        }
        if (FMT == FMT_PT) {             // every lane takes part in the shuffles
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(u[i]), fabsf(w[i])));
            m = group_max<LPR>(m);
            if (!is_q && there) {
                const int64_t page = slot / a.c.page.d, place = slot - page * a.c.page.d;
                uint8_t* row = (is_k ? a.c.k : a.c.v) + page * a.c.ps + head * a.c.hs + place * a.c.ts;
                const float2 sr = per_token_scale(m);
                auto codes = [&](const float(&v)[8]) {
                    float f[8];
                    if (sr.x >= 0x1p-126f || sr.x == 0.0f) {     // the reciprocal is 0 for a scale of 0: every code is 0
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float2 q = div2_rn(make_float2(v[i], v[i + 1]), f2(-sr.x), f2(sr.y));
                            f[i] = q.x;
                            f[i + 1] = q.y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(v[i], sr.x);
                    }
                    return make_uint2(f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]), f32x4_to_e4m3x4(f[4], f[5], f[6], f[7]));
                };
                st8_if(row + c0 * 8, codes(u), c0 < nch);
                st8_if(row + c1 * 8, codes(w), c1 < nch);
                st_f32_if((is_k ? a.c.ks : a.c.vs) + (page * a.c.heads + head) * a.c.page.d + place, sr.x, lane == 0);
            }
        } else if (!is_q && there) {
            const int64_t page = slot / a.c.page.d, place = slot - page * a.c.page.d;
            uint8_t* row = (is_k ? a.c.k : a.c.v) + page * a.c.ps + head * a.c.hs + place * a.c.ts;
            st16_if(row + c0 * 16, pack8<DT>(u), c0 < nch);
            st16_if(row + c1 * 16, pack8<DT>(w), c1 < nch);
        }
    }
}

template <int FMT, int DT, bool INTERLEAVED>
auto pick(int lpr) {
    return lpr == 4 ? cache_write_kernel<FMT, DT, INTERLEAVED, 4>
           : lpr == 8 ? cache_write_kernel<FMT, DT, INTERLEAVED, 8> : cache_write_kernel<FMT, DT, INTERLEAVED, 16>;
}

template <int FMT, int DT>
auto pick(int lpr, bool interleaved) {
    return interleaved ? pick<FMT, DT, true>(lpr) : pick<FMT, DT, false>(lpr);
}

}  // namespace

cudaError_t launch_cache_write(int fmt, int dt, bool interleaved, const Device& dev, const WriteArgs& w, cudaStream_t stream) {
    WriteArgs a = w;
    const int units = (a.D + 15) / 16, lpr = units <= 4 ? 4 : units <= 8 ? 8 : 16;
    const int rows = a.q.n + 2 * a.k.n, per = kThreads / lpr;
    // Few tokens: a CTA for each pass over a token's rows, so that none waits for another; many: a
    // CTA walks over the rows of a token, or of several narrow ones, and shares their angles.
    const int sms = dev.sms > 0 ? dev.sms : 152;
    int split = 1;
    a.tpc = 1;
    if (a.T < 4 * (int64_t)sms) split = (rows + per - 1) / per;
    else while (a.tpc < 8 && a.tpc * rows < 4 * per && a.T >= 16 * (int64_t)sms * a.tpc) a.tpc *= 2;
    const int64_t ctas = (a.T + a.tpc - 1) / a.tpc;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const int smem = a.tpc * a.rope.half * (int)sizeof(float2);
    const auto k = fmt == FMT_PT ? (dt == DT_F16 ? pick<FMT_PT, DT_F16>(lpr, interleaved) : pick<FMT_PT, DT_BF16>(lpr, interleaved))
                                 : (dt == DT_F16 ? pick<FMT_16BIT, DT_F16>(lpr, interleaved) : pick<FMT_16BIT, DT_BF16>(lpr, interleaved));
    return launch_grid(k, dim3((unsigned)ctas, (unsigned)split), kThreads, smem, 1, dev.id, a, stream);
}

}  // namespace sgq
