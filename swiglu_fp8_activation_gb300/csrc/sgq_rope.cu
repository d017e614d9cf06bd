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
// the angle does and keeps 2^-64 of a turn for every 1 in position. The angle is that, rounded to
// fp32: its upper 32 bits alone would leave a slow pair near the beginning, 2^-30 of a turn and less a position
// in contexts stretched far, a sine of a few bits.
#include "sgq_cache.cuh"

namespace sgq {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ uint4 ld16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// LPR lanes a row, 16 values a lane; a.per threads (a multiple of a warp) work on one token, its heads one after the other.
// Eight CTAs of 128 threads a multiprocessor: nine (56 registers, a few spilled) are better at large sizes without rows asked for ahead (33.3 us for
// 34.0: 8192 tokens, 32 heads of 128 and 8 of k and v, E4M3) but not with them (31.2 for 30.0, 168 MB, 6170 GB/s), nor at small ones (2048 tokens: 8.9
// for 7.7). Reads of the next row held in registers cost more warps than they gain (40 heads of 16384 tokens turned: 65 us for 55).
template <int FMT, int DT, bool INTERLEAVED, int LPR>
__global__ void __launch_bounds__(kThreads, 8) cache_write_kernel(const WriteArgs a) {
    extern __shared__ float2 turn[];     // [tokens][8][pairs / 8]: factor * (cos, sin), a lane's 8 pairs a row apart (no bank twice)
    pdl_wait();
    pdl_trigger();
    const int tokens = kThreads / a.per, token = (int)threadIdx.x / a.per;
    const int64_t t0 = (int64_t)blockIdx.x * tokens, t = t0 + token;
    const bool live = t < a.T;
    const int half = a.rope.half, nch = a.D >> 3, turned = half >> 2;            // 16-byte pieces of a row, of its rotated part
    const int lane = (int)threadIdx.x % LPR, heads = a.per / LPR * (int)gridDim.y;       // that are worked on at once
    const int first = ((int)threadIdx.x % a.per) / LPR + (int)blockIdx.y * (a.per / LPR);
    const bool rot = lane * 2 < turned;
    // the lane's pieces of a rotated row (of another: 2 lane, 2 lane + 1)
    const int c0 = INTERLEAVED || !rot ? 2 * lane : lane, c1 = INTERLEAVED || !rot ? 2 * lane + 1 : lane + (turned >> 1);

    const bool on0 = live && c0 < nch, on1 = live && c1 < nch;
    // The lane's two pieces of a row at p, the second `apart` values behind the first.
    auto read = [&](const uint16_t* p, int apart, bool first_on, bool second_on, uint4& u, uint4& w) {
        u = w = make_uint4(0, 0, 0, 0);
        if (first_on) u = ld16(p);
        if (second_on) w = ld16(p + apart);
    };
    const int apart = (c1 - c0) * 8;

    // Rows that L2 does not hold: q's are on their way to it while the angles are computed.
    if (a.ahead && live && (lane & 3) == 0 && lane * 16 < a.D) {
        const uint16_t* x = a.q.p + t * a.q.ts + first * a.q.hs + lane * 16;
        for (int h = first; h < a.q.n; h += heads, x += heads * a.q.hs) asm volatile("prefetch.global.L2 [%0];" ::"l"(x) : "memory");
    }

    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int at = i / half;
        if (t0 + at >= a.T) break;
        const int pair = i - at * half;
        const uint64_t phase = (uint64_t)load_index(a.rope.positions, a.rope.wide, t0 + at) * a.rope.freqs[pair];
        // half a turn is 1: sincospi's argument in [-1, 1]
        float s, c;
        sincospif((float)(int64_t)phase * 0x1p-63f, &s, &c);
        turn[at * half + (pair & 7) * (half >> 3) + (pair >> 3)] = make_float2(a.rope.factor * c, a.rope.factor * (a.rope.inverse ? -s : s));
    }
    __syncthreads();
    const float2* cs = turn + token * half + lane;
    const int apart_cs = half >> 3;
    auto rotate = [&](float (&u)[8], float (&w)[8]) {
        if (!rot) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 e = cs[i * apart_cs];
            float& p = INTERLEAVED ? (i < 4 ? u[2 * (i & 3)] : w[2 * (i & 3)]) : u[i];
            float& o = INTERLEAVED ? (i < 4 ? u[2 * (i & 3) + 1] : w[2 * (i & 3) + 1]) : w[i];
            const float x = p * e.x - o * e.y, y = p * e.y + o * e.x;
            p = x;
            o = y;
        }
    };
    if (gridDim.z == 1 || blockIdx.z == 0) {
        const uint16_t* x = a.q.p + t * a.q.ts + first * a.q.hs + c0 * 8;
        uint16_t* y = a.qo.p + t * a.qo.ts + first * a.qo.hs + c0 * 8;
        const int64_t xs = heads * a.q.hs, ys = heads * a.qo.hs;
        for (int h = first; h < a.q.n; h += heads, x += xs, y += ys) {
            uint4 r, e;
            read(x, apart, on0, on1, r, e);
            float u[8], w[8];
            load8<DT>(r, u);
            load8<DT>(e, w);
            rotate(u, w);
            st16_if(y, pack8<DT>(u), on0);
            st16_if(y + apart, pack8<DT>(w), on1);
        }
    }
    if (a.k.n == 0 || (gridDim.z > 1 && blockIdx.z == 0)) return;

    const int64_t slot = live ? load_index(a.slots, a.wide, t) : -1;
    const bool there = slot >= 0 && slot < a.c.pages * a.c.page.d;
    int place = 0;
    const int64_t page = there ? page_of_slot(slot, a.c.page, place) : 0;
    // A row of 16 values a lane into the cache; every lane takes part in the shuffles.
    constexpr int kPiece = FMT == FMT_PT ? 8 : 16;               // bytes of 8 values
    auto put = [&](const float (&u)[8], const float (&w)[8], uint8_t* row, float* scale, int off, bool first_on, bool second_on, bool on) {
        if (FMT != FMT_PT) {
            st16_if(row, pack8<DT>(u), on && first_on);
            st16_if(row + off * 2, pack8<DT>(w), on && second_on);
            return;
        }
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(u[i]), fabsf(w[i])));
        const float2 sr = per_token_scale(group_max<LPR>(m));
        auto codes = [&](const float(&v)[8]) {
            float f[8];
            if (sr.x >= 0x1p-126f || sr.x == 0.0f) {             // the reciprocal is 0 for a scale of 0: every code is 0
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
        st8_if(row, codes(u), on && first_on);
        st8_if(row + off, codes(w), on && second_on);
        st_f32_if(scale, sr.x, on && lane == 0);
    };
    const bool v0 = live && 2 * lane < nch, v1 = live && 2 * lane + 1 < nch;
    for (int h = first; h - first < a.k.n; h += heads) {         // the same number of turns for all lanes
        const bool on = there && h < a.k.n;
        uint4 k0, k1, w0, w1;
        read(a.k.p + t * a.k.ts + h * a.k.hs + c0 * 8, apart, on && on0, on && on1, k0, k1);
        read(a.v.p + t * a.v.ts + h * a.v.hs + lane * 16, 8, on && v0, on && v1, w0, w1);
        const int64_t row = page * a.c.ps + h * a.c.hs + place * a.c.ts, scale = (page * a.c.heads + h) * a.c.page.d + place;
        float u[8], w[8];
        load8<DT>(k0, u);
        load8<DT>(k1, w);
        rotate(u, w);
        put(u, w, a.c.k + row + c0 * kPiece, a.c.ks + scale, apart, on0, on1, on);
        load8<DT>(w0, u);
        load8<DT>(w1, w);
        put(u, w, a.c.v + row + lane * 2 * kPiece, a.c.vs + scale, 8, v0, v1, on);
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
    const int most = a.q.n > a.k.n ? a.q.n : a.k.n;
    // Few tokens: as many threads a token as it has heads, in several CTAs where they do not fit in one, and q beside k and v, so
    // that none waits for another; many: two warps a token, one where it has few heads, whose lanes keep their part of the angles.
    const int sms = dev.sms > 0 ? dev.sms : 152;
    int split = 1;
    a.per = most * lpr < 128 ? 32 : 64;
    if (a.T < 8 * (int64_t)sms) {
        while (a.per < kThreads && a.per / lpr < most) a.per *= 2;
        if (a.T < 2 * (int64_t)sms) split = (most + a.per / lpr - 1) / (a.per / lpr);
    }
    const int tokens = kThreads / a.per;
    // Rows are asked for ahead where what is read and written passes L2 by (128 MB). 8192 tokens, 32 heads of 128 and 8 of k and v: bf16 31.5 us, else
    // 33.8, E4M3 30.0 and 34.0; 40 heads of 16384 tokens turned: 50.2 and 54.6; but in L2, 2048 tokens, E4M3: 8.0 and 7.7; k and v too: 30.3 and 50.3.
    a.ahead = a.T * (a.q.n + 2 * (int64_t)a.k.n) * a.D * 4 > (int64_t)128 << 20;
    const int64_t ctas = (a.T + tokens - 1) / tokens;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const int smem = tokens * a.rope.half * (int)sizeof(float2);
    const auto k = fmt == FMT_PT ? (dt == DT_F16 ? pick<FMT_PT, DT_F16>(lpr, interleaved) : pick<FMT_PT, DT_BF16>(lpr, interleaved))
                                 : (dt == DT_F16 ? pick<FMT_16BIT, DT_F16>(lpr, interleaved) : pick<FMT_16BIT, DT_BF16>(lpr, interleaved));
    return launch_grid(k, dim3((unsigned)ctas, (unsigned)split, (unsigned)(a.q.n > 0 && a.k.n > 0 && a.T < 2 * (int64_t)sms ? 2 : 1)), kThreads, smem, 1, dev.id, a, stream);
}

}  // namespace sgq
