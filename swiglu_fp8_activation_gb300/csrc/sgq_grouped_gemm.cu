// sgq_grouped_gemm.cu -- matrix products grouped by ragged sets of rows
// (include/sgq_group.h, grouped_gemm).
//
// A first form, right for every case: 64 x 64 output tiles, operands widened
// to fp32 in shared memory, fp32 multiply-adds, each 32 products scaled.
#include "sgq_group.cuh"

namespace sgq {

namespace {

constexpr int kTile = 64, kStep = 32;

__device__ __forceinline__ float e4m3_value(uint32_t c) {
    uint32_t h;
    asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(h) : "r"(c));
    return f16x2_to_f32x2(h).x;
}

template <int DT>
__device__ __forceinline__ float value16(uint16_t v) {
    return DT == DT_BF16 ? __uint_as_float((uint32_t)v << 16) : f16x2_to_f32x2(v).x;
}

// Stored value k of row r of x, and of channel n of group g; 0 outside.
template <int FMT, int DT>
__device__ __forceinline__ float x_value(const GroupGemmArgs& a, int64_t r, int k) {
    if (r < 0 || r >= a.x_rows || k >= a.K) return 0.0f;
    const int64_t i = r * a.K + k;
    return FMT == FMT_16BIT ? value16<DT>(static_cast<const uint16_t*>(a.x)[i]) : e4m3_value(static_cast<const uint8_t*>(a.x)[i]);
}

template <int FMT, int DT>
__device__ __forceinline__ float w_value(const GroupGemmArgs& a, int g, int n, int k) {
    if (n >= a.N || k >= a.K) return 0.0f;
    const int64_t i = ((int64_t)g * a.N + n) * a.K + k;
    return FMT == FMT_16BIT ? value16<DT>(static_cast<const uint16_t*>(a.w)[i]) : e4m3_value(static_cast<const uint8_t*>(a.w)[i]);
}

// The scale of the 32 products from k on (one MX block, part of a 128-block).
template <int FMT>
__device__ __forceinline__ float scale_of(const GroupGemmArgs& a, int64_t r, int g, int n, int k) {
    if (FMT == FMT_16BIT || r < 0 || r >= a.x_rows || n >= a.N) return 1.0f;
    if (FMT == FMT_MX) {
        const int64_t Np = (a.N + 127) / 128 * 128, Kp = (a.K / 32 + 3) / 4;
        const int b = k / 32;
        const int64_t tile = ((int64_t)g * Np + n / 128 * 128) * Kp * 4 + (int64_t)(b / 4) * 512;
        const int cw = static_cast<const uint8_t*>(a.ws)[tile + (n % 32) * 16 + (n / 32 % 4) * 4 + b % 4];
        const int cx = static_cast<const uint8_t*>(a.xs)[r * (a.K / 32) + b];
        return ldexpf(1.0f, cw + cx - 254);
    }
    if (FMT == FMT_B128)
        return static_cast<const float*>(a.xs)[r * (a.K / 128) + k / 128] *
               static_cast<const float*>(a.ws)[((int64_t)g * ((a.N + 127) / 128) + n / 128) * (a.K / 128) + k / 128];
    return static_cast<const float*>(a.xs)[r] * static_cast<const float*>(a.ws)[(int64_t)g * a.N + n];
}

template <int FMT, int DT>
__global__ void __launch_bounds__(256) grouped_gemm_kernel(const GroupGemmArgs a) {
    __shared__ float xs[kStep][kTile + 1], ws[kStep][kTile + 1];
    pdl_wait();
    pdl_trigger();
    // the group and first slot of this CTA's tile
    int tile = blockIdx.x, g = 0, lo = 0, hi = 0, prev = 0;
    for (;; ++g) {
        if (g == a.groups) return;
        lo = held(a.offsets[g], prev, a.S);
        hi = held(a.offsets[g + 1], lo, a.S);
        prev = lo;
        const int tiles = (hi - lo + kTile - 1) / kTile;
        if (tile < tiles) break;
        tile -= tiles;
    }
    const int s0 = lo + tile * kTile, n0 = blockIdx.y * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
            const int r = i / kStep, k = i % kStep, s = s0 + r;
            const int64_t row = s < hi ? (a.rows ? a.rows[s] : s) : -1;
            xs[k][r] = x_value<FMT, DT>(a, row, k0 + k);
            ws[k][r] = w_value<FMT, DT>(a, g, n0 + r, k0 + k);
        }
        __syncthreads();
        float part[4][4] = {};
        for (int k = 0; k < kStep; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) part[i][j] = fmaf(xs[k][ty * 4 + i], ws[k][tx + 16 * j], part[i][j]);
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + ty * 4 + i;
            const int64_t row = s < hi ? (a.rows ? a.rows[s] : s) : -1;
            for (int j = 0; j < 4; ++j)
                acc[i][j] = fmaf(part[i][j], scale_of<FMT>(a, row, g, n0 + tx + 16 * j, k0), acc[i][j]);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int s = s0 + ty * 4 + i, n = n0 + tx + 16 * j;
            if (s < hi && n < a.N)
                a.out[(int64_t)s * a.N + n] =
                    (uint16_t)(DT == DT_F16 ? f32x2_to_f16x2(acc[i][j], 0.0f) : f32x2_to_bf16x2(acc[i][j], 0.0f));
        }
}

template <int DT>
cudaError_t run(int fmt, const Device& dev, const GroupGemmArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.S + kTile - 1) / kTile + a.groups), (unsigned)((a.N + kTile - 1) / kTile));
    auto k = fmt == FMT_MX ? grouped_gemm_kernel<FMT_MX, DT>
             : fmt == FMT_B128 ? grouped_gemm_kernel<FMT_B128, DT>
             : fmt == FMT_PT ? grouped_gemm_kernel<FMT_PT, DT> : grouped_gemm_kernel<FMT_16BIT, DT>;
    return launch_grid(k, grid, 256, 0, 1, dev.id, a, stream);
}

}  // namespace

cudaError_t launch_grouped_gemm(int fmt, int dt, const Device& dev, const GroupGemmArgs& a, cudaStream_t stream) {
    return dt == DT_F16 ? run<DT_F16>(fmt, dev, a, stream) : run<DT_BF16>(fmt, dev, a, stream);
}

}  // namespace sgq
