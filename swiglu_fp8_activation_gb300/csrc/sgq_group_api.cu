// sgq_group_api.cu -- the C ABI declared in include/sgq_group.h: host-side
// argument checks, then the operation's launches.
#include "sgq_cache.cuh"

#include "sgq_group.h"

using namespace sgq;

namespace {

constexpr int64_t kMaxRows = SGQ_MAX_ROWS;   // counted in 32 bits, with room for a tile behind the last

bool bad_count(int64_t v) { return v < 0 || v > kMaxRows; }

}  // namespace

extern "C" {

int group_rows(int id_bytes, int64_t T, int64_t k, int64_t groups, const void* ids, int32_t* offsets, int32_t* rows,
               int32_t* slots, sgq_stream_t stream) {
    if (id_bytes != 4 && id_bytes != 8) return SGQ_ERR_INVALID_ARG;
    if (bad_count(T) || k < 1 || k > kMaxRows || groups < 1 || T > kMaxRows / k) return SGQ_ERR_INVALID_ARG;
    if (groups > SGQ_MAX_GROUPS) return SGQ_ERR_UNSUPPORTED;
    const size_t n = (size_t)(T * k);
    if (!offsets || (n && (!ids || !rows))) return SGQ_ERR_INVALID_ARG;
    if (!aligned(ids, (uintptr_t)id_bytes) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4))
        return SGQ_ERR_MISALIGNED;
    const Span spans[] = {{ids, n * id_bytes}, {offsets, (size_t)(groups + 1) * 4}, {rows, n * 4}, {slots, n * 4}};
    if (any_overlap(spans, 4)) return SGQ_ERR_INVALID_ARG;
    GroupRowsArgs a;
    a.ids = ids;
    a.offsets = offsets;
    a.rows = rows;
    a.slots = slots;
    a.n = (uint32_t)n;
    a.k = (uint32_t)k;
    a.groups = (int)groups;
    a.wide = id_bytes == 8;
    return launched(launch_group_rows(current_device(), a, static_cast<cudaStream_t>(stream)));
}

int grouped_gemm(int fmt, uint32_t flags, int64_t S, int64_t groups, int64_t N, int64_t K, int64_t x_rows,
                 const void* x, const void* x_scale, const void* w, const void* w_scale, const int32_t* offsets,
                 const int32_t* rows, void* out, sgq_stream_t stream) {
    if (fmt < SGQ_FMT_MXFP8 || fmt > SGQ_FMT_16BIT || (flags & ~SGQ_F_FP16)) return SGQ_ERR_INVALID_ARG;
    if (bad_count(S) || bad_count(x_rows) || groups < 1 || N <= 0 || K <= 0) return SGQ_ERR_INVALID_ARG;
    if (S > 0 && !rows && x_rows != S) return SGQ_ERR_INVALID_ARG;
    const int unit = fmt == SGQ_FMT_MXFP8 ? 32 : fmt == SGQ_FMT_FP8_BLOCK128 ? 128 : fmt == SGQ_FMT_FP8_PER_TOKEN ? 16 : 8;
    if (groups > SGQ_MAX_GROUPS || N % 8 != 0 || N > SGQ_MAX_WIDTH || K % unit != 0 || K > SGQ_MAX_WIDTH)
        return SGQ_ERR_UNSUPPORTED;
    if (S == 0) return SGQ_OK;
    const bool scaled = fmt != SGQ_FMT_16BIT;
    if (!w || !offsets || !out || (x_rows > 0 && !x) || (scaled && (!w_scale || (x_rows > 0 && !x_scale))) ||
        (!scaled && (x_scale || w_scale)))
        return SGQ_ERR_INVALID_ARG;
    const uintptr_t xsa = fmt == SGQ_FMT_MXFP8 ? 1 : 4, wsa = fmt == SGQ_FMT_MXFP8 ? 16 : 4;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(x_scale, xsa) || !aligned(w_scale, wsa) ||
        !aligned(offsets, 4) || !aligned(rows, 4))
        return SGQ_ERR_MISALIGNED;
    const size_t e = scaled ? 1 : 2;
    size_t xs_bytes = 0, ws_bytes = 0;
    if (fmt == SGQ_FMT_MXFP8) {
        xs_bytes = (size_t)(x_rows * (K / 32));
        ws_bytes = (size_t)(groups * round_up(N, 128) * round_up(K / 32, 4));
    } else if (fmt == SGQ_FMT_FP8_BLOCK128) {
        xs_bytes = (size_t)(x_rows * (K / 128)) * 4;
        ws_bytes = (size_t)(groups * ((N + 127) / 128) * (K / 128)) * 4;
    } else if (fmt == SGQ_FMT_FP8_PER_TOKEN) {
        xs_bytes = (size_t)x_rows * 4;
        ws_bytes = (size_t)(groups * N) * 4;
    }
    const size_t out_bytes = (size_t)(S * N) * 2;
    const Span in[] = {{x, (size_t)(x_rows * K) * e}, {x_scale, xs_bytes}, {w, (size_t)(groups * N * K) * e},
                       {w_scale, ws_bytes}, {offsets, (size_t)(groups + 1) * 4}, {rows, (size_t)S * 4}};
    for (const Span& s : in)
        if (overlap(s.p, s.n, out, out_bytes)) return SGQ_ERR_INVALID_ARG;
    GroupGemmArgs a;
    a.x = x;
    a.xs = x_scale;
    a.w = w;
    a.ws = w_scale;
    a.offsets = offsets;
    a.rows = rows;
    a.out = static_cast<uint16_t*>(out);
    a.x_rows = x_rows;
    a.S = (int)S;
    a.groups = (int)groups;
    a.N = (int)N;
    a.K = (int)K;
    return launched(launch_grouped_gemm(fmt, (flags & SGQ_F_FP16) ? DT_F16 : DT_BF16, current_device(), a,
                                        static_cast<cudaStream_t>(stream)));
}

int combine_rows(uint32_t flags, int64_t T, int64_t k, int64_t S, int64_t N, const void* y, const int32_t* slots,
                 const float* weights, void* out, sgq_stream_t stream) {
    if (flags & ~SGQ_F_FP16) return SGQ_ERR_INVALID_ARG;
    if (bad_count(T) || k < 1 || k > kMaxRows || T > kMaxRows / k || bad_count(S) || N <= 0) return SGQ_ERR_INVALID_ARG;
    if (N % 8 != 0 || N > SGQ_MAX_WIDTH || T > 0x7FFFFFFF / ((N + 511) / 512)) return SGQ_ERR_UNSUPPORTED;   // a CTA each 512 columns
    if (T == 0) return SGQ_OK;
    if (!slots || !out || (S > 0 && !y)) return SGQ_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(out, 16) || !aligned(slots, 4) || !aligned(weights, 4)) return SGQ_ERR_MISALIGNED;
    const size_t out_bytes = (size_t)(T * N) * 2, n = (size_t)(T * k) * 4;
    if (overlap(out, out_bytes, y, (size_t)(S * N) * 2) || overlap(out, out_bytes, slots, n) ||
        overlap(out, out_bytes, weights, n))
        return SGQ_ERR_INVALID_ARG;
    CombineArgs a;
    a.y = static_cast<const uint16_t*>(y);
    a.slots = slots;
    a.weights = weights;
    a.out = static_cast<uint16_t*>(out);
    a.T = T;
    a.S = S;
    a.k = (int)k;
    a.N = (int)N;
    a.nblk = 0;
    return launched(launch_combine((flags & SGQ_F_FP16) ? DT_F16 : DT_BF16, current_device(), a,
                                   static_cast<cudaStream_t>(stream)));
}

int64_t sgq_lora_workspace_bytes(int64_t S, int64_t groups, int64_t R) {
    if (S < 0 || S > kMaxRows || groups < 1 || groups > SGQ_MAX_GROUPS || R < 1 || R > SGQ_MAX_RANK) return 0;
    return lora_few(S, groups, R) ? 0 : S * lora_row_bytes((int)R);
}

int lora_add(uint32_t flags, int64_t T, int64_t S, int64_t groups, int64_t R, int64_t K, int64_t N, const void* x,
             const void* a, const void* b, const float* scaling, const int32_t* offsets, const int32_t* rows,
             const int32_t* slots, void* y, void* workspace, sgq_stream_t stream) {
    if (flags & ~SGQ_F_FP16) return SGQ_ERR_INVALID_ARG;
    if (bad_count(T) || bad_count(S) || groups < 1 || R <= 0 || K <= 0 || N <= 0) return SGQ_ERR_INVALID_ARG;
    if (groups > SGQ_MAX_GROUPS || R % 8 != 0 || R > SGQ_MAX_RANK || K % 8 != 0 || K > SGQ_MAX_WIDTH || N % 8 != 0 ||
        N > SGQ_MAX_WIDTH)
        return SGQ_ERR_UNSUPPORTED;
    if (S == 0 || T == 0) return SGQ_OK;
    if (!rows != !slots || (!rows && S != T)) return SGQ_ERR_INVALID_ARG;
    const int64_t ws_bytes = sgq_lora_workspace_bytes(S, groups, R);
    if (!x || !a || !b || !offsets || !y || (ws_bytes > 0 && !workspace)) return SGQ_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(y, 16) || !aligned(workspace, 16) ||
        !aligned(scaling, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4))
        return SGQ_ERR_MISALIGNED;
    const Span out[] = {{y, (size_t)(T * N) * 2}, {workspace, (size_t)ws_bytes}};
    const Span in[] = {{x, (size_t)(T * K) * 2}, {a, (size_t)(groups * R * K) * 2}, {b, (size_t)(groups * N * R) * 2},
                       {scaling, (size_t)groups * 4}, {offsets, (size_t)(groups + 1) * 4}, {rows, (size_t)S * 4},
                       {slots, (size_t)T * 4}};
    if (any_overlap(out, 2)) return SGQ_ERR_INVALID_ARG;
    for (const Span& o : out)
        for (const Span& i : in)
            if (overlap(o.p, o.n, i.p, i.n)) return SGQ_ERR_INVALID_ARG;
    LoraArgs l;
    l.x = static_cast<const uint16_t*>(x);
    l.a = static_cast<const uint16_t*>(a);
    l.b = static_cast<const uint16_t*>(b);
    l.scaling = scaling;
    l.offsets = offsets;
    l.rows = rows;
    l.slots = slots;
    l.y = static_cast<uint16_t*>(y);
    l.v = workspace;
    l.T = T;
    l.S = (int)S;
    l.groups = (int)groups;
    l.R = (int)R;
    l.K = (int)K;
    l.N = (int)N;
    return launched(launch_lora((flags & SGQ_F_FP16) ? DT_F16 : DT_BF16, current_device(), l,
                                static_cast<cudaStream_t>(stream)));
}

int sgq_wait_timeouts(uint32_t* count) {
    if (!count) return SGQ_ERR_INVALID_ARG;
    uint32_t gemm = 0, lora = 0, attend = 0;
    // the copies of the counts wait for the default stream alone, which streams
    // made not to block it do not wait for either
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = gemm_gave_up(&gemm);
    if (e == cudaSuccess) e = lora_gave_up(&lora);
    if (e == cudaSuccess) e = attend_gave_up(&attend);
    if (e == cudaSuccess) *count = gemm + lora + attend;
    return launched(e);
}

}  // extern "C"
