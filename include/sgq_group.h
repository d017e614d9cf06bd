/*
 * sgq_group.h -- products over ragged groups of rows, for the rows that
 * sgq.h's operations write (NVIDIA GB300, sm_103a):
 *
 *   group_rows     group ids -> rows in group order (the routing of an expert
 *                  layer, or the adapters of a batch's requests)
 *   grouped_gemm   out[s] = x[rows[s]] . w[g]^T for the slots s of group g:
 *                  FP8 rows and weights in the three formats of sgq.h, or
 *                  16-bit ones
 *   combine_rows   out[t] = sum_j weights[t][j] * y[slots[t][j]]: the end of
 *                  an expert layer
 *   lora_add       y[t] += scaling[g] * (x[t] . a[g]^T) . b[g]^T: the low-rank
 *                  adapters of many requests beside a shared projection
 *
 * An expert layer in these terms: rmsnorm_add_quant writes quantised rows,
 * group_rows orders the router's choices, grouped_gemm gathers the rows of
 * each expert (gate and up), swiglu_quant quantises the activation,
 * grouped_gemm runs the down product and combine_rows sums each token's rows.
 *
 * Slots and groups. S slots hold rows in group order. offsets [groups + 1]
 * (int32, on the device) ascends; the slots of group g are offsets[g] <= s <
 * offsets[g + 1], so a group may be empty, and slots before offsets[0] or from
 * offsets[groups] on belong to no group. No host copy of it is needed.
 * Offsets are held to 0 <= offsets[g] <= S and to ascending order by the
 * kernels: a value outside reads as the nearest one inside, so no offsets
 * make a kernel touch memory outside the tensors.
 *
 * Conventions are sgq.h's: pointers of the current device, owned by the caller, contiguous
 * row-major tensors, E4M3 bytes, status codes, host checks before any launch
 * with every buffer untouched by a refused call, nothing allocated, no
 * synchronisation, CUDA-graph capture allowed, programmatic dependent launch
 * (every kernel here waits for the kernel before it before it reads or
 * writes any tensor). Outputs may not overlap inputs or each other except
 * where stated. Every result is the same on every run: no float atomics. (The
 * order of grouped_gemm's and lora_add's sums follows the call's sizes and the
 * count of multiprocessors, which sgq_set_sm_budget replaces; so may its last bit.)
 * Non-finite FP8 codes, scales or 16-bit values give non-finite or
 * unspecified results in the rows that they enter, and in no others.
 *
 * State kept between calls, beside sgq.h's: for group_rows, whether the device
 * runs clusters of 16 CTAs; and a count that sgq_wait_timeouts returns. Every
 * wait inside grouped_gemm and lora_add is limited to some seconds. A launch in
 * which one runs out (the device made no progress, or was held by others for that
 * long) ends and leaves its outputs unspecified; its call has returned SGQ_OK
 * by then, and sgq_wait_timeouts is where it shows.
 */
#ifndef SGQ_GROUP_H
#define SGQ_GROUP_H

#include "sgq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SGQ_MAX_GROUPS 1024     /* groups of one call */
#define SGQ_MAX_RANK 128        /* rank of lora_add */
#define SGQ_MAX_ROWS 0x7FFF0000 /* rows, slots or ids of one call */

/* grouped_gemm's fmt beside sgq_format_t: 16-bit rows and weights, no scales. */
#define SGQ_FMT_16BIT 3

/*
 * Rows in group order, stable: ids of one group keep their order.
 *
 *   offsets[g] = number of ids in [0, g)                        g = 0 .. groups
 *   slots[i]   = offsets[ids[i]] + number of j < i with ids[j] = ids[i];
 *                -1 where ids[i] is outside [0, groups) (a dropped token, an
 *                expert of another rank)
 *   rows[slots[i]] = i / k                 (the token that id i belongs to)
 *   rows[s] = -1 for the slots s >= offsets[groups]
 *
 * Arguments:
 *   id_bytes      4 (int32 ids) or 8 (int64 ids)
 *   T, k          ids is [T, k]; T * k <= SGQ_MAX_ROWS; k >= 1
 *   groups        1 .. SGQ_MAX_GROUPS
 *   ids           [T, k], read; aligned to id_bytes
 *   offsets       [groups + 1] int32, written (also when T = 0)
 *   rows          [T * k] int32, written
 *   slots         [T, k] int32, written, or NULL
 */
int group_rows(int id_bytes, int64_t T, int64_t k, int64_t groups, const void* ids, int32_t* offsets,
               int32_t* rows, int32_t* slots, sgq_stream_t stream);

/*
 * Matrix products grouped by ragged sets of rows. For group g and slot s of it,
 * with r = rows[s] (r = s where rows is NULL):
 *
 *   MXFP8      out[s][n] = sum_k x[r][k] 2^(xs[r][k/32]-127) * w[g][n][k] 2^(ws[g][n][k/32]-127)
 *   1x128      out[s][n] = sum_b xs[r][b] * ws[g][n/128][b] * sum_{k in block b} x[r][k] w[g][n][k]
 *   per-token  out[s][n] = xs[r] * ws[g][n] * sum_k x[r][k] w[g][n][k]
 *   16-bit     out[s][n] = sum_k x[r][k] w[g][n][k]
 *
 * summed in fp32 and rounded once. The scales enter in fp32: MXFP8's with every
 * term, exactly; 1x128's as xs * ws; per-token's one after the other, xs first. What leaves
 * fp32's range on the way is 0 or infinite (or NaN: the sum of both infinities).
 * A row index outside [0, x_rows) stands for
 * a row of zeros. Slots of no group keep what out held.
 *
 * The width of the tiles is chosen for S / groups slots a group, those of no
 * group among them, and has no influence on which slots are computed.
 *
 * Arguments:
 *   fmt           sgq_format_t or SGQ_FMT_16BIT
 *   flags         SGQ_F_FP16: out is fp16, not bf16, and so are x and w with
 *                 SGQ_FMT_16BIT (others rejected)
 *   S             slots, at most SGQ_MAX_ROWS
 *   groups        1 .. SGQ_MAX_GROUPS
 *   N             output width, a multiple of 8, at most SGQ_MAX_WIDTH
 *   K             length of the products, at most SGQ_MAX_WIDTH: a multiple of
 *                 32 (MXFP8), 128 (1x128), 16 (per-token) or 8 (16-bit)
 *   x_rows        rows of x, at most SGQ_MAX_ROWS; S where rows is NULL
 *   x             [x_rows, K], read
 *   x_scale       what sgq.h's quantisation wrote row-major: [x_rows, K/32]
 *                 E8M0, [x_rows, K/128] or [x_rows, 1] fp32; NULL for 16-bit
 *   w             [groups, N, K], read
 *   w_scale       weights' scales, laid out once:
 *                 MXFP8      each group's codes in the swizzled tiles of
 *                            SGQ_F_SCALE_SWIZZLED, [groups, N up to 128, K/32
 *                            up to 4]; quantize_fp8 of [groups * N, K] rows
 *                            leaves this when N % 128 == 0; 16-byte aligned
 *                 1x128      fp32 [groups, ceil(N/128), K/128]: one scale per
 *                            128 x 128 block
 *                 per-token  fp32 [groups, N]: one scale per output channel
 *                 16-bit     NULL
 *   offsets       [groups + 1] int32, read
 *   rows          [S] int32, read, or NULL
 *   out           [S, N], written
 */
int grouped_gemm(int fmt, uint32_t flags, int64_t S, int64_t groups, int64_t N, int64_t K, int64_t x_rows,
                 const void* x, const void* x_scale, const void* w, const void* w_scale,
                 const int32_t* offsets, const int32_t* rows, void* out, sgq_stream_t stream);

/*
 * The weighted sum of each token's k rows:
 *
 *   out[t][n] = sum_j weights[t][j] * y[slots[t][j]][n]      (fp32, in order of j; rounded once)
 *
 * A slot outside [0, S) adds nothing and its weight is not used; a token with
 * no slot inside gets zeros.
 *
 * Arguments:
 *   flags         SGQ_F_FP16: y and out are fp16, not bf16 (others rejected)
 *   T, k          tokens, rows a token (k >= 1); T * k <= SGQ_MAX_ROWS
 *   S             rows of y, at most SGQ_MAX_ROWS
 *   N             width, a multiple of 8, at most SGQ_MAX_WIDTH;
 *                 T * ceil(N / 512) < 2^31
 *   y             [S, N], read
 *   slots         [T, k] int32, read
 *   weights       [T, k] fp32, read, or NULL (every weight 1)
 *   out           [T, N], written
 */
int combine_rows(uint32_t flags, int64_t T, int64_t k, int64_t S, int64_t N, const void* y,
                 const int32_t* slots, const float* weights, void* out, sgq_stream_t stream);

/*
 * The low-rank adapters of many requests, added in place to the output of a
 * shared projection. For group (adapter) g and slot s of it, with t = rows[s]
 * (t = s where rows is NULL):
 *
 *   v       = x[t] . a[g]^T                                  (fp32, not rounded)
 *   y[t]    = y[t] + scaling[g] * (v . b[g]^T)               (fp32, rounded once)
 *
 * (v is multiplied in 16-bit parts that together hold its 24 bits; with fp16
 * rows and a workspace, the last of them may lack up to 2^-39 of the row's
 * largest |v|.)
 *
 * Rows of y that belong to no slot are left as they are. rows must come with
 * slots (both from group_rows with k = 1): a slot s whose token t does not
 * hold slots[t] = s, or whose t is outside [0, T), is passed over, so no row
 * of y is updated twice whatever rows holds. One launch on the stream, without a
 * workspace, where the slots are few for the adapters (S up to 512, S * R up to
 * 8192 and 128 * groups), two else: the two add in different orders.
 *
 * Arguments:
 *   flags         SGQ_F_FP16: x, a, b and y are fp16, not bf16 (others rejected)
 *   T             rows of x and y, at most SGQ_MAX_ROWS
 *   S             slots, at most SGQ_MAX_ROWS; T where rows is NULL
 *   groups        adapters, 1 .. SGQ_MAX_GROUPS
 *   R             rank, a multiple of 8, at most SGQ_MAX_RANK
 *   K, N          widths of x and y, multiples of 8, at most SGQ_MAX_WIDTH
 *   x             [T, K], read
 *   a             [groups, R, K], read
 *   b             [groups, N, R], read
 *   scaling       [groups] fp32, read, or NULL (every factor 1)
 *   offsets       [groups + 1] int32, read
 *   rows, slots   [S] and [T] int32, read, or both NULL
 *   y             [T, N], read and written
 *   workspace     sgq_lora_workspace_bytes(S, groups, R) bytes, written
 *                 (16-byte aligned; may be NULL where that is 0); calls that
 *                 may run at the same time (other streams, graphs) need
 *                 workspaces of their own
 */
int lora_add(uint32_t flags, int64_t T, int64_t S, int64_t groups, int64_t R, int64_t K, int64_t N,
             const void* x, const void* a, const void* b, const float* scaling, const int32_t* offsets,
             const int32_t* rows, const int32_t* slots, void* y, void* workspace, sgq_stream_t stream);

/* Bytes of lora_add's workspace; 0 where it needs none, or an argument is outside its range. */
int64_t sgq_lora_workspace_bytes(int64_t S, int64_t groups, int64_t R);

/*
 * Launches of grouped_gemm and lora_add on the current device, since the
 * library was loaded, in which a wait inside the kernel ran out of time (see
 * above). A diagnosis: it waits for the device, all streams of it, and may not be
 * called during graph capture. NULL returns SGQ_ERR_INVALID_ARG.
 */
int sgq_wait_timeouts(uint32_t* count);

#ifdef __cplusplus
}
#endif

#endif /* SGQ_GROUP_H */
