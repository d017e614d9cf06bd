/*
 * sgq_cache.h -- a paged key-value cache and the attention that reads it, for
 * the step between a decoder layer's projections (NVIDIA GB300, sm_103a):
 *
 *   rope             rotary positions on heads, and their gradient
 *   cache_write      rotates keys, quantises keys and values and writes them
 *                    into the cache; rotates the queries in the same launch
 *   cache_read       rows of the cache as 16-bit values
 *   paged_attention  attention of one new token a sequence over its pages
 *
 * A decode step in these terms: a projection leaves q, k and v side by side,
 * cache_write rotates q and k and puts k and v into the cache, paged_attention
 * attends over it, and the rows go on to the output projection
 * (quantize_fp8 or rmsnorm_add_quant of sgq.h, grouped_gemm of sgq_group.h).
 *
 * Rows, pages and slots. A row is the D values of one head of one token. The
 * cache holds `pages` pages of page_size tokens for each of its heads: value i
 * of head h of the token at place p of page b is element
 *     b * page_stride + h * head_stride + p * token_stride + i
 * of k (or v), so that a page's tokens of one head may lie side by side, or a
 * token's heads. A slot names a token's place: slot = b * page_size + p.
 *
 * Formats. SGQ_FMT_16BIT: rows of bf16, or fp16 with SGQ_F_FP16.
 * SGQ_FMT_FP8_PER_TOKEN: E4M3 codes and one fp32 scale a row by sgq.h's rule for
 * rows (s = fp32(amax / 448), q = E4M3_rn_satfinite(fp32(src / s))), the scales in
 * k_scale and v_scale at (b * heads + h) * page_size + p; the 16-bit tensors beside
 * the cache are bf16, or fp16 with SGQ_F_FP16. Two rows a token and head of two
 * times D bytes are 2 (D + 4) bytes with it, not 4 D. The 1x128 rule on heads of 128 is
 * the same as this one.
 *
 * Conventions are sgq.h's: device pointers of the current device, owned by the
 * caller (the structs here are host structs, read during the call only), status
 * codes, host checks before any launch with every buffer untouched by a refused
 * call, nothing allocated, no synchronisation, CUDA-graph capture allowed, programmatic
 * dependent launch (every kernel here waits for the kernel before it before it
 * reads or writes any tensor). 16-bit tensors and E4M3 rows start and step on
 * 16-byte boundaries; positions, slots, tables, scales and fp32 tensors on their own
 * size. No two elements of one strided tensor may share an address.
 * Outputs may not overlap inputs or each other except where stated. Every result
 * is the same on every run: no float atomics. (The order of
 * paged_attention's sums follows the lengths, the call's sizes and the count of
 * multiprocessors, which sgq_set_sm_budget replaces; so may its last bit.)
 * Values that are not finite in a row give non-finite or unspecified results in what
 * is computed from that row, and in nothing else: not where the row is masked.
 * Every wait inside paged_attention is limited to some seconds, as those of
 * sgq_group.h's products are: sgq_wait_timeouts counts them too.
 */
#ifndef SGQ_CACHE_H
#define SGQ_CACHE_H

#include "sgq_group.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SGQ_MAX_HEAD 256          /* widest head, D */
#define SGQ_MAX_HEADS 1024        /* heads of one tensor */
#define SGQ_MAX_PAGE 65536        /* tokens of one page */

#define SGQ_F_ROPE_INTERLEAVED (1u << 6) /* pairs are columns (2i, 2i + 1), not (i, i + R/2) */
#define SGQ_F_ROPE_INVERSE     (1u << 7) /* rope: turned the other way, the gradient of the rotation */

/* Heads of T tokens: value i of head h of token t is element t * token_stride +
 * h * head_stride + i. Strides in elements, multiples of 8. */
typedef struct sgq_heads {
    void* p;
    int64_t heads;
    int64_t token_stride, head_stride;
} sgq_heads_t;

/* A paged cache (see above): pages 1 .. SGQ_MAX_ROWS, page_size 1 .. SGQ_MAX_PAGE,
 * heads 1 .. SGQ_MAX_HEADS. Strides in elements of the format's type, of k and v
 * alike: multiples of 16 bytes, below 2^40 bytes. k and v may lie between one
 * another (the halves of each page). k_scale and v_scale are NULL with SGQ_FMT_16BIT. */
typedef struct sgq_kv_cache {
    int64_t pages, page_size, heads, D;
    int64_t page_stride, head_stride, token_stride;
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
} sgq_kv_cache_t;

/* Rotary positions. Pair i of the first R columns of a head is turned by
 * positions[t] * freqs[i] / 2^64 of a full turn and multiplied by factor:
 *
 *   y_a = factor * (x_a cos - x_b sin),  y_b = factor * (x_a sin + x_b cos)
 *
 * Columns from R on are passed on as they are. A frequency in 2^-64 of a turn (freq / (2 pi) * 2^64,
 * an unsigned 64-bit number in an int64) makes the product with a position exact modulo
 * a turn, at any distance; slower and stretched frequencies for long contexts, and the
 * factor that goes with some, are the caller's choice. */
typedef struct sgq_rope {
    int64_t R;                 /* a multiple of 16, at most D */
    const int64_t* freqs;      /* [R / 2], read */
    const void* positions;     /* [T], read: int32 or int64, any sign */
    int position_bytes;        /* 4 or 8 */
    float factor;              /* finite */
} sgq_rope_t;

/*
 * Rotary positions on heads. Computed in fp32 (the angles in 64-bit integers, each
 * rounded once to fp32), rounded once.
 *
 * Arguments:
 *   flags         SGQ_F_FP16, SGQ_F_ROPE_INTERLEAVED, SGQ_F_ROPE_INVERSE
 *   T             tokens, at most SGQ_MAX_ROWS
 *   D             width of a head, a multiple of 8, at most SGQ_MAX_HEAD
 *   rope          see above
 *   x             [T, heads, D], read; heads at most SGQ_MAX_HEADS
 *   out           [T, heads, D], written; may be x (the same address and strides).
 *                 The rows of x and out may lie in the same tensor, each token's
 *                 beside the other's
 *
 * With SGQ_F_ROPE_INVERSE the angles are negated: dx = rope(dy) is then the
 * gradient of y = rope(x) with the same factor.
 */
int rope(uint32_t flags, int64_t T, int64_t D, const sgq_rope_t* rope, const sgq_heads_t* x, const sgq_heads_t* out,
         sgq_stream_t stream);

/*
 * New rows into the cache, one launch: for token t with slots[t] in [0, pages * page_size),
 *
 *   k row at slots[t] = fmt(R(positions[t]) k[t])         (R: rope's rotation; the identity with rope NULL)
 *   v row at slots[t] = fmt(v[t])
 *   q_out[t] = R(positions[t]) q[t]                       (every t, where q is given)
 *
 * k is quantised from its fp32 rotation (one rounding). A token whose slot is
 * outside the cache (-1: padding, another rank's) is not written. The slots of
 * one call have to be distinct: where two tokens name one slot, its rows hold
 * an unspecified mixture of theirs. Rows at other slots stay as they are.
 *
 * Arguments:
 *   fmt           SGQ_FMT_16BIT or SGQ_FMT_FP8_PER_TOKEN
 *   flags         SGQ_F_FP16, SGQ_F_ROPE_INTERLEAVED (with rope only)
 *   T             tokens, at most SGQ_MAX_ROWS
 *   cache         written; D a multiple of 8 (16 with FP8), at most SGQ_MAX_HEAD
 *   rope          or NULL
 *   q, q_out      [T, q->heads, D], read and written, or both NULL (they need
 *                 rope); q_out may be q as in rope
 *   k, v          [T, cache->heads, D], read
 *   slots         [T] int32 or int64, read
 *   slot_bytes    4 or 8
 */
int cache_write(int fmt, uint32_t flags, int64_t T, const sgq_kv_cache_t* cache, const sgq_rope_t* rope,
                const sgq_heads_t* q, const sgq_heads_t* q_out, const sgq_heads_t* k, const sgq_heads_t* v,
                const void* slots, int slot_bytes, sgq_stream_t stream);

/*
 * Rows of the cache as 16-bit values, code times scale rounded once: k_out[s] and
 * v_out[s] are the rows at slots[s], zeros where slots[s] is outside the cache.
 * A slot may be named many times.
 *
 * Arguments:
 *   fmt, cache    as in cache_write; read
 *   flags         SGQ_F_FP16
 *   S             rows, at most SGQ_MAX_ROWS
 *   slots         [S] int32 or int64, read
 *   k_out, v_out  [S, heads, D], written, contiguous; either may be NULL
 */
int cache_read(int fmt, uint32_t flags, int64_t S, const sgq_kv_cache_t* cache, const void* slots, int slot_bytes,
               void* k_out, void* v_out, sgq_stream_t stream);

/*
 * Attention of one new token a sequence over its pages, one launch where the table is
 * short and two else. For sequence b, its
 * length n = lengths[b] held to [0, width * page_size], and head h of q with
 * j = h / (Hq / heads) the head of the cache that it reads:
 *
 *   token t of b is at place t % page_size of page pages[b][t / page_size]
 *   x_t   = scale * (q[b][h] . k row of t)      for max(0, n - window) <= t < n (all t < n with window 0)
 *   p_t   = exp(x_t) / (sum_t exp(x_t) + exp(sinks[h]))        (without sinks: no last term)
 *   out[b][h] = sum_t p_t * (v row of t)
 *   lse[b][h] = log(sum_t exp(x_t) + exp(sinks[h]))
 *
 * n counts the new token itself where its row has been written. Tokens whose
 * page is outside [0, pages) are masked as those outside the window are: what masked
 * rows hold has no influence, and no page outside is read. Where nothing is left out[b] is zeros and lse the sink, or -infinity.
 *
 * Products in 16 bits by 16 bits, exact; sums, the softmax and its statistics in
 * fp32, exp2 to 2^-22 of its value and 0 below 2^-126: a token 87 nats under the largest,
 * or under the sink, counts as nothing, whatever its row's scale. FP8 codes enter as they are
 * and the rows' scales in fp32. The probabilities enter their product with v in two
 * 16-bit parts, or in 11 bits (FP8 cache beside bf16). Beside an FP8 or fp16 cache these
 * are fp16: a probability (with FP8, times its row's scale) is kept to 2^-30 of the largest
 * that the same warp has met, however small it is itself; the sum
 * counts it in fp32. q beside an FP8 cache enters as 11 bits and an exponent a head, so that
 * a bf16 value under 2^-17 of the head's largest loses its last bits. A row's scale
 * in v_scale has to be 0 or positive and at most 2^100; the sum counts rows alike,
 * however far apart their scales are.
 *
 * Arguments:
 *   fmt, cache    as in cache_write; read
 *   flags         SGQ_F_FP16
 *   B             sequences, at most SGQ_MAX_SEQUENCES
 *   q             [B, Hq, D], read; Hq = q->heads a multiple of cache->heads
 *   pages         [B, width] int32, read
 *   width         pages a sequence, >= 0; width * page_size < 2^31, and B * Hq *
 *                 (width * page_size / 64 + 3) < 2^31
 *   lengths       [B] int32, read
 *   scale         finite
 *   window        >= 0; 0 for none, as is any beyond the longest sequence
 *   sinks         [Hq] fp32, read, or NULL; -infinity is no sink
 *   out           [B, Hq, D], written, contiguous
 *   lse           [B, Hq] fp32, written, or NULL
 *   workspace     sgq_attention_workspace_bytes(...) bytes, written (16-byte
 *                 aligned; may be NULL where that is 0); calls that may run at
 *                 the same time (other streams, graphs) need workspaces of their own
 */
#define SGQ_MAX_SEQUENCES 65536
int paged_attention(int fmt, uint32_t flags, int64_t B, const sgq_kv_cache_t* cache, const sgq_heads_t* q,
                    const int32_t* pages, int64_t width, const int32_t* lengths, float scale, int64_t window,
                    const float* sinks, void* out, float* lse, void* workspace, sgq_stream_t stream);

/* Bytes of paged_attention's workspace; 0 where it needs none (one launch), or an argument is outside its range. */
int64_t sgq_attention_workspace_bytes(int fmt, int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t width,
                                      int64_t page_size, int64_t window);

#ifdef __cplusplus
}
#endif

#endif /* SGQ_CACHE_H */
