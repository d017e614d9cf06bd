// sgq_cache_api.cu -- the C ABI declared in include/sgq_cache.h: host-side
// argument checks, then the operation's launches.
#include <math.h>

#include "sgq_cache.cuh"

#include "sgq_cache.h"

using namespace sgq;

namespace {

constexpr int64_t kMaxRows = SGQ_MAX_ROWS;
constexpr int64_t kMaxStride = int64_t(1) << 40;     // bytes, of a tensor map

bool bad_count(int64_t v) { return v < 0 || v > kMaxRows; }

struct Dim {
    int64_t size, stride;
};

// Bytes from the first to behind the last element of a strided tensor of `elem`-byte
// values whose innermost `width` lie side by side; false when a stride is
// negative or the extent is out of range. Strides in elements; an axis of one has none.
bool extent(const Dim* d, int n, int64_t width, int64_t elem, size_t* bytes) {
    int64_t e = width;
    for (int i = 0; i < n; ++i) {
        if (d[i].size < 1) {
            *bytes = 0;
            return true;
        }
        if (d[i].size == 1) continue;
        if (d[i].stride < 0 || d[i].stride > kMaxElements / d[i].size) return false;
        e += d[i].stride * (d[i].size - 1);
        if (e > kMaxElements) return false;
    }
    *bytes = (size_t)(e * elem);
    return true;
}

// Whether no two elements share an address: each axis, from the smallest stride on, steps over all within.
bool distinct(Dim* d, int n, int64_t width) {
    for (int i = 1; i < n; ++i)
        for (int j = i; j > 0 && d[j].stride < d[j - 1].stride; --j) {
            const Dim t = d[j];
            d[j] = d[j - 1];
            d[j - 1] = t;
        }
    int64_t e = width;
    for (int i = 0; i < n; ++i) {
        if (d[i].size <= 1) continue;
        if (d[i].stride < e) return false;
        e += d[i].stride * (d[i].size - 1);
    }
    return true;
}

// Heads of T tokens, checked (status) and taken over with the strides of axes of one set to 0.
int take_heads(const sgq_heads_t* h, int64_t T, int64_t D, bool written, Heads* to, size_t* bytes) {
    if (!h || h->heads < 1) return SGQ_ERR_INVALID_ARG;
    if (h->heads > SGQ_MAX_HEADS) return SGQ_ERR_UNSUPPORTED;
    Dim d[2] = {{T, h->token_stride}, {h->heads, h->head_stride}};
    if (!extent(d, 2, D, 2, bytes)) return SGQ_ERR_INVALID_ARG;
    if (!h->p) return SGQ_ERR_INVALID_ARG;
    for (const Dim& x : d)
        if (x.size > 1 && x.stride % 8 != 0) return SGQ_ERR_MISALIGNED;
    if (!aligned(h->p, 16)) return SGQ_ERR_MISALIGNED;
    to->p = static_cast<uint16_t*>(h->p);
    to->ts = T > 1 ? h->token_stride : 0;
    to->hs = h->heads > 1 ? h->head_stride : 0;
    to->n = (int)h->heads;
    if (written && !distinct(d, 2, D)) return SGQ_ERR_INVALID_ARG;
    return SGQ_OK;
}

// Whether the written heads `w` meet the heads `r`: exactly where both have the same stride of tokens and
// a token's heads within it (rows of one projection), else by their spans.
bool meet(const Heads& w, size_t wn, const Heads& r, size_t rn, int64_t D) {
    if (!overlap(w.p, wn, r.p, rn)) return false;
    const int64_t we = ((int64_t)(w.n - 1) * w.hs + D) * 2, re = ((int64_t)(r.n - 1) * r.hs + D) * 2, s = w.ts * 2;
    if (w.ts != r.ts || we > s || re > s) return true;
    int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(r.p) - reinterpret_cast<uintptr_t>(w.p)) % s;
    if (d < 0) d += s;
    return d < we || d + re > s;
}

bool same(const Heads& a, const Heads& b) { return a.p == b.p && a.ts == b.ts && a.hs == b.hs && a.n == b.n; }

struct CacheSpans {
    Span s[4];
};

int take_cache(int fmt, const sgq_kv_cache_t* c, CacheArgs* to, CacheSpans* spans) {
    if (fmt != SGQ_FMT_16BIT && fmt != SGQ_FMT_FP8_PER_TOKEN) return SGQ_ERR_INVALID_ARG;
    if (!c || c->pages < 1 || bad_count(c->pages) || c->page_size < 1 || c->heads < 1 || c->D < 1) return SGQ_ERR_INVALID_ARG;
    const bool fp8 = fmt == SGQ_FMT_FP8_PER_TOKEN;
    const int64_t unit = fp8 ? 16 : 8, elem = fp8 ? 1 : 2;
    if (c->page_size > SGQ_MAX_PAGE || c->heads > SGQ_MAX_HEADS || c->D > SGQ_MAX_HEAD || c->D % unit != 0) return SGQ_ERR_UNSUPPORTED;
    if (fp8 ? !c->k_scale || !c->v_scale : c->k_scale || c->v_scale) return SGQ_ERR_INVALID_ARG;
    if (!c->k || !c->v) return SGQ_ERR_INVALID_ARG;
    const intptr_t apart = reinterpret_cast<intptr_t>(c->v) - reinterpret_cast<intptr_t>(c->k);
    Dim d[4] = {{c->pages, c->page_stride}, {c->heads, c->head_stride}, {c->page_size, c->token_stride}, {2, 0}};
    size_t bytes = 0;
    if (!extent(d, 3, c->D, elem, &bytes)) return SGQ_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if (d[i].size > 1 && d[i].stride * elem % 16 != 0) return SGQ_ERR_MISALIGNED;
    for (int i = 0; i < 3; ++i)
        if (d[i].size > 1 && d[i].stride * elem >= kMaxStride) return SGQ_ERR_UNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return SGQ_ERR_MISALIGNED;
    to->k = static_cast<uint8_t*>(c->k);
    to->v = static_cast<uint8_t*>(c->v);
    to->ks = c->k_scale;
    to->vs = c->v_scale;
    to->pages = c->pages;
    to->ps = c->pages > 1 ? c->page_stride * elem : 0;
    to->hs = c->heads > 1 ? c->head_stride * elem : 0;
    to->ts = c->page_size > 1 ? c->token_stride * elem : 0;
    to->heads = (int)c->heads;
    to->D = (int)c->D;
    to->page = make_div((uint32_t)c->page_size);
    // k and v may lie between one another (two halves of each page): an axis of two
    d[3].stride = (apart < 0 ? -apart : apart) / elem;
    if (!distinct(d, 4, c->D)) return SGQ_ERR_INVALID_ARG;
    const size_t rows = fp8 ? (size_t)(c->pages * c->heads * c->page_size) * 4 : 0;
    *spans = {{{c->k, bytes}, {c->v, bytes}, {c->k_scale, rows}, {c->v_scale, rows}}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (j > 1 && overlap(spans->s[i].p, spans->s[i].n, spans->s[j].p, spans->s[j].n)) return SGQ_ERR_INVALID_ARG;
    return SGQ_OK;
}

int take_rope(const sgq_rope_t* r, int64_t T, int64_t D, uint32_t flags, RopeArgs* to, Span* spans) {
    if (r->R < 1 || (r->position_bytes != 4 && r->position_bytes != 8) || !isfinite(r->factor)) return SGQ_ERR_INVALID_ARG;
    if (r->R % 16 != 0 || r->R > D) return SGQ_ERR_UNSUPPORTED;
    if (!r->freqs || !r->positions) return SGQ_ERR_INVALID_ARG;
    if (!aligned(r->freqs, 8) || !aligned(r->positions, (uintptr_t)r->position_bytes)) return SGQ_ERR_MISALIGNED;
    to->freqs = reinterpret_cast<const uint64_t*>(r->freqs);
    to->positions = r->positions;
    to->factor = r->factor;
    to->half = (int)(r->R / 2);
    to->wide = r->position_bytes == 8;
    to->inverse = (flags & SGQ_F_ROPE_INVERSE) != 0;
    spans[0] = {r->freqs, (size_t)(r->R / 2) * 8};
    spans[1] = {r->positions, (size_t)T * r->position_bytes};
    return SGQ_OK;
}

int dt_of(uint32_t flags) { return (flags & SGQ_F_FP16) ? DT_F16 : DT_BF16; }

int fmt_of(int fmt) { return fmt == SGQ_FMT_FP8_PER_TOKEN ? (int)FMT_PT : FMT_16BIT; }

// How paged_attention's items are cut: false when a size is out of range.
struct AttendPlan {
    int DP, cols, chunks, split;
    int64_t items, tiles;            // of a sequence; of the longest item
};

bool plan_attend(int fmt, int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t width, int64_t page_size, int64_t window, AttendPlan* p) {
    if ((fmt != SGQ_FMT_16BIT && fmt != SGQ_FMT_FP8_PER_TOKEN) || B < 1 || B > SGQ_MAX_SEQUENCES || heads < 1 || heads > SGQ_MAX_HEADS || Hq < heads ||
        Hq > SGQ_MAX_HEADS || Hq % heads != 0 || D < 1 || D % (fmt == SGQ_FMT_FP8_PER_TOKEN ? 16 : 8) != 0 || D > SGQ_MAX_HEAD || width < 0 || page_size < 1 || page_size > SGQ_MAX_PAGE || width > 0x7FFFFFFF / page_size || window < 0)
        return false;
    const int64_t group = Hq / heads;
    const bool fp8 = fmt == SGQ_FMT_FP8_PER_TOKEN;
    p->DP = attend_padded((int)D);
    p->cols = attend_columns((int)group, p->DP);
    p->chunks = (int)((group + p->cols - 1) / p->cols);
    p->items = heads * p->chunks;
    p->tiles = attend_tiles(fp8, p->DP, width * page_size, window);
    p->split = attend_split(fp8, p->DP, B * p->items, p->tiles, p->cols);
    return B * p->items * (p->tiles + kAttendEnd) <= 0x7FFFFFFF;         // counted in 32 bits
}

}  // namespace

extern "C" {

int rope(uint32_t flags, int64_t T, int64_t D, const sgq_rope_t* rope, const sgq_heads_t* x, const sgq_heads_t* out,
         sgq_stream_t stream) {
    if (flags & ~(SGQ_F_FP16 | SGQ_F_ROPE_INTERLEAVED | SGQ_F_ROPE_INVERSE)) return SGQ_ERR_INVALID_ARG;
    if (bad_count(T) || D < 1 || !rope || !x || !out) return SGQ_ERR_INVALID_ARG;
    if (D > SGQ_MAX_HEAD || D % 8 != 0) return SGQ_ERR_UNSUPPORTED;
    if (T == 0) return SGQ_OK;
    if (x->heads != out->heads) return SGQ_ERR_INVALID_ARG;
    WriteArgs a = {};
    Span r[2];
    size_t xn = 0, on = 0;
    int st = take_rope(rope, T, D, flags, &a.rope, r);
    if (st == SGQ_OK) st = take_heads(x, T, D, false, &a.q, &xn);
    if (st == SGQ_OK) st = take_heads(out, T, D, true, &a.qo, &on);
    if (st != SGQ_OK) return st;
    if (!same(a.q, a.qo) && meet(a.qo, on, a.q, xn, D)) return SGQ_ERR_INVALID_ARG;
    for (const Span& s : r)
        if (overlap(s.p, s.n, a.qo.p, on)) return SGQ_ERR_INVALID_ARG;
    a.c.page = make_div(1);
    a.T = T;
    a.D = (int)D;
    return launched(launch_cache_write(FMT_16BIT, dt_of(flags), (flags & SGQ_F_ROPE_INTERLEAVED) != 0, current_device(), a,
                                       static_cast<cudaStream_t>(stream)));
}

int cache_write(int fmt, uint32_t flags, int64_t T, const sgq_kv_cache_t* cache, const sgq_rope_t* rope,
                const sgq_heads_t* q, const sgq_heads_t* q_out, const sgq_heads_t* k, const sgq_heads_t* v,
                const void* slots, int slot_bytes, sgq_stream_t stream) {
    if (flags & ~(SGQ_F_FP16 | SGQ_F_ROPE_INTERLEAVED)) return SGQ_ERR_INVALID_ARG;
    if (bad_count(T) || !cache || (!rope && (flags & SGQ_F_ROPE_INTERLEAVED))) return SGQ_ERR_INVALID_ARG;
    if (!q != !q_out || (q && !rope) || (slot_bytes != 4 && slot_bytes != 8)) return SGQ_ERR_INVALID_ARG;
    WriteArgs a = {};
    CacheSpans written;
    int st = take_cache(fmt, cache, &a.c, &written);
    if (st != SGQ_OK) return st;
    if (T == 0) return SGQ_OK;
    const int64_t D = cache->D;
    Span in[5] = {};
    size_t qn = 0, on = 0, kn = 0, vn = 0;
    if (rope) st = take_rope(rope, T, D, flags, &a.rope, in);
    if (st == SGQ_OK && q) st = take_heads(q, T, D, false, &a.q, &qn);
    if (st == SGQ_OK && q) st = take_heads(q_out, T, D, true, &a.qo, &on);
    if (st == SGQ_OK) st = take_heads(k, T, D, false, &a.k, &kn);
    if (st == SGQ_OK) st = take_heads(v, T, D, false, &a.v, &vn);
    if (st != SGQ_OK) return st;
    if (k->heads != cache->heads || v->heads != cache->heads || (q && q->heads != q_out->heads) || !slots) return SGQ_ERR_INVALID_ARG;
    if (!aligned(slots, (uintptr_t)slot_bytes)) return SGQ_ERR_MISALIGNED;
    in[2] = {slots, (size_t)T * slot_bytes};
    in[3] = {a.k.p, kn};
    in[4] = {a.v.p, vn};
    for (const Span& w : written.s) {
        for (const Span& i : in)
            if (overlap(w.p, w.n, i.p, i.n)) return SGQ_ERR_INVALID_ARG;
        if (q && (overlap(w.p, w.n, a.q.p, qn) || overlap(w.p, w.n, a.qo.p, on))) return SGQ_ERR_INVALID_ARG;
    }
    if (q) {
        if (!same(a.q, a.qo) && meet(a.qo, on, a.q, qn, D)) return SGQ_ERR_INVALID_ARG;
        if (meet(a.qo, on, a.k, kn, D) || meet(a.qo, on, a.v, vn, D)) return SGQ_ERR_INVALID_ARG;
        for (int i = 0; i < 3; ++i)
            if (overlap(in[i].p, in[i].n, a.qo.p, on)) return SGQ_ERR_INVALID_ARG;
    }
    a.slots = slots;
    a.wide = slot_bytes == 8;
    a.T = T;
    a.D = (int)D;
    return launched(launch_cache_write(fmt_of(fmt), dt_of(flags), (flags & SGQ_F_ROPE_INTERLEAVED) != 0, current_device(), a,
                                       static_cast<cudaStream_t>(stream)));
}

int cache_read(int fmt, uint32_t flags, int64_t S, const sgq_kv_cache_t* cache, const void* slots, int slot_bytes,
               void* k_out, void* v_out, sgq_stream_t stream) {
    if ((flags & ~SGQ_F_FP16) || bad_count(S) || (slot_bytes != 4 && slot_bytes != 8)) return SGQ_ERR_INVALID_ARG;
    ReadArgs a = {};
    CacheSpans in;
    const int st = take_cache(fmt, cache, &a.c, &in);
    if (st != SGQ_OK) return st;
    if (S == 0) return SGQ_OK;
    if (!slots || (!k_out && !v_out)) return SGQ_ERR_INVALID_ARG;
    if (!aligned(slots, (uintptr_t)slot_bytes) || !aligned(k_out, 16) || !aligned(v_out, 16)) return SGQ_ERR_MISALIGNED;
    const size_t n = (size_t)(S * cache->heads * cache->D) * 2;
    const Span out[] = {{k_out, n}, {v_out, n}}, s = {slots, (size_t)S * slot_bytes};
    if (any_overlap(out, 2)) return SGQ_ERR_INVALID_ARG;
    for (const Span& o : out) {
        if (overlap(o.p, o.n, s.p, s.n)) return SGQ_ERR_INVALID_ARG;
        for (const Span& i : in.s)
            if (overlap(o.p, o.n, i.p, i.n)) return SGQ_ERR_INVALID_ARG;
    }
    a.slots = slots;
    a.wide = slot_bytes == 8;
    a.S = S;
    a.k = static_cast<uint16_t*>(k_out);
    a.v = static_cast<uint16_t*>(v_out);
    return launched(launch_cache_read(fmt_of(fmt), dt_of(flags), current_device(), a, static_cast<cudaStream_t>(stream)));
}

int64_t sgq_attention_workspace_bytes(int fmt, int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t width, int64_t page_size,
                                      int64_t window) {
    AttendPlan p;
    if (!plan_attend(fmt, B, Hq, heads, D, width, page_size, window, &p) || p.split > 0) return 0;
    const int64_t most = B * p.items * p.tiles, ctas = most < kAttendCtas ? most : kAttendCtas;
    return attend_header_bytes() + ctas * 2 * attend_part(p.cols, p.DP) * 4;
}

int paged_attention(int fmt, uint32_t flags, int64_t B, const sgq_kv_cache_t* cache, const sgq_heads_t* q,
                    const int32_t* pages, int64_t width, const int32_t* lengths, float scale, int64_t window,
                    const float* sinks, void* out, float* lse, void* workspace, sgq_stream_t stream) {
    if ((flags & ~SGQ_F_FP16) || B < 0 || width < 0 || window < 0 || !isfinite(scale) || !q) return SGQ_ERR_INVALID_ARG;
    AttendArgs a = {};
    CacheSpans in;
    int st = take_cache(fmt, cache, &a.c, &in);
    if (st != SGQ_OK) return st;
    if (B > SGQ_MAX_SEQUENCES || width > 0x7FFFFFFF / cache->page_size) return SGQ_ERR_UNSUPPORTED;
    if (B == 0) return SGQ_OK;
    size_t qn = 0;
    st = take_heads(q, B, cache->D, false, &a.q, &qn);
    if (st != SGQ_OK) return st;
    if (q->heads % cache->heads != 0) return SGQ_ERR_INVALID_ARG;
    AttendPlan p;
    if (!plan_attend(fmt, B, q->heads, cache->heads, cache->D, width, cache->page_size, window, &p)) return SGQ_ERR_UNSUPPORTED;
    const int64_t ws = sgq_attention_workspace_bytes(fmt, B, q->heads, cache->heads, cache->D, width, cache->page_size, window);
    if (!lengths || !out || (width > 0 && !pages) || (ws > 0 && !workspace)) return SGQ_ERR_INVALID_ARG;
    if (!aligned(pages, 4) || !aligned(lengths, 4) || !aligned(sinks, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
        return SGQ_ERR_MISALIGNED;
    const size_t rows = (size_t)(B * q->heads);
    const Span w[] = {{out, rows * (size_t)cache->D * 2}, {lse, rows * 4}, {workspace, (size_t)ws}};
    const Span r[] = {in.s[0], in.s[1], in.s[2], in.s[3], {q->p, qn}, {pages, (size_t)(B * width) * 4}, {lengths, (size_t)B * 4},
                      {sinks, (size_t)q->heads * 4}};
    if (any_overlap(w, 3)) return SGQ_ERR_INVALID_ARG;
    for (const Span& o : w)
        for (const Span& i : r)
            if (overlap(o.p, o.n, i.p, i.n)) return SGQ_ERR_INVALID_ARG;
    a.table = pages;
    a.lengths = lengths;
    a.sinks = sinks;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.ws = workspace;
    a.width = width;
    a.scale = scale;
    a.limit = (int)(width * cache->page_size);
    a.window = (int)(window > a.limit ? 0 : window);     // a window over all tokens is none
    a.B = (int)B;
    a.group = (int)(q->heads / cache->heads);
    a.chunks = p.chunks;
    a.items = (int)p.items;
    a.tiles = (int)p.tiles;
    a.split = p.split;
    a.DP = p.DP;
    return launched(launch_attend(fmt_of(fmt), dt_of(flags), current_device(), a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
