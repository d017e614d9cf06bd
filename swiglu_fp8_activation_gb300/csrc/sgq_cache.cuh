// sgq_cache.cuh -- arguments and host-side launchers of the paged cache's
// kernels (rope, cache_write, cache_read, paged_attention).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sgq_group.cuh"

namespace sgq {

constexpr int kMaxHead = 256;
constexpr int kMaxHeads = 1024;
constexpr int kMaxPage = 65536;

// n / d for 0 <= n < 2^31 by one multiplication: with 2^(s-1) < d <= 2^s and
// m = floor(2^(31+s) / d) + 1, n m / 2^(31+s) lies above n / d by less than 1 / d.
struct Div {
    uint32_t m;
    int s;
    uint32_t d;
};

inline Div make_div(uint32_t d) {
    int s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    return {(uint32_t)((uint64_t(1) << (31 + s)) / d + 1), 31 + s, d};
}

__device__ __forceinline__ uint32_t quotient(uint32_t n, const Div& d) { return (uint32_t)(((uint64_t)n * d.m) >> d.s); }

// The page of a slot, and its place in it.
__device__ __forceinline__ int64_t page_of_slot(int64_t slot, const Div& d, int& place) {
    const int64_t page = (uint64_t)slot >> 31 ? slot / d.d : (int64_t)quotient((uint32_t)slot, d);
    place = (int)(slot - page * d.d);
    return page;
}

__device__ __forceinline__ int64_t load_index(const void* p, int wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(p)[i] : (int64_t) static_cast<const int32_t*>(p)[i];
}

struct Heads {
    uint16_t* p;
    int64_t ts, hs;      // strides of tokens and heads, in elements
    int n;
};

struct CacheArgs {
    uint8_t* k;
    uint8_t* v;
    float* ks;           // null with 16-bit rows
    float* vs;
    int64_t pages;
    int64_t ps, hs, ts;  // strides of pages, heads and tokens, in bytes
    int heads;
    int D;
    Div page;            // tokens a page
};

struct RopeArgs {
    const uint64_t* freqs;
    const void* positions;
    float factor;
    int half;            // pairs, R / 2; 0 for no rotation
    int wide;            // 64-bit positions
    int inverse;
};

struct WriteArgs {
    RopeArgs rope;
    Heads q, qo, k, v;   // q.n heads are rotated, k.n rotated and written, v.n (equal to k.n) written
    CacheArgs c;
    const void* slots;
    int wide;            // 64-bit slots
    int64_t T;
    int per;             // threads a token
    int ahead;           // whether q's rows are asked for before the angles
    int D;
};

struct ReadArgs {
    CacheArgs c;
    const void* slots;
    int wide;
    int64_t S;
    int tpc;             // tokens a CTA
    Div pieces, row;     // pieces of a token and of a row
    uint16_t* k;         // either may be null
    uint16_t* v;
};

struct AttendArgs {
    CUtensorMap km, vm;  // of the cache's rows
    CacheArgs c;
    Heads q;
    const int32_t* table;
    const int32_t* lengths;
    const float* sinks;  // or null
    uint16_t* out;
    float* lse;          // or null
    void* ws;
    int64_t width;       // pages a sequence
    float scale;
    int window;          // 0 for none
    int B;
    int group;           // heads of q a head of the cache
    int limit;           // width * page size: the longest sequence
    int chunks;          // column chunks a head of the cache
    int items;           // heads * chunks a sequence
    int joined;          // how a second launch finds what several CTAs have computed
    int split;           // CTAs of a cluster, where each takes one item; 0 for shares
    int tiles;           // of the longest item
    int DP;              // attend_padded's width
    int stages;          // tiles copied ahead
    int boxes;           // tokens of the copy engine's boxes; 0 where lanes copy
};

// Pairs of times in the comments on paged_attention's rules, here and in sgq_attend.cuh, are of the two sides of a rule when it was made, the rest
// alike; either side may have become faster since.

// Most CTAs that take shares of one paged_attention, for which its workspace has room.
constexpr int kAttendCtas = 512;

// Columns (heads of q) a CTA takes at once.
constexpr int attend_columns(int group, int DP) { return group <= 8 ? 8 : group <= 16 || DP > 128 ? 16 : 32; }
constexpr int attend_padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// Tokens of a tile: of E4M3 rows twice as many, up to heads of 128 (8 sequences up to 131072: 281 us, with 64 tokens 369).
__host__ __device__ constexpr int attend_tokens(bool fp8, int DP) { return fp8 && DP <= 128 ? 128 : 64; }
// Tiles of the longest item; a window may begin anywhere in its first tile.
constexpr int64_t attend_tiles(bool fp8, int DP, int64_t limit, int64_t window) {
    const int tokens = attend_tokens(fp8, DP);
    if (window > 0 && window < limit && limit > window + tokens - 1) limit = window + tokens - 1;    // (a window may be any number)
    return limit <= tokens ? 1 : (limit + tokens - 1) / tokens;
}
// What an item's end costs a CTA that takes shares, in tiles. (256 sequences up to 4000, 2 heads, E4M3: 59.5 us with 0, 56.1 with 2, 57.9 with 5.)
constexpr int kAttendEnd = 2;
// CTAs of paged_attention on a multiprocessor at most. Three CTAs that each take a short item hide one another's beginnings (64 sequences up to
// 4096, bf16: 82 us, with two 89); CTAs that take long shares are two, but for narrow rows (8 sequences of
// 65536, D 64, bf16: 152 us with two, 140 with three; 4 of 32768, E4M3: 50 and 33; 8 up to 131072, D 128, E4M3: 281 and 298).
__host__ __device__ constexpr int attend_resident(bool fp8, int DP, int cols, bool direct) {
    return DP == 256 ? (fp8 && cols == 8 ? 2 : 1) : cols == 32 ? 1 : cols == 16 ? 2 : direct || DP == 64 ? 3 : 2;
}
// CTAs in clusters of `split` that surely run at once, n a multiprocessor: clusters do not fill the device's processor groups. (At most 120, 288
// and 408 in clusters of 8 with n of 1, 2 and 3, and 144, 296 and 440 in clusters of 4, by the occupancy calculator; this gives 120, 272, 408 and 136, 288, 432.)
constexpr int64_t attend_room(int64_t sms, int n, int split) { return n * sms - (split == 1 ? 0 : (n > 2 ? 6 : 4) * split); }
// CTAs of a cluster, where each cluster takes one item; 0 where CTAs take shares of all items' tiles. A cluster needs no workspace
// and no second launch; but it is 8 CTAs at most, and where long items are to be taken, or many sequences are empty, some multiprocessors
// end long before others. The host knows the table's width alone: up to 8 tiles a CTA, or 1024 tokens where all CTAs run
// at once. (Times in a graph, clusters and shares: 32 of 1024, 8 heads, bf16: 24.6 and 28.2 us; 24 of 2000, E4M3: 20.6 and 24.9; 1 of 4000, bf16: 11.1
// and 9.4, but 5 us of the host's time less; 33 up to 5001, 3 heads, E4M3, 10 tiles a CTA: 24.1 and 19.7; 128 up to 8000, bf16, 16 tiles in 9 rounds: 318 and 283.)
// The plan is for the 152 multiprocessors of the device, whatever sgq_set_sm_budget says: the workspace's size goes by it, and has to hold for
// a call with another budget. The budget sets the CTAs that take shares.
constexpr int attend_split(bool fp8, int DP, int64_t items, int64_t tiles, int cols) {
    const int n = attend_resident(fp8, DP, cols, true);
    int split = 1;
    while (split < 8 && split * 2 <= tiles && (items * split * 2 <= attend_room(152, n, split * 2) || tiles > split * 16)) split *= 2;
    const int64_t each = (tiles + split - 1) / split, ctas = items * split;
    const bool once = cols == 8 && ctas >= 152 && ctas <= attend_room(152, n, split);
    return (each <= 8 || (once && each * attend_tokens(fp8, DP) <= 1024)) && ctas <= 0x7FFFFFFF ? split : 0;
}
// Floats of what one CTA leaves of an unfinished item: the sums, then the maxima and the totals.
__host__ __device__ constexpr int attend_part(int cols, int DP) { return cols * (DP + 2); }

// An item of paged_attention that a CTA has begun and not ended: that CTA, and the last that
// has some of it; first is -1 where there is none. The workspace begins with these entries.
struct Shared {
    int b, j, first, last;
};

__host__ __device__ constexpr int attend_header_bytes() { return kAttendCtas * (int)sizeof(Shared); }

cudaError_t launch_cache_write(int fmt, int dt, bool interleaved, const Device& dev, const WriteArgs& a, cudaStream_t stream);
cudaError_t launch_cache_read(int fmt, int dt, const Device& dev, const ReadArgs& a, cudaStream_t stream);
// Boxes of `tokens` tokens by `block` bytes of the rows of k or v, in the order of that block's swizzle, zeros outside a row. False when the
// driver refuses the strides.
bool encode_cache(CUtensorMap* m, const CacheArgs& c, const void* rows, int tokens, int block, int elem);

cudaError_t launch_attend(int fmt, int dt, const Device& dev, const AttendArgs& a, cudaStream_t stream);
// CTAs of paged_attention on the current device in which a wait ran out of time (waits for the device).
cudaError_t attend_gave_up(uint32_t* n);

}  // namespace sgq
