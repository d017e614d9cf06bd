// sgq_host.h -- what the C entry points' host checks share: alignment and
// overlap of argument tensors, sizes, the current device.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "sgq.h"
#include "sgq_launch.h"

namespace sgq {

// Largest element count of one tensor: its byte sizes (at most 4 bytes an
// element) stay far inside size_t and the kernels' 64-bit offsets.
constexpr int64_t kMaxElements = int64_t(1) << 56;

inline bool aligned(const void* p, uintptr_t a) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Half-open byte ranges [a, a+na) and [b, b+nb) intersect (null or empty never does).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

struct Device {
    int id;
    int sms;
};

Device current_device();

// Dynamic shared memory one CTA may use (227 KB on sm_100-class parts).
constexpr int kMaxDynamicSmem = 227 * 1024;

struct Span {
    const void* p;
    size_t n;
};

// True when any two of the spans intersect.
inline bool any_overlap(const Span* s, int k) {
    for (int i = 0; i < k; ++i)
        for (int j = i + 1; j < k; ++j)
            if (overlap(s[i].p, s[i].n, s[j].p, s[j].n)) return true;
    return false;
}

inline int launched(cudaError_t e) {
    if (e == cudaSuccess) return SGQ_OK;
    note_launch_error(e);
    return SGQ_ERR_LAUNCH;
}

}  // namespace sgq
