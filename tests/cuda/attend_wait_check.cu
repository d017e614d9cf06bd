// Test-only build of paged_attention whose waits are limited to milliseconds and in which one copy of one tile is never issued, or late, compiled by
// tests/test_gpu_attend_waits.py together with the library's entry points. Nothing else differs from the library's kernels.
#include <cuda_runtime.h>

namespace {

struct Copy {
    int mode;            // 0: all copies, 1: this one never, 2: this one after `cycles`
    int item, part, tile;
    long long cycles;
};
__device__ Copy chosen;

// Whether a tile's copies are issued; uniform in a warp.
__device__ bool issued(int item, int part, int tile) {
    const Copy c = chosen;
    if (c.mode == 0 || item != c.item || part != c.part || tile != c.tile) return true;
    if (c.mode == 1) return false;
    const long long start = clock64();
    while (clock64() - start < c.cycles) {
    }
    __syncwarp();
    return true;
}

__global__ void spin(long long cycles) {
    const long long start = clock64();
    while (clock64() - start < cycles) {
    }
}

}  // namespace

#define SGQ_ATTEND_COPIES(item, part, tile) issued(item, part, tile)
#define SGQ_ATTEND_WAIT (1LL << 25)
// names of its own for the kernels, beside the library's in one process
#define attend attend_with_short_waits
#include "sgq_attend.cuh"

namespace sgq {

cudaError_t launch_attend(int fmt, int dt, const Device& dev, const AttendArgs& a, cudaStream_t stream) {
    if (dt != DT_BF16 || a.DP != 64) return cudaErrorInvalidValue;
    if (fmt == FMT_PT) return a.group <= 8 ? attend::launch<attend::FP8_BF16, 64, 1, 1>(dev, a, stream) : cudaErrorInvalidValue;
    return a.group <= 8 ? attend::launch<attend::BF16, 64, 1, 1>(dev, a, stream) : attend::launch<attend::BF16, 64, 2, 2>(dev, a, stream);
}

}  // namespace sgq

extern "C" long long check_limit() { return SGQ_ATTEND_WAIT; }

extern "C" int check_choose(int mode, int item, int part, int tile, long long cycles) {
    const Copy c = {mode, item, part, tile, cycles};
    return (int)cudaMemcpyToSymbol(chosen, &c, sizeof c);
}

// A kernel that takes so many cycles.
extern "C" int check_spin(long long cycles, cudaStream_t stream) {
    spin<<<1, 1, 0, stream>>>(cycles);
    return (int)cudaGetLastError();
}

extern "C" int check_gave_up(uint32_t* n) { return (int)sgq::attend::read_gave_up(n); }
