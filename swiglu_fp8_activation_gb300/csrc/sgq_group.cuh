// sgq_group.cuh -- arguments and host-side launchers of the ragged-group
// kernels (group_rows, grouped_gemm, combine_rows, lora_add), one translation
// unit per operation.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sgq_host.h"

namespace sgq {

constexpr int FMT_16BIT = 3;         // beside Fmt: 16-bit rows and weights
constexpr int kMaxGroups = 1024;
constexpr int kMaxRank = 128;

struct GroupRowsArgs {
    const void* ids;
    int32_t* offsets;
    int32_t* rows;
    int32_t* slots;      // or null
    uint32_t n;          // T * k ids
    uint32_t k;
    int groups;
    int wide;            // 64-bit ids
};

struct GroupGemmArgs {
    const void* x;
    const void* xs;
    const void* w;
    const void* ws;
    const int32_t* offsets;
    const int32_t* rows;  // or null
    uint16_t* out;
    int64_t x_rows;
    int S, groups, N, K;
};

struct CombineArgs {
    const uint16_t* y;
    const int32_t* slots;
    const float* weights;  // or null
    uint16_t* out;
    int64_t T;
    int64_t S;
    int k;
    int N;
    int nblk;              // column blocks a token
};

struct LoraArgs {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const float* scaling;  // or null
    const int32_t* offsets;
    const int32_t* rows;   // or null
    const int32_t* slots;  // null exactly when rows is
    uint16_t* y;
    void* v;               // workspace, S rows of lora_row_bytes(R); null with lora_few
    int64_t T;
    int S, groups, R, K, N;
};

// A byte tensor of `dims` (innermost first, rows of dims[0] bytes, a multiple
// of 16), box of 128 bytes by `box_rows` rows, 128-byte
// swizzle, zeros outside. False when the driver refuses it.
bool encode_rows(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, int box_rows);

// `tiles` pieces of 512 bytes, one below the other, box one piece, no swizzle.
bool encode_tiles512(CUtensorMap* m, const void* base, int64_t tiles);

// Bytes of a row of lora_add's workspace: R values of v, then the row's
// factor (fp16 rows), all fp32, and 12 bytes over.
__host__ __device__ constexpr int lora_row_bytes(int R) { return 4 * R + 16; }

// Whether lora_add runs its form for few slots an adapter (one launch, no
// workspace): slots an adapter (on average) x rank up to 128. K = N = 4096, this
// form and the tensor cores' in a graph: rank 16, 2 slots an adapter 8.0 and 21.8
// us, 8 slots 13.9 and 21.8, 16 slots 25.9 and 21.8; rank 64, 2 slots 20.6 and 25.9, 4 slots
// 28.9 and 25.9 (32 adapters, the same number of slots each).
// The host does not know how many adapters are in use, and where it is one or a few
// of many the slots are not few: up to 512 slots, and 8192 slots x rank, the worse
// of the two mistakes is the smaller one. 1024 adapters, one in use and all: rank 16,
// 256 slots 21.7 and 30.9 us, 40.6 and 94.4; 512 slots 41.6 and 30.9, 82.5 and 167; 1024
// slots 79.5 and 32.3, 147 and 244; 8192 slots 499 and 59.6, 545 and 384. Rank 64, 128 slots
// 41.1 and 34.0, 64.2 and 67.8; 256 slots 46.8 and 33.9, 112 and 125; 512 slots 87.2 and
// 34.0, 186 and 199.
constexpr bool lora_few(int64_t S, int64_t groups, int64_t R) {
    return S <= 512 && S * R <= (groups < 64 ? 128 * groups : 8192);
}

cudaError_t launch_group_rows(const Device& dev, const GroupRowsArgs& a, cudaStream_t stream);
cudaError_t launch_grouped_gemm(int fmt, int dt, const Device& dev, const GroupGemmArgs& a, cudaStream_t stream);
cudaError_t launch_combine(int dt, const Device& dev, const CombineArgs& a, cudaStream_t stream);
cudaError_t launch_lora(int dt, const Device& dev, const LoraArgs& a, cudaStream_t stream);

// Launches on the current device in which a wait ran out of time (waits for the device).
cudaError_t gemm_gave_up(uint32_t* n);
cudaError_t lora_gave_up(uint32_t* n);

// Launch k on `stream` with programmatic stream serialisation (as launch_pdl,
// for any grid), in clusters of `cluster` CTAs along x.
template <typename Args>
cudaError_t launch_grid(void (*k)(const Args), dim3 grid, int threads, int smem, int cluster, int device,
                        const Args& a, cudaStream_t stream) {
    if (smem > 40 * 1024) {
        const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(k), device, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

// The range of slots of group g, held inside [0, S] and ascending: what the
// kernels take for offsets[g], offsets[g + 1] whatever they hold.
__device__ __forceinline__ int held(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

}  // namespace sgq
