// Helpers shared by the kernels of the expert FFNs' gradient.
#pragma once

#include "grad.h"

// Matrix of group g: routed experts stacked, the shared expert apart.
template <typename T>
__device__ __forceinline__ T *of_group(void *routed, void *shared, int g,
                                       int E, size_t per) {
    return g < E ? (routed ? (T *)routed + g * per : nullptr) : (T *)shared;
}
template <typename T>
__device__ __forceinline__ const T *of_group(const void *routed,
                                             const void *shared, int g, int E,
                                             size_t per) {
    return g < E ? (routed ? (const T *)routed + g * per : nullptr)
                 : (const T *)shared;
}

// Rows of group g: [start, start + rows).  By scalar loads (the kernels of a
// gradient only read the offsets), which do not wait behind stores in flight.
__device__ __forceinline__ void group_rows(const FfnGradParams &p, int g,
                                           int &start, int &rows) {
    if (g < p.E) {
        typedef const __attribute__((address_space(4))) int *cptr;
        const cptr offsets = (cptr)(uint64_t)p.offsets;
        start = offsets[g];
        rows = offsets[g + 1] - start;
    } else {
        start = 0;
        rows = p.T;
    }
}

// Row tiles of a grid: at most ceil(rows / bm) plus one per group.
inline long long ffn_row_tiles(const FfnGradParams &p, int bm) {
    return (p.rows + bm - 1) / bm + p.E + p.n_shared;
}

// The bf16 layer's products on the matrix cores (ffn_grad_mfma.hip).
hipError_t launch_act_grad_mfma(const FfnGradParams &p, hipStream_t s);
hipError_t launch_row_grad_mfma(const FfnGradParams &p, hipStream_t s);
hipError_t launch_weight_grad_mfma(const FfnGradParams &p, hipStream_t s);
// Whether the products take the small tiles: routed groups of few rows each,
// or a narrow layer.
bool mfma_few_rows(long long routed, int E, int d, int d_ff);
int mfma_dw_tiles(int d_ff, int act, bool few);
int mfma_splits(long long routed, int E, int shared_rows, int N, int K);
