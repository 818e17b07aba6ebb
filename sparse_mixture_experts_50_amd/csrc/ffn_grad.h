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

// Rows of group g: [start, start + rows).
__device__ __forceinline__ void group_rows(const FfnGradParams &p, int g,
                                           int &start, int &rows) {
    if (g < p.E) {
        start = p.offsets[g];
        rows = p.offsets[g + 1] - start;
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
// Whether the routed groups have few rows each (another choice of tiles).
bool mfma_few_rows(long long routed, int E);
int mfma_dw_tiles(int d_ff, int act, bool few);
int mfma_splits(long long routed, int E, int shared_rows, int N, int K);
