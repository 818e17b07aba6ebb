// Launch interface of the AdamW step (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

// Elements of an 8-bit state that share a scale.
#define MOE_ADAMW_BLOCK 32
// Elements of the unit of work that tensors are dealt out in: multiples of the
// least, at most the other.
#define MOE_ADAMW_LEAST 2048
#define MOE_ADAMW_CHUNK 16384
// Tensors of one launch (the table travels as a kernel argument).
#define MOE_ADAMW_TENSORS 40

enum { ADAMW_PARAM_F32 = 1, ADAMW_GRAD_F32 = 2, ADAMW_ALIGNED = 4 };

struct AdamwTensor {
    void *param;
    const void *grad;
    float *master;            // or null
    void *m, *v;              // fp32, or e4m3 codes
    uint8_t *m_scale, *v_scale;
    long long n;
    double decay;             // weight decay
    int32_t flags, pad;
};
struct AdamwTable {
    AdamwTensor t[MOE_ADAMW_TENSORS];
    int32_t first[MOE_ADAMW_TENSORS + 1];   // first chunk of each tensor
    int32_t count;
};
struct AdamwParams {
    double lr, log_b1, log_b2;
    double bias1, bias2;      // 1 - beta^t (without `steps`)
    const int64_t *steps;     // steps done before this one, or null
    int64_t step;             // number of this step (without `steps`)
    const float *lr_scale;    // or null
    const float *norm;        // or null
    double max_norm;
    float b1, c1, b2, c2, eps;
    uint32_t seed;
    int32_t index0;           // index of the table's first tensor
    int32_t chunk;
    int32_t stochastic;       // bf16 parameters without a master copy
};
hipError_t launch_adamw(const AdamwTable &tab, const AdamwParams &p, int bits,
                        int grid, hipStream_t s);
// *steps += 1.
hipError_t launch_adamw_tick(int64_t *steps, hipStream_t s);
