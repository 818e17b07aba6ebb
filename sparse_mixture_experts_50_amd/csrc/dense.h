// Launch interfaces of the dense layer's kernels: linear layers with an
// epilogue, the feed-forward block, and their gradients (internal to the
// library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"

// What a product of rows leaves behind.
enum DenseEpilogue {
    DENSE_PLANE,      // fp32 sums, one plane for each range of K (and panel)
    DENSE_FORWARD,    // y = res + act(sum + bias)
    DENSE_GRAD        // h, dz, du from z (and u) and the gradient of h
};

// How a product is cut: tiles of 32 * rb rows (small: 64) by 256 (small: 128)
// columns (fp32: 128 by 128, small: 64 by 64), which two panels share, and K in
// `splits` ranges of `per` stages.  stream: the kernel for few
// rows, which cuts by itself.  The last nt2 columns of tiles may be lower ones
// (rb2, mt2 of them a column), which come after the others.
struct DensePlan {
    bool small, stream;
    int rb, mt, nt, splits, per;
    int rb2, mt2, nt2;
    __host__ __device__ long long tiles() const {
        return (long long)mt * (nt - nt2) * splits + (long long)mt2 * nt2;
    }
};

// out[M][N] = A B over K: A [M][K]; B [N][K] (transposed product), or [K][N]
// (bk: the rows' gradient).  Two panels: two products on one output tile
// (gated).  two: the sum of two products.
struct DenseRows {
    const void *a, *a2;       // a2: two
    const void *b, *b2;       // b2: the second panel's, or two
    int M, N, K;
    bool bk, two;
    int act, epilogue;
    const void *bias, *bias2; // [N] or null
    const void *res;          // [M][N] or null
    void *y;                  // DENSE_FORWARD
    float *plane;             // DENSE_PLANE: [splits][panels][M][N]
    // DENSE_GRAD: the gradient of h, as the sum of fp32 planes (q) or in the
    // layer's type (dy); h may be null.  h, dz and du, operands of the products
    // behind this one, are stored in the layer's type: the matrix cores take
    // bf16, and the two bf16 parts that hold an fp32 value would double those
    // products.  Each value is off by 0.0017 of itself in the mean of squares, as
    // a result's own rounding is: gradients end 0.0023 of their norm from the
    // definition, the forward 0.0019, and 99 % of the results are bit for bit the
    // definition's with these roundings alone
    const float *q;
    int q_planes;
    const void *dy;
    void *h, *dz, *du;
    DensePlan plan;
    __host__ __device__ int panels() const { return act == ACT_SWIGLU || act == ACT_GEGLU ? 2 : 1; }
};

// dtype: a moe_dtype.
DensePlan dense_rows_plan(int dtype, int M, int N, int K, int panels, bool bk, bool two);
hipError_t launch_dense_rows(const DenseRows &p, int dtype, hipStream_t s);
// (a split one's sums are left in p.plane)
hipError_t launch_dense_product(const DenseRows &p, int dtype, hipStream_t s);
// The epilogue of a product whose sums lie in p.plane (plan.splits of them).
hipError_t launch_dense_finish(const DenseRows &p, int dtype, hipStream_t s);
// (parts of launch_dense_rows, by source file)
hipError_t launch_dense_forward_mfma(const DenseRows &p, hipStream_t s);
hipError_t launch_dense_gated_mfma(const DenseRows &p, hipStream_t s);
hipError_t launch_dense_dx_mfma(const DenseRows &p, hipStream_t s);
hipError_t launch_dense_grad_mfma(const DenseRows &p, hipStream_t s);
hipError_t launch_dense_plane_mfma(const DenseRows &p, hipStream_t s);
hipError_t launch_dense_rows_f32(const DenseRows &p, hipStream_t s);
hipError_t launch_dense_stream(const DenseRows &p, int dtype, hipStream_t s);

// Weight gradients: up to three products out[R][C] = A^T B over M rows, A
// [M][R], B [M][C].  a2, b2: where the rows from M / 64 * 64 on are, 64 of
// them, zero from M on (bf16; not read if M % 64 == 0).
#define MOE_DENSE_MATS 3
struct DenseMat {
    const void *a, *b, *a2, *b2;
    void *out;
    int R, C;
};
struct DenseWeights {
    DenseMat m[MOE_DENSE_MATS];
    int count, M;
    bool small;
    int splits, per;          // ranges of the M axis, of `per` 64-row stages
    float *plane;             // splits > 1: of matrix k at plane + offset[k],
    size_t offset[MOE_DENSE_MATS];   // [splits][R][C]
};
// Fills in small, splits, per and offset; returns the planes' elements.
size_t dense_weights_plan(DenseWeights &p, int dtype);
hipError_t launch_dense_weights_mfma(const DenseWeights &p, hipStream_t s);   // large tiles

// Rows copied and rows zeroed, up to five items: dst[0, copied) = src, then
// zeros up to rows.
#define MOE_DENSE_TAILS 5
struct DenseTails {
    struct Item {
        const void *src;
        void *dst;
        int row_bytes, copied, rows;
    } t[MOE_DENSE_TAILS];
    int count;
};
// Column sums (bias gradients) of up to three [M][C] tensors: by ranges of
// rows into part, then joined.
#define MOE_DENSE_SUM_ROWS 256
struct DenseSums {
    struct Item {
        const void *src;
        void *out;
        float *part;          // [ranges][C]
        int C;
    } t[MOE_DENSE_MATS];
    int count, M;
};
__host__ __device__ inline int dense_sum_ranges(int M) {
    return (M + MOE_DENSE_SUM_ROWS - 1) / MOE_DENSE_SUM_ROWS;
}
// The sums by ranges (one range: the results) and the tails (bf16).
hipError_t launch_dense_sums(const DenseSums &p, const DenseTails &t, hipStream_t s);

// What a backward pass does once the pre-activations' gradients are there,
// each part of which may be missing: the rows' gradient, the weights', the
// biases'.
struct DenseBack {
    bool rows;
    DenseRows dx;
    DenseWeights w;
    DenseSums b;
    DenseTails t;
};
hipError_t launch_dense_back(const DenseBack &p, int dtype, hipStream_t s);
// The weights' gradients in small tiles, and what a launch before left to join
// (blocks of the rows' gradient, and of the column sums), bf16.
hipError_t launch_dense_weights_joins(const DenseWeights &p, const DenseRows &dx,
                                      const DenseSums &b, int rows, int sums, hipStream_t s);
// Products and sums of ranges, not yet joined (fp32).
hipError_t launch_dense_back_f32(const DenseBack &p, hipStream_t s);
// The rows' gradient (small tiles; a split one's sums are left in its plane)
// and launch_dense_sums, bf16.
hipError_t launch_dense_dx_sums(const DenseRows &p, const DenseSums &b, const DenseTails &t,
                                hipStream_t s);
