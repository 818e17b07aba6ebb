// Launch interfaces of the training kernels: expert-sorted rows, the
// layer's gradient, gradient clipping (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"

// ------------------------------------------------ expert-sorted rows
// Row space: routed rows 0 .. shared_base - 1 in expert order, then (with a
// shared expert) one row per token.
struct RowsParams {
    const void *tok;          // [T][d] token-order input (dispatch: x; combine_grad: dy)
    const void *tok2;         // second token-order input, or null
    const void *rows_in;      // [rows][d] (dispatch_grad, combine, combine_grad)
    void *rows_out;           // [rows][d] (dispatch, combine_grad)
    void *rows_out2;          // rows of tok2, or null
    void *tok_out;            // [T][d] (dispatch_grad, combine)
    const int32_t *slot_of;   // [T][k]
    const float *topk_w;      // [T][k]
    // dispatch of two inputs (the gradient's): the padded row space of
    // FfnGradParams, whose offsets are pad
    const int32_t *topk_idx;  // [T][k] (null: expert choice)
    const int32_t *offsets, *pad;   // [E+1]
    int32_t *pad_slot;        // [T][k]: slot_of in the padded space
    float *row_w;             // [rows] routing weight of each row (1: shared)
    float *dw;                // combine_grad: [T][k]
    int T, d, k, n_shared, shared_base;
};
hipError_t launch_dispatch_rows(const RowsParams &p, int dtype, hipStream_t s);
// tok_out[t] = sum over kept j of rows_in[slot] (times topk_w if weighted)
// + the shared row.
hipError_t launch_sum_rows(const RowsParams &p, int dtype, bool weighted,
                           hipStream_t s);
hipError_t launch_combine_rows_grad(const RowsParams &p, int dtype,
                                    hipStream_t s);

// ------------------------------------------------ the layer's gradient
// Row space: the shared expert's T rows, then the routed groups, every group
// padded with zero rows to a multiple of MOE_GRAD_ROWS, so that the products
// that sum over a group's rows take whole stages.
#define MOE_GRAD_ROWS 64
// Weight matrices and gradients by group: routed experts stacked, the
// shared expert apart.
struct FfnGradParams {
    const int32_t *offsets;   // [E+1]: padded group starts
    const void *xs, *dys;     // [rows][d] dispatched x and dy, zero in padding
    const float *row_w;       // [rows], zero in padding
    const void *w1, *w2, *w3, *ws1, *ws2, *ws3;
    const void *b1, *b2, *b3, *bs1, *bs2, *bs3;
    // h times the row weight, and the gradients of the pre-activations,
    // [rows][d_ff] each (du: SwiGLU)
    void *h, *dz, *du;
    float *q;                 // bf16: [q_splits][rows][d_ff], dy W2
    int q_splits, dx_splits;  // partial sums of q and dxs
    float *dw_part;           // [rows][dw_tiles]: <dy W2, h> by column tile
    int dw_tiles;
    float *dxs;               // [dx_splits][rows][d] fp32
    void *g_w1, *g_w2, *g_w3, *g_ws1, *g_ws2, *g_ws3;
    void *g_b1, *g_b2, *g_b3, *g_bs1, *g_bs2, *g_bs3;
    int E, n_shared, d, d_ff, act;
    int T;                    // shared rows, padded: [0, T)
    int rows;                 // upper bound of all rows
    int routed;           // routed rows (at most)
};
// Rows of the padded space for T tokens and R routed rows of E experts.
// Partial sums of q (its depth d) and of dxs (depth d_ff, or 2 d_ff gated).
int ffn_grad_q_splits(int dtype, long long routed, int E, int shared_rows, int d, int d_ff);
int ffn_grad_dx_splits(int dtype, long long routed, int E, int shared_rows, int d, int d_ff,
                       int act);
size_t padded_rows(long long T, int n_shared, long long R, int E);
// Group starts of the padded space, and its padding rows zeroed.
struct PadParams {
    const int32_t *offsets;   // [E+1]
    int32_t *pad;             // [E+1]
    void *xs, *dys;
    float *row_w;
    int E, n_shared, T, d;
};
hipError_t launch_pad_groups(const PadParams &p, int dtype, hipStream_t s);
// Column tiles that launch_ffn_act_grad writes to dw_part.
int ffn_grad_dw_tiles(int dtype, int d, int d_ff, int act, long long routed, int E);
hipError_t launch_ffn_act_grad(const FfnGradParams &p, int dtype, hipStream_t s);
hipError_t launch_ffn_row_grad(const FfnGradParams &p, int dtype, hipStream_t s);
hipError_t launch_ffn_weight_grad(const FfnGradParams &p, int dtype, hipStream_t s);
hipError_t launch_ffn_bias_grad(const FfnGradParams &p, int dtype, hipStream_t s);

struct RouterGradParams {
    const void *x;            // [T][d]
    const void *wr;           // [E][d]
    const float *add, *sub;   // [E] or null
    const int32_t *topk_idx;  // [T][k]
    const float *topk_w;      // [T][k]
    const int32_t *slot_of;   // [T][k]
    const float *f;           // [E] (aux != 0)
    const float *dw;          // [T][k], or null: from the row partials
    const float *dw_part;     // [rows][dw_tiles]
    int dw_tiles;
    // logits without the biases (where the losses need them): logit_splits
    // partial sums [T][E] over depth ranges of logit_depth
    float *logits;
    int logit_splits, logit_depth;
    void *dl;                 // [T][ep] fp32 (bf16: [T][ep / 64][2][64], two
                              // parts of each), columns E.. zero
    float *db_part;           // [ceil(T / MOE_ROUTER_GRAD_TOKENS)][E]
    float *wr_part;           // [splits][E][d]
    int splits;
    const void *dx_add;       // [T][d] in the layer's type, or null
    const float *dxs;         // [dx_splits][rows][d] expert row gradients, or null
    int dx_splits;
    size_t dx_plane;          // elements of one of them
    void *dx, *dwr;           // [T][d], [E][d]; null = not wanted
    float *db;                // [E] or null
    float aux, z;             // d L / d (sum_t f p) and d L / d (sum lse^2)
    int T, d, E, k, choice, n_shared, shared_base;
    int ep;                   // E rounded up to 64
};
// Tokens of one partial sum of the bias gradient.
#define MOE_ROUTER_GRAD_TOKENS 16
// Token ranges that the router weight gradient is split into.
int router_grad_splits(int dtype, int T, int d, int E);
// The forward's split bf16 router alone: partial logits of p.S ranges into
// p.part (router.hip).
struct RouterParams;
hipError_t launch_router_logits(const RouterParams &p, hipStream_t s);
hipError_t launch_router_grad(const RouterGradParams &p, int dtype, hipStream_t s);

// Zero bytes [0, n) (n a multiple of 2) with a kernel.
hipError_t launch_zero(void *dst, size_t n, hipStream_t s);

// ------------------------------------------------------------- clipping
// Tensors of one launch; more take several launches.
#define MOE_CLIP_TENSORS 96
struct ClipTensor {
    const void *src;
    void *dst;
    long long n;
};
struct ClipTable {
    ClipTensor t[MOE_CLIP_TENSORS];
    int32_t first[MOE_CLIP_TENSORS + 1];   // first block of each tensor
    uint32_t f32[(MOE_CLIP_TENSORS + 31) / 32];
    int32_t count;
};
// 32 KB chunks of a tensor (0 for an empty one), the unit of first[].
long long clip_chunks(long long n, int f32);
// One partial sum of squares per block.
hipError_t launch_clip_norm(const ClipTable &tab, double *part, int grid,
                            hipStream_t s);
hipError_t launch_clip_scale(const ClipTable &tab, const double *part,
                             int parts, float max_norm, float *norm, int grid,
                             hipStream_t s);
