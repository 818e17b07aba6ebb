/*
 * moe.h -- C ABI of the MI355X (gfx950) sparse Mixture-of-Experts FFN layer:
 * forward, gradient, and what a training step needs around them; dense linear
 * and feed-forward layers beside it, and the optimizer's step.
 *
 * The layer (sources are the pages' titles and sections):
 *   1. router logits  l[t,e] = x[t,:] . Wr[e,:] + add[e] - b[e], softmax
 *      ("MoE architecture deep dive", sec. 1.2 gating network; sec. 2.4
 *      aux-loss-free balancing subtracts b);
 *   2. top-k with renormalised weights (same page, sec. 1.3 steps 2-3;
 *      "AI-Research-SKILLs MoE training guide", sec. 3.1 and 4.2);
 *   3. per-expert counts, optional capacity C = floor(T/E * cf), stable
 *      token-order dispatch; overflow assignments skip the expert
 *      ("MoE architecture deep dive", sec. 2.3);
 *   4. each expert: W2 GELU(W1 x + b1) + b2 with exact erf GELU
 *      ("The expert group activated per token", sec. 3.1 FFN formula), or
 *      with SiLU, or gated: W2 (SiLU(W1 x + b1) * (W3 x + b3)) + b2
 *      (SwiGLU) ("AI-Research-SKILLs MoE training guide", sec. 6.1
 *      Mixtral block: its code uses Linear, SiLU, Linear, its text SwiGLU);
 *      optional always-on shared expert ("MoE architecture deep dive",
 *      sec. 3, DeepSeek-V3 shared expert);
 *   5. y[t] = sum_j w[t,j] Expert_{idx[t,j]}(x[t]) (+ Shared(x[t]))
 *      ("MoE architecture deep dive", sec. 1.1);
 *   6. f_i = count_i / (T k), p_i = mean_t p[t,i],
 *      L_aux = alpha * E * sum f_i p_i (same page, sec. 2.2; "AI-Research-
 *      SKILLs MoE training guide", sec. 4.3);
 *   7. balancing-bias step b_i += gamma * sign(count_i - target)
 *      ("MoE architecture deep dive", sec. 2.4).
 *
 * Expert-Choice routing (desc->routing == MOE_ROUTE_EXPERT_CHOICE;
 * "AI-Research-SKILLs MoE training guide", sec. 4.2, Expert Choice):
 * instead of steps 2-3 every expert picks its own C = desc->capacity
 * tokens, the C largest router logits l[t,e] in its column (ties to the
 * lower token index), so each expert holds exactly C tokens.  A pick is
 * weighted by the token's softmax probability p[t,e], not renormalised; a
 * token no expert picked gets y = 0 (plus the shared expert).  The mode
 * reuses the top-k data layout with k = E: each token is a candidate of
 * every expert, in expert order, and the capacity rule becomes the
 * per-expert top-C.  So for every t and e:
 *   topk_idx[t][e] = e,  topk_w[t][e] = p[t,e],
 *   slot_of[t][e]  = e*C + (rank of t among the picks of e in token
 *                    order), or -1 if e did not pick t,
 *   slot_token[e*C + r] = the r-th picked token of e (ascending),
 *   counts[e] = T, kept[e] = C, offsets[e] = e*C,
 * and f, p, L_aux and the monitors follow from those counts with k = E
 * (f_i = 1/E, L_aux = alpha * sum_i p_i = alpha).  The expert FFN and
 * combine steps are the same as for top-k.
 *
 * Conventions for every entry point:
 *   - Pointers named in the structs and arguments are DEVICE pointers unless
 *     stated otherwise; arrays are row-major and contiguous.
 *   - The caller owns every buffer, including the workspace sized by
 *     moe_workspace_size().  The library allocates nothing and only
 *     enqueues work on `stream` (a hipStream_t; NULL is the default
 *     stream).  No call synchronises the device or reads device data back
 *     to the host.  The one piece of state kept between calls is a
 *     per-device cache of the compute-unit count (filled on first use,
 *     atomically, with a value that never changes).
 *   - Tuning variables.  The environment variables MOE_ROUTER_SPLIT (0 / 1:
 *     fused or split bf16 router), MOE_TAIL_SPLIT (1..8: cap of the
 *     four-wave GEMM's K split of half-height tiles) and
 *     MOE_GEMM_VARIANT_UP / MOE_GEMM_VARIANT_DOWN (a tile variant id,
 *     used only where valid for the shape) are read at every call.  The
 *     first two change the workspace layout, so they are part of the
 *     workspace contract: keep them unchanged between moe_workspace_size()
 *     and the calls that use that workspace (a call whose workspace is then
 *     too small returns MOE_ERR_WORKSPACE).  Unset, every choice is a
 *     function of the descriptor and the device.
 *   - Arguments are validated on the host before any HIP call; a failed
 *     check returns a negative moe_status and enqueues nothing.  A failed
 *     kernel launch returns MOE_ERR_HIP.  T == 0 is valid: once the
 *     descriptor passes its checks the call returns MOE_OK, enqueues
 *     nothing and does not look at the pointers (but see moe_router_grad
 *     and moe_backward, which then zero weight gradients).  Non-finite
 *     inputs are not checked.
 *   - Calls on distinct streams with distinct workspaces may run
 *     concurrently.
 *   - The residual is not applied: a token whose every assignment
 *     overflowed capacity gets y = 0 exactly, so the caller's x + y passes
 *     it through unchanged.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1, /* null pointer, bad size, k out of range */
    MOE_ERR_UNSUPPORTED = -2, /* shape or dtype this library cannot run */
    MOE_ERR_WORKSPACE = -3,   /* workspace missing, too small or misaligned */
    MOE_ERR_HIP = -4,         /* a HIP launch failed */
    MOE_ERR_SCRATCH = -5      /* moe_forward_noalloc: the shape needs more
                                 than MOE_NOALLOC_SCRATCH_BYTES of scratch */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

typedef enum {
    MOE_ROUTE_TOPK = 0,          /* tokens choose k experts (default) */
    MOE_ROUTE_EXPERT_CHOICE = 1  /* experts choose C tokens */
} moe_routing_mode;

typedef enum {
    MOE_ACT_GELU = 0,    /* h = GELU(W1 x + b1), exact erf form */
    MOE_ACT_SILU = 1,    /* h = SiLU(W1 x + b1), SiLU(z) = z / (1 + e^-z) */
    MOE_ACT_SWIGLU = 2,  /* h = SiLU(W1 x + b1) * (W3 x + b3) */
    MOE_ACT_NONE = 3,    /* h = W1 x + b1 (moe_linear) */
    MOE_ACT_GEGLU = 4    /* h = GELU(W1 x + b1) * (W3 x + b3) (moe_linear,
                            moe_dense_*) */
} moe_activation;

/* Layer shape, host struct passed by pointer.
 *   T         tokens (>= 0)
 *   d         model width; multiple of 64
 *   E         routed experts, 1 <= E <= 256
 *   k         experts per token, 1 <= k <= min(E, 64); must equal E for
 *             expert choice
 *   d_ff      expert hidden width; multiple of 64
 *   n_shared  0 or 1 always-on shared expert (weight 1)
 *   dtype     MOE_F32 or MOE_BF16 for x, all weight matrices, the expert
 *             Linear biases and y (arithmetic accumulates in fp32)
 *   capacity  top-k: -1 = no limit, else C >= 0 assignments kept per
 *             expert (see moe_capacity); expert choice: tokens picked per
 *             expert, 0 <= C <= T (required)
 *   aux_alpha coefficient of L_aux (0.01 is the pages' usual value)
 *   routing   a moe_routing_mode
 *   expert_fp8 0: w1, w2, ws1, ws2 are in dtype; 1: they are OCP FP8 E4M3
 *             bytes with fp32 per-output-channel scales (moe_weights
 *             *_scale), a weight being e4m3(byte) * scale[row].  Needs
 *             dtype MOE_BF16 and d, d_ff multiples of 1024; activations,
 *             biases and y stay bf16.  The pages quote FP8 serving of the
 *             Mixtral layer ("MoE inference with vLLM"; "AI-Research-
 *             SKILLs MoE training guide", sec. 9); its target is the
 *             weight-streaming decode shape, whose bytes it halves.
 *   activation MOE_ACT_GELU, _SILU or _SWIGLU (routed and shared experts);
 *             MOE_ACT_SWIGLU needs d_ff a multiple of 128 for bf16 */
typedef struct moe_desc {
    int32_t T, d, E, k, d_ff;
    int32_t n_shared;
    int32_t dtype;
    int32_t capacity;
    float aux_alpha;
    int32_t routing;
    int32_t expert_fp8;
    int32_t activation;
} moe_desc;

/* Weights: caller-owned, read-only device buffers; NULL = absent.
 *   w_router    [E][d]        dtype                 (required)
 *   b_router    [E]           fp32, ADDED to logits (nn.Linear bias, or a
 *                             fixed per-expert skew)
 *   expert_bias [E]           fp32, SUBTRACTED from logits (aux-loss-free
 *                             balancing); enters softmax, selection and
 *                             weights
 *   w1, b1      [E][d_ff][d], [E][d_ff]   dtype (w1 required)
 *   w2, b2      [E][d][d_ff], [E][d]      dtype (w2 required)
 *   ws1..bs2    shared expert, same shapes without the E axis; ws1/ws2
 *               required iff n_shared == 1
 *   w1_scale    [E][d_ff] fp32, w2_scale [E][d], ws1_scale [d_ff],
 *   ws2_scale   [d]: per-output-channel scales of FP8 expert matrices
 *               (required iff expert_fp8, for the matrices present)
 *   w3, b3      [E][d_ff][d], [E][d_ff]  SwiGLU up projection (w3
 *               required iff activation == MOE_ACT_SWIGLU); ws3, bs3 the
 *               shared expert's; w3_scale [E][d_ff], ws3_scale [d_ff] for
 *               FP8.  W1 is then the gate projection. */
typedef struct moe_weights {
    const void *w_router;
    const float *b_router;
    const float *expert_bias;
    const void *w1, *b1;
    const void *w2, *b2;
    const void *ws1, *bs1, *ws2, *bs2;
    const float *w1_scale, *w2_scale, *ws1_scale, *ws2_scale;
    const void *w3, *b3, *ws3, *bs3;
    const float *w3_scale, *ws3_scale;
} moe_weights;

/* Routing results and statistics: caller-owned device buffers.
 *   topk_idx   [T][k] int32  selected experts, descending probability,
 *                            ties to the lower index
 *   topk_w     [T][k] fp32   renormalised weights (sum 1 per token)
 *   counts     [E]    int32  assignments per expert, before capacity
 *   kept       [E]    int32  min(counts, C)
 *   offsets    [E+1]  int32  exclusive prefix sum of kept
 *   slot_token [T*k]  int32  token of each expert-sorted slot; slots at
 *                            and beyond offsets[E] hold -1 (expert
 *                            choice: [E*C], every slot used; may be NULL
 *                            when E*C == 0)
 *   slot_of    [T][k] int32  slot of each assignment, -1 if it overflowed
 *   f, p       [E]    fp32   f_i = counts_i/(T k), p_i = mean_t p[t,i]
 *   l_aux      [1]    fp32   alpha * E * sum_i f_i p_i
 *   monitor    [6]    fp32   optional (NULL = not computed) router and load
 *                            monitors, in this order:
 *                            z-loss = mean_t (logsumexp_e logit[t,e])^2
 *                            ("AI-Research-SKILLs MoE training guide",
 *                            sec. 4.3), routing entropy in bits =
 *                            mean_t -sum_e p log2 p ("The expert group
 *                            activated per token", sec. 4.4), load imbalance
 *                            = max count / min count (+inf if an expert is
 *                            empty), utilization = nonempty experts / E,
 *                            drop rate = assignments over capacity / (T k)
 *                            (training guide, sec. 10.1), max share =
 *                            largest count / T ("MoE architecture deep
 *                            dive", sec. 4: collapse above 0.4) */
typedef struct moe_routing {
    int32_t *topk_idx;
    float *topk_w;
    int32_t *counts, *kept, *offsets;
    int32_t *slot_token, *slot_of;
    float *f, *p, *l_aux;
    float *monitor;
} moe_routing;

/* Host.  floor((double)T / E * cf): the capacity formula of "MoE
 * architecture deep dive", sec. 2.3.  Returns -1 if cf < 0 (no limit) and
 * MOE_ERR_INVALID_ARG if T < 0 or E < 1. */
int32_t moe_capacity(int32_t T, int32_t E, double cf);

/* Host.  Bytes of workspace the calls below need for this shape, or 0 if
 * the descriptor is invalid; a function of the descriptor alone (and of the
 * MOE_ROUTER_SPLIT and MOE_TAIL_SPLIT tuning variables, when set; a call
 * whose workspace is then too small returns MOE_ERR_WORKSPACE).  One
 * workspace serves every entry point;
 * moe_router_topk writes router partial sums into it that moe_permute reads,
 * and moe_grouped_ffn writes the expert outputs that moe_combine reads, so
 * run a sequence of calls with one workspace. */
size_t moe_workspace_size(const moe_desc *desc);

/* Host.  The grouped-GEMM kernel variant moe_ffn_up (up != 0) or
 * moe_ffn_down would run for this descriptor on the current device (an
 * internal id, for diagnostics and benchmark reports), or a negative
 * status if the descriptor is invalid.  Depends on the descriptor, the
 * device's CU count and the MOE_GEMM_VARIANT_UP / _DOWN tuning variables. */
int moe_gemm_variant(const moe_desc *desc, int up);

/* Host.  Number of K ranges S the four-wave 256-row grouped GEMM splits
 * each half-height (last <= 128 rows of a group) tile into for moe_ffn_up
 * (up != 0) or moe_ffn_down: 1 when there is no split or another variant
 * runs, else 2..8 with (K / 64) divisible by 2 S, so every unit covers a
 * whole number of 64-deep stage pairs.  A negative status if the
 * descriptor is invalid.  For diagnostics and tests. */
int moe_gemm_tail_split(const moe_desc *desc, int up);

/* Router GEMM with bias, softmax, top-k and renormalisation (layer steps
 * 1-2); bf16 layers run it as one kernel or, for deep or few-token shapes,
 * as partial logits over depth ranges (fp32, in the workspace) followed by
 * the routing kernel.  Reads x [T][d] and the router weights; writes
 * r->topk_idx, r->topk_w and per-token-tile probability column sums into
 * the workspace (consumed by moe_permute for p_i).  Expert choice: writes
 * topk_idx = e and topk_w = p[t,e] for all E experts, sets every entry of
 * r->slot_of (required) to -1, and writes the logits, transposed to
 * [E][T], into the workspace for moe_permute.  Top-k: also writes each
 * 32-token tile's count of picks per expert into the workspace. */
int moe_router_topk(const moe_desc *desc, const void *x,
                    const moe_weights *w, moe_routing *r, void *ws,
                    size_t ws_bytes, void *stream);

/* Counts, capacity, stable dispatch and statistics (layer steps 3 and 6).
 * Reads r->topk_idx and what moe_router_topk left in the workspace (the
 * probability partial sums and each 32-token tile's expert counts); writes
 * counts, kept, offsets, slot_token, slot_of, f, p, l_aux and, if
 * r->monitor is not NULL, the six monitors.  Expert choice: each expert's
 * top-C selection over the workspace logits replaces the capacity cut
 * (r->topk_idx is not read), and only the picked entries of slot_of are
 * written, over the -1 that moe_router_topk left there. */
int moe_permute(const moe_desc *desc, moe_routing *r, void *ws,
                size_t ws_bytes, void *stream);

/* moe_router_topk followed by moe_permute (layer steps 1-3 and 6), with
 * the same arguments, checks and results.  Where a decode-sized step
 * allows (bf16, top-k routing, E <= 32, T <= 32, T*k <= 256) the routing
 * and the dispatch run in one workgroup after the partial logits: two
 * kernel launches instead of three, with results equal to the two calls'
 * bit for bit.  The pages give fewer kernel launches as the reason for
 * fused MoE kernels in serving ("MoE inference with vLLM";
 * "AI-Research-SKILLs MoE training guide", sec. 9.2). */
int moe_route_dispatch(const moe_desc *desc, const void *x,
                       const moe_weights *w, moe_routing *r, void *ws,
                       size_t ws_bytes, void *stream);

/* Grouped expert FFNs (layer step 4): for every kept slot s of expert e,
 *   Yp[s] = W2_e GELU(W1_e x[slot_token[s]] + b1_e) + b2_e,
 * and, with a shared expert, Yp[R + t] = Shared(x[t]) for every token,
 * where R = T*k routed slots (expert choice: R = E*C).  Yp is written
 * into the workspace (dtype, [R + n_shared*T][d]); the hidden activations
 * are rounded to dtype between the two GEMMs.  Equivalent to moe_ffn_up
 * followed by moe_ffn_down. */
int moe_grouped_ffn(const moe_desc *desc, const void *x,
                    const moe_weights *w, const moe_routing *r, void *ws,
                    size_t ws_bytes, void *stream);

/* First half of moe_grouped_ffn: H[s] = GELU(W1_e x[token(s)] + b1_e)
 * (or the SiLU / SwiGLU form of desc->activation) into the workspace (one
 * kernel launch). */
int moe_ffn_up(const moe_desc *desc, const void *x, const moe_weights *w,
               const moe_routing *r, void *ws, size_t ws_bytes,
               void *stream);

/* Second half of moe_grouped_ffn: Yp[s] = W2_e H[s] + b2_e (one launch). */
int moe_ffn_down(const moe_desc *desc, const moe_weights *w,
                 const moe_routing *r, void *ws, size_t ws_bytes,
                 void *stream);

/* Weighted combine (layer step 5): y[t] = sum over kept j, in j order, of
 * topk_w[t,j] * Yp[slot_of[t,j]], plus Yp[R + t] with a shared expert;
 * fp32 accumulation, one rounding to dtype.  y is [T][d], dtype. */
int moe_combine(const moe_desc *desc, const moe_routing *r, void *y,
                void *ws, size_t ws_bytes, void *stream);

/* The whole forward: moe_route_dispatch (= moe_router_topk and
 * moe_permute), moe_grouped_ffn and moe_combine on one stream. */
int moe_forward(const moe_desc *desc, const void *x, const moe_weights *w,
                moe_routing *r, void *y, void *ws, size_t ws_bytes,
                void *stream);

/* Bytes of the static device scratch moe_forward_noalloc uses (16 MiB per
 * GPU the library runs on, held until the process ends). */
#define MOE_NOALLOC_SCRATCH_BYTES (16u << 20)

/* moe_forward without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation).  Same arguments and results as
 * moe_forward, minus ws / ws_bytes: the scratch (router partials, dispatch
 * histograms, hidden activations, expert outputs) lives in a file-scope
 * device array of MOE_NOALLOC_SCRATCH_BYTES per GPU, whose address is
 * looked up once per device on the first call there.  Allocates nothing:
 * no hipMalloc, hipFree or allocating library call.  Returns
 * MOE_ERR_SCRATCH, enqueuing nothing, when moe_workspace_size(desc)
 * exceeds the buffer (decode-sized layers fit: the Mixtral-shaped T = 32
 * step needs 2.4 MB).  No part of the scratch has to start at zero.  Every
 * call on one GPU shares that GPU's buffer, which keeps the last call's
 * contents: calls that overlap on one GPU (distinct streams, or host
 * threads) race and must be serialised by the caller. */
int moe_forward_noalloc(const moe_desc *desc, const void *x,
                        const moe_weights *w, moe_routing *r, void *y,
                        void *stream);

/* Balancing-bias step (layer step 7), in place on fp32 state:
 * bias[e] = bias[e] + gamma * sign(counts[e] - target), sign(0) = 0, one
 * fp32 add.  Apply after a forward; it affects the next call. */
int moe_bias_update(int32_t E, const int32_t *counts, float target,
                    float gamma, float *expert_bias, void *stream);

/* ------------------------------------------------------------------
 * Training.  Rows of an "expert-sorted" tensor are laid out as the expert
 * outputs of moe_grouped_ffn: R routed rows (T*k, or E*C for expert
 * choice) in the order of slot_token, then, with a shared expert, one row
 * per token (row R + t).  Routed rows at and beyond offsets[E] (capacity
 * drops) belong to no token: they are neither read nor written.  A row
 * tensor may be NULL when it has no rows.  Tensors of x's, the weights' and
 * the gradients' kinds start at 16-byte boundaries (MOE_ERR_INVALID_ARG), and
 * so do workspaces (MOE_ERR_WORKSPACE).
 * An output overlaps neither an input, the workspace nor another output,
 * except where that is allowed below; one that starts where one of them does
 * is refused (MOE_ERR_INVALID_ARG; moe_clip_grads: *norm only).
 * Everything here is written without atomics: the same inputs give the same
 * bits.
 * ------------------------------------------------------------------ */

/* Tokens into expert-sorted rows: xs[slot_of[t,j]] = x[t] for every kept
 * assignment, and xs[R + t] = x[t] with a shared expert.  Needs r->slot_of;
 * x [T][d], xs [R + n_shared*T][d], dtype. */
int moe_dispatch_rows(const moe_desc *desc, const moe_routing *r,
                      const void *x, void *xs, void *stream);

/* Gradient of moe_dispatch_rows: dx[t] = sum over kept j of
 * dxs[slot_of[t,j]], plus dxs[R + t] with a shared expert; summed in that
 * order in fp32, rounded once. */
int moe_dispatch_rows_grad(const moe_desc *desc, const moe_routing *r,
                           const void *dxs, void *dx, void *stream);

/* Expert-sorted rows back into token order with the routing weights
 * applied: y[t] = sum over kept j of topk_w[t,j] * ys[slot_of[t,j]], plus
 * ys[R + t] with a shared expert (moe_combine, of the caller's own rows).
 * Needs r->slot_of and r->topk_w. */
int moe_combine_rows(const moe_desc *desc, const moe_routing *r,
                     const void *ys, void *y, void *stream);

/* Gradient of moe_combine_rows, for dy [T][d]:
 *   dys[slot_of[t,j]] = topk_w[t,j] * dy[t],   dys[R + t] = dy[t],
 *   dw[t,j] = <dy[t], ys[slot_of[t,j]]>, 0 for a dropped assignment.
 * dw is [T][k] fp32; dys may be ys (in place). */
int moe_combine_rows_grad(const moe_desc *desc, const moe_routing *r,
                          const void *dy, const void *ys, void *dys,
                          float *dw, void *stream);

/* Gradients of a layer: caller-owned device buffers, each of its weight's
 * shape and type (b_router fp32; x [T][d]), written whole, not added to.
 * NULL = not wanted.  There is no gradient of expert_bias (balancing state,
 * stepped by moe_bias_update).  Groups without rows get zeros, and so do
 * (from moe_backward) gradients of weights that the descriptor's layer does
 * not have: w3, b3 without SwiGLU, the shared expert's without one. */
typedef struct moe_grads {
    void *x;
    void *w_router;
    float *b_router;
    void *w1, *b1, *w2, *b2;
    void *ws1, *bs1, *ws2, *bs2;
    void *w3, *b3, *ws3, *bs3;
} moe_grads;

/* Host.  Bytes of workspace of moe_router_grad and moe_backward, functions
 * of the descriptor alone (0 if it is invalid or d or d_ff exceeds 2^20,
 * and for moe_backward if expert_fp8: FP8 experts have no gradient).  The
 * workspace holds nothing between calls; it is not the forward's. */
size_t moe_router_grad_workspace_size(const moe_desc *desc);
size_t moe_grad_workspace_size(const moe_desc *desc);

/* Gradient of the router: of
 *   sum dw * topk_w + aux_scale * l_aux + z_scale * z-loss
 * (monitor[0]), with dw [T][k] fp32 the gradient of the routing weights (as
 * moe_combine_rows_grad leaves it) and the selection and the counts behind
 * f constant.  Top-k: through the renormalised weights; expert choice:
 * through the probabilities.  Reads x, w->w_router, b_router, expert_bias
 * (logits, where the losses need them) and of r topk_idx, topk_w, slot_of
 * and, for aux_scale != 0, f.  Writes g->x = dx_add + the router's part
 * (dx_add [T][d] dtype, NULL = 0, may be g->x), g->w_router, g->b_router.
 * The logits' gradient is fp32; into products of dtype bf16 it enters as the
 * sum of two bf16 values (to 2^-16), so each result is rounded to dtype once.
 * T == 0: the weights' gradients are zeroed. */
int moe_router_grad(const moe_desc *desc, const void *x,
                    const moe_weights *w, const moe_routing *r,
                    const float *dw, const void *dx_add, float aux_scale,
                    float z_scale, const moe_grads *g, void *ws,
                    size_t ws_bytes, void *stream);

/* Gradient of the whole layer (moe_forward) for dy [T][d]: of
 *   sum dy * y + aux_scale * l_aux + z_scale * z-loss,
 * through the experts, the shared expert, the combine and the router.  x, w
 * and r are the forward's (r needs topk_idx, topk_w, offsets, slot_of and,
 * for aux_scale != 0, f); nothing else of the forward is kept: hidden
 * activations are computed again.  Matrix products accumulate in fp32; the
 * hidden activations and their gradients are rounded to dtype between two
 * products.  Refuses expert_fp8 (MOE_ERR_UNSUPPORTED).  T == 0: the
 * weights' gradients are zeroed. */
int moe_backward(const moe_desc *desc, const void *x, const moe_weights *w,
                 const moe_routing *r, const void *dy, float aux_scale,
                 float z_scale, const moe_grads *g, void *ws,
                 size_t ws_bytes, void *stream);

/* One tensor of a clipping call: numel elements of dtype (a moe_dtype) at
 * src, aligned to their size; the result goes to dst (src for in place,
 * else not overlapping any other tensor; NULL = only counted). */
typedef struct moe_tensor {
    const void *src;
    void *dst;
    int64_t numel;
    int32_t dtype;
} moe_tensor;

/* Host.  Bytes of workspace moe_clip_grads needs for n tensors. */
size_t moe_clip_workspace_size(int32_t n);

/* Global gradient norm over n tensors and clipping:
 *   *norm = sqrt(sum over all tensors of src^2)      (device, fp32)
 *   dst = src * min(1, max_norm / (norm + 1e-6)),
 * rounded once to the tensor's type.  `tensors` is a HOST array, read during
 * the call; max_norm is finite and >= 0.  Squares are summed in double.  A
 * norm that is not a number reaches every dst; an infinite one gives zeros
 * (and not-a-number where src is infinite).  Tensors of any mix of sizes
 * and types, n == 0 included (norm 0). */
int moe_clip_grads(int32_t n, const moe_tensor *tensors, float max_norm,
                   float *norm, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------
 * Dense layers beside the sparse one: linear layers with an epilogue, the
 * feed-forward block of a model's layers that are not sparse, and their
 * gradients.  Row-major and contiguous as above; x, weights, outputs and
 * gradients are all of the descriptor's dtype and start at 16-byte
 * boundaries, workspaces too.  Outputs overlap neither inputs, the
 * workspace nor each other (refused where one starts where another does).
 * Written without atomics: the same inputs give the same bits.  Sums are
 * fp32, and a result is rounded to dtype once.
 * ------------------------------------------------------------------ */

/* M rows (0 <= M <= 2^22) of K features to N features; N and K multiples of
 * 64, at most 2^20; any moe_activation, gated for MOE_ACT_SWIGLU and _GEGLU. */
typedef struct moe_linear_desc {
    int32_t M, N, K;
    int32_t dtype;
    int32_t activation;
} moe_linear_desc;

/* w [N][K] (required), b [N]; gated: w3 [N][K] (required then), b3 [N]. */
typedef struct moe_linear_weights {
    const void *w, *b, *w3, *b3;
} moe_linear_weights;

/* Of x's and the weights' shapes, written whole; NULL = not wanted.  w3, b3
 * of a layer that is not gated get zeros. */
typedef struct moe_linear_grads {
    void *x, *w, *b, *w3, *b3;
} moe_linear_grads;

/* Host.  Workspace bytes, functions of the descriptor alone (0 if it is
 * invalid); nothing is held between calls. */
size_t moe_linear_workspace_size(const moe_linear_desc *desc);
size_t moe_linear_grad_workspace_size(const moe_linear_desc *desc);

/* y = residual + act(x w^T + b), gated: residual + a(x w^T + b) *
 * (x w3^T + b3) with a SiLU or GELU, in one kernel.  x [M][K], y and residual
 * (NULL = 0) [M][N]. */
int moe_linear(const moe_linear_desc *desc, const void *x,
               const moe_linear_weights *w, const void *residual, void *y,
               void *ws, size_t ws_bytes, void *stream);

/* Gradients of sum(dy * y) for dy [M][N], from the forward's x and weights
 * alone: the pre-activations are computed again.  g->x gets dx_add (NULL = 0)
 * as well.  (The residual's gradient is dy.)  Pre-activations' gradients are
 * rounded to dtype before the products.  M == 0: the weights' are zeroed. */
int moe_linear_grad(const moe_linear_desc *desc, const void *x,
                    const moe_linear_weights *w, const void *dy,
                    const void *dx_add, const moe_linear_grads *g, void *ws,
                    size_t ws_bytes, void *stream);

/* The feed-forward block: T tokens (0 <= T <= 2^22), width d, hidden width
 * d_ff, both multiples of 64 and at most 2^20; an activation that is not
 * MOE_ACT_NONE. */
typedef struct moe_dense_desc {
    int32_t T, d, d_ff;
    int32_t dtype;
    int32_t activation;
} moe_dense_desc;

/* w1 [d_ff][d], b1 [d_ff], w2 [d][d_ff], b2 [d]; gated: w3, b3 like w1, b1
 * (biases may be NULL). */
typedef struct moe_dense_weights {
    const void *w1, *b1, *w2, *b2, *w3, *b3;
} moe_dense_weights;
typedef struct moe_dense_grads {
    void *x, *w1, *b1, *w2, *b2, *w3, *b3;
} moe_dense_grads;

size_t moe_dense_workspace_size(const moe_dense_desc *desc);
size_t moe_dense_grad_workspace_size(const moe_dense_desc *desc);

/* y = residual + W2 h + b2 with h = act(W1 x + b1), gated: a(W1 x + b1) *
 * (W3 x + b3); h is rounded to dtype.  x, y, residual (NULL = 0) [T][d]. */
int moe_dense_forward(const moe_dense_desc *desc, const void *x,
                      const moe_dense_weights *w, const void *residual,
                      void *y, void *ws, size_t ws_bytes, void *stream);

/* Gradients of sum(dy * y); nothing of the forward is kept but x and the
 * weights.  g->x gets dx_add (NULL = 0) as well: dy itself where x is the
 * residual too.  h and the pre-activations' gradients are rounded to dtype
 * between products, dy W2 is not.  T == 0: the weights' are zeroed. */
int moe_dense_backward(const moe_dense_desc *desc, const void *x,
                       const moe_dense_weights *w, const void *dy,
                       const void *dx_add, const moe_dense_grads *g, void *ws,
                       size_t ws_bytes, void *stream);

/* One tensor of an AdamW step: numel elements, param (param_dtype) and
 * master updated in place, grad read.
 *   master         fp32 copy of a MOE_BF16 param, or NULL: the step is then
 *                  taken on it, and param is its value rounded to nearest
 *   m, v           the moments: fp32 [numel], or (state_bits 8) OCP E4M3
 *                  bytes [numel] in blocks of 32 elements, the second moment
 *                  as its square root
 *   m_scale,       (state_bits 8) uint8 [ceil(numel / 32)]: a block's values
 *   v_scale        are e4m3(byte) * 2^(scale - 127)
 * Fresh states and scales are zero bytes.  param and grad are aligned to
 * their elements, the others to 16 bytes (scales: 1).  numel == 0: skipped. */
typedef struct moe_adamw_tensor {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;
    uint8_t *m_scale, *v_scale;
    int64_t numel;
    double weight_decay;
    int32_t param_dtype, grad_dtype;
} moe_adamw_tensor;

/* What the tensors of a step share.  Host struct; steps, lr_scale and norm
 * are device pointers, or NULL:
 *   step        number t of this step, from 1 (steps == NULL)
 *   steps       steps done so far; t is one more, and the call adds 1 at its
 *               end (for a step captured into a graph)
 *   lr_scale    [1], multiplies lr (a schedule that a graph replays)
 *   norm        [1] of moe_clip_grads: gradients enter as
 *               grad * min(1, max_norm / (norm + 1e-6))
 *   state_bits  32 or 8
 *   stochastic  1: a MOE_BF16 param without master is rounded at random, up
 *               with the probability of the part that is lost; 0: to nearest.
 *               8-bit states always are
 *   seed        the random bits are a function of seed, t, the tensor's place
 *               in the list and the element alone */
typedef struct moe_adamw {
    double lr, beta1, beta2, eps;
    int64_t step;
    int64_t *steps;
    const float *lr_scale;
    const float *norm;
    double max_norm;
    int32_t state_bits;
    int32_t stochastic;
    uint32_t seed;
} moe_adamw;

/* One AdamW step over n tensors, with g the (clipped) gradient:
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   x = x - (lr weight_decay x
 *            + lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps))
 * in fp32, from m and v before they are rounded to 8 bits.  That rounding is
 * right in the mean for m and sqrt(v), so v gains its variance: 2 to 5 % in a
 * long run with normal gradients, 2/7 at most (but for values under 2^-28 of
 * their block's largest).  A block of 8-bit
 * states with a value that is not finite becomes not-a-number throughout.
 * Needs 0 <= beta1, beta2 < 1, eps >= 2^-126, lr and weight_decay >= 0, all
 * below 1e30.
 * `tensors` is a HOST array, read during the call.  No buffer of one tensor
 * may be one of another's (only a tensor's own are compared). */
int moe_adamw_step(const moe_adamw *h, int32_t n,
                   const moe_adamw_tensor *tensors, void *stream);

/* Host.  Static English text of a moe_status value. */
const char *moe_status_string(int status);

/* Host.  Library version string. */
const char *moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
