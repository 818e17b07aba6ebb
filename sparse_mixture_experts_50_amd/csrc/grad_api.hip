// Host side of the training entry points of include/moe.h: argument checks,
// workspace layout and launches, as for the forward in moe_api.hip.
#include <initializer_list>

#include "../../include/moe.h"
#include "grad.h"
#include "host.h"

namespace {

using namespace moe_host;

struct GradLayout {
    // the router's part, then the experts'
    size_t logits, dl, db_part, wr_part, router_total;
    size_t pad, pad_slot, row_w, xs, dys, h, dz, du, q, dw_part, dxs, total;
    size_t rows;
    int ep, splits, dw_tiles, q_splits, dx_splits;
    RouterPlan logit_plan;
};

GradLayout layout(const moe_desc *d) {
    GradLayout L;
    const size_t es = elem_bytes(d->dtype);
    size_t off = 0;
    auto take = [&off](size_t bytes) {
        const size_t at = off;
        off += align_up(bytes);
        return at;
    };
    L.ep = (d->E + 63) / 64 * 64;
    L.splits = router_grad_splits(d->dtype, d->T, d->d, d->E);
    L.logit_plan = router_plan(d->T, d->d, d->E, 256);
    if (d->dtype == MOE_F32) L.logit_plan.S = 1;
    L.logits = take((size_t)L.logit_plan.S * d->T * d->E * 4);
    L.dl = take((size_t)d->T * L.ep * 4);      // (bf16: two parts)
    L.db_part = take((size_t)((d->T + MOE_ROUTER_GRAD_TOKENS - 1) /
                              MOE_ROUTER_GRAD_TOKENS) * d->E * 4);
    L.wr_part = take(L.splits > 1 ? (size_t)L.splits * d->E * d->d * 4 : 0);
    L.router_total = off > 0 ? off : kAlign;
    L.rows = padded_rows(d->T, d->n_shared, routed_rows(d), d->E);
    L.pad = take((size_t)(d->E + 1) * 4);
    L.pad_slot = take((size_t)d->T * d->k * 4);
    // column tiles of <dy W2, h>, and <dy, b2>
    L.dw_tiles = ffn_grad_dw_tiles(d->dtype, d->d, d->d_ff, d->activation, routed_rows(d), d->E);
    L.row_w = take(L.rows * 4);
    L.xs = take(L.rows * d->d * es);
    L.dys = take(L.rows * d->d * es);
    L.h = take(L.rows * d->d_ff * es);
    L.dz = take(L.rows * d->d_ff * es);
    L.du = take(d->activation == MOE_ACT_SWIGLU ? L.rows * d->d_ff * es : 0);
    const int shared = d->n_shared * d->T;
    L.q_splits = ffn_grad_q_splits(d->dtype, routed_rows(d), d->E, shared, d->d, d->d_ff);
    L.dx_splits = ffn_grad_dx_splits(d->dtype, routed_rows(d), d->E, shared, d->d, d->d_ff,
                                     d->activation);
    L.q = take(d->dtype == MOE_BF16 ? L.q_splits * L.rows * d->d_ff * 4 : 0);
    L.dw_part = take(L.rows * (L.dw_tiles + 1) * 4);
    L.dxs = take(L.dx_splits * L.rows * d->d * 4);
    // a row tile of 256 may reach past the last row of any operand
    take((size_t)256 * (d->d > d->d_ff ? d->d : d->d_ff) * es);
    L.total = off;
    return L;
}

RowsParams rows_params(const moe_desc *d, const moe_routing *r) {
    RowsParams p = {};
    p.slot_of = r->slot_of;
    p.topk_w = r->topk_w;
    p.T = d->T;
    p.d = d->d;
    p.k = d->k;
    p.n_shared = d->n_shared;
    p.shared_base = (int)routed_rows(d);
    return p;
}

// Row tensors may be NULL when they have no rows (expert choice with C = 0
// and no shared expert).
bool have_rows(const moe_desc *d) {
    return routed_rows(d) + (long long)d->n_shared * d->T > 0;
}

// Vectors of 16 bytes are moved: operands are aligned to them.
template <typename... P> bool aligned(const P *...p) {
    return ((((uintptr_t)p & 15) == 0) && ...);
}
bool aligned_weights(const moe_weights *w) {
    return aligned(w->w_router, w->w1, w->w2, w->w3, w->ws1, w->ws2, w->ws3, w->b1,
                   w->b2, w->b3, w->bs1, w->bs2, w->bs3);
}
bool aligned_grads(const moe_grads *g) {
    return aligned(g->x, g->w_router, g->w1, g->w2, g->w3, g->ws1, g->ws2, g->ws3,
                   g->b1, g->b2, g->b3, g->bs1, g->bs2, g->bs3);
}

// Whether an output starts where an input or another output does.
bool clash(std::initializer_list<const void *> outs,
           std::initializer_list<const void *> ins) {
    for (const void *const *o = outs.begin(); o != outs.end(); ++o) {
        if (!*o) continue;
        for (const void *i : ins)
            if (*o == i) return true;
        for (const void *const *q = outs.begin(); q != o; ++q)
            if (*o == *q) return true;
    }
    return false;
}

// The gradient's kernels hold row offsets within a tile in 32 bits.
int check_grad_desc(const moe_desc *d) {
    const int st = check_desc(d);
    if (st != MOE_OK) return st;
    return d->d > (1 << 20) || d->d_ff > (1 << 20) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_router(const moe_desc *d, const moe_weights *w,
                 const moe_routing *r, float aux_scale) {
    if (!w || !w->w_router || !r || !r->topk_w || !r->slot_of ||
        (!r->topk_idx && !expert_choice(d)) || (aux_scale != 0.0f && !r->f))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

RouterGradParams router_params(const moe_desc *d, const void *x,
                               const moe_weights *w, const moe_routing *r,
                               float aux_scale, float z_scale,
                               const moe_grads *g, void *ws,
                               const GradLayout &L) {
    RouterGradParams p = {};
    p.x = x;
    p.wr = w->w_router;
    p.add = w->b_router;
    p.sub = w->expert_bias;
    p.topk_idx = r->topk_idx;
    p.topk_w = r->topk_w;
    p.slot_of = r->slot_of;
    p.f = r->f;
    p.logits = (float *)at(ws, L.logits);
    p.logit_splits = L.logit_plan.S;
    p.logit_depth = L.logit_plan.kc;
    p.dl = at(ws, L.dl);
    p.db_part = (float *)at(ws, L.db_part);
    p.wr_part = (float *)at(ws, L.wr_part);
    p.splits = L.splits;
    p.dx = g->x;
    p.dwr = g->w_router;
    p.db = g->b_router;
    p.aux = (float)((double)aux_scale * d->aux_alpha * d->E / d->T);
    p.z = (float)(2.0 * z_scale / d->T);
    p.T = d->T;
    p.d = d->d;
    p.E = d->E;
    p.k = d->k;
    p.choice = expert_choice(d);
    p.n_shared = d->n_shared;
    p.shared_base = (int)routed_rows(d);
    p.ep = L.ep;
    return p;
}

int check_ffn(const moe_desc *d, const moe_weights *w, const moe_routing *r) {
    if (!w || !w->w1 || !w->w2 || !r || !r->offsets) return MOE_ERR_INVALID_ARG;
    if (d->n_shared && (!w->ws1 || !w->ws2)) return MOE_ERR_INVALID_ARG;
    if (d->activation == MOE_ACT_SWIGLU &&
        (!w->w3 || (d->n_shared && !w->ws3)))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// The gradient of a call without tokens is zero.
int zero_grads(const moe_desc *d, const moe_grads *g, hipStream_t s) {
    const size_t es = elem_bytes(d->dtype), E = d->E;
    const size_t mat = (size_t)d->d * d->d_ff * es;
    const size_t up = d->d_ff * es, down = d->d * es;
    const struct {
        void *p;
        size_t n;
    } all[] = {
        {g->w_router, E * d->d * es}, {g->b_router, E * 4},
        {g->w1, E * mat}, {g->b1, E * up}, {g->w2, E * mat}, {g->b2, E * down},
        {g->w3, E * mat}, {g->b3, E * up}, {g->ws1, mat}, {g->bs1, up},
        {g->ws2, mat}, {g->bs2, down}, {g->ws3, mat}, {g->bs3, up},
    };
    for (const auto &a : all)
        if (a.p && launch_zero(a.p, a.n, s) != hipSuccess) return MOE_ERR_HIP;
    return MOE_OK;
}

// The wanted gradients of weights that take no part in the layer.
moe_grads absent_grads(const moe_desc *d, const moe_grads *g) {
    moe_grads a = {};
    const bool gated = d->activation == MOE_ACT_SWIGLU;
    if (!gated) {
        a.w3 = g->w3;
        a.b3 = g->b3;
    }
    if (!d->n_shared) {
        a.ws1 = g->ws1;
        a.bs1 = g->bs1;
        a.ws2 = g->ws2;
        a.bs2 = g->bs2;
    }
    if (!gated || !d->n_shared) {
        a.ws3 = g->ws3;
        a.bs3 = g->bs3;
    }
    return a;
}

constexpr int kClipBlocks = 2048;
constexpr int kClipLeast = 64;

// Tables of a clip call, and the blocks of each table's norm launch.
int clip_tables(int n) { return (n + MOE_CLIP_TENSORS - 1) / MOE_CLIP_TENSORS; }
int clip_blocks(int tables) {
    if (tables < 1) return 0;
    const int b = kClipBlocks / tables;
    return b < kClipLeast ? kClipLeast : b;
}

}  // namespace

extern "C" {

int moe_dispatch_rows(const moe_desc *desc, const moe_routing *r,
                      const void *x, void *xs, void *stream) {
    int st = check_desc(desc);
    if (st != MOE_OK) return st;
    if (desc->T == 0) return MOE_OK;
    if (!x || !r || !r->slot_of || (!xs && have_rows(desc)) || !aligned(x, xs) ||
        clash({xs}, {x, r->slot_of}))
        return MOE_ERR_INVALID_ARG;
    RowsParams p = rows_params(desc, r);
    p.tok = x;
    p.rows_out = xs;
    return to_status(launch_dispatch_rows(p, desc->dtype, (hipStream_t)stream));
}

int moe_dispatch_rows_grad(const moe_desc *desc, const moe_routing *r,
                           const void *dxs, void *dx, void *stream) {
    int st = check_desc(desc);
    if (st != MOE_OK) return st;
    if (desc->T == 0) return MOE_OK;
    if (!dx || !r || !r->slot_of || (!dxs && have_rows(desc)) ||
        !aligned(dx, dxs) || clash({dx}, {dxs, r->slot_of}))
        return MOE_ERR_INVALID_ARG;
    RowsParams p = rows_params(desc, r);
    p.rows_in = dxs;
    p.tok_out = dx;
    return to_status(launch_sum_rows(p, desc->dtype, false, (hipStream_t)stream));
}

int moe_combine_rows(const moe_desc *desc, const moe_routing *r,
                     const void *ys, void *y, void *stream) {
    int st = check_desc(desc);
    if (st != MOE_OK) return st;
    if (desc->T == 0) return MOE_OK;
    if (!y || !r || !r->slot_of || !r->topk_w || (!ys && have_rows(desc)) ||
        !aligned(y, ys) || clash({y}, {ys, r->slot_of, r->topk_w}))
        return MOE_ERR_INVALID_ARG;
    RowsParams p = rows_params(desc, r);
    p.rows_in = ys;
    p.tok_out = y;
    return to_status(launch_sum_rows(p, desc->dtype, true, (hipStream_t)stream));
}

int moe_combine_rows_grad(const moe_desc *desc, const moe_routing *r,
                          const void *dy, const void *ys, void *dys, float *dw,
                          void *stream) {
    int st = check_desc(desc);
    if (st != MOE_OK) return st;
    if (desc->T == 0) return MOE_OK;
    if (!dy || !dw || !r || !r->slot_of || !r->topk_w ||
        ((!ys || !dys) && have_rows(desc)) || !aligned(dy, ys, dys) ||
        clash({dys, dw}, {dy, r->slot_of, r->topk_w}) || dw == ys)
        return MOE_ERR_INVALID_ARG;
    RowsParams p = rows_params(desc, r);
    p.tok = dy;
    p.rows_in = ys;
    p.rows_out = dys;
    p.dw = dw;
    return to_status(launch_combine_rows_grad(p, desc->dtype, (hipStream_t)stream));
}

size_t moe_router_grad_workspace_size(const moe_desc *desc) {
    if (check_grad_desc(desc) != MOE_OK) return 0;
    return layout(desc).router_total;
}

size_t moe_grad_workspace_size(const moe_desc *desc) {
    if (check_grad_desc(desc) != MOE_OK || desc->expert_fp8) return 0;
    return layout(desc).total;
}

int moe_router_grad(const moe_desc *desc, const void *x, const moe_weights *w,
                    const moe_routing *r, const float *dw, const void *dx_add,
                    float aux_scale, float z_scale, const moe_grads *g,
                    void *ws, size_t ws_bytes, void *stream) {
    int st = check_grad_desc(desc);
    if (st != MOE_OK) return st;
    if (!g) return MOE_ERR_INVALID_ARG;
    if (desc->T == 0) {
        moe_grads only = {};
        only.w_router = g->w_router;
        only.b_router = g->b_router;
        return zero_grads(desc, &only, (hipStream_t)stream);
    }
    if (!x || !dw) return MOE_ERR_INVALID_ARG;
    if ((st = check_router(desc, w, r, aux_scale)) != MOE_OK) return st;
    if (!aligned(x, dx_add, w->w_router, g->x, g->w_router)) return MOE_ERR_INVALID_ARG;
    const GradLayout L = layout(desc);
    if (!ws || ws_bytes < L.router_total || !aligned(ws)) return MOE_ERR_WORKSPACE;
    if (clash({g->x, g->w_router, g->b_router},
              {x, dw, ws, w->w_router, w->b_router, w->expert_bias, r->topk_idx,
               r->topk_w, r->slot_of, r->f}) ||
        clash({g->w_router, g->b_router}, {dx_add}))
        return MOE_ERR_INVALID_ARG;
    RouterGradParams p =
        router_params(desc, x, w, r, aux_scale, z_scale, g, ws, L);
    p.dw = dw;
    p.dx_add = dx_add;
    return to_status(launch_router_grad(p, desc->dtype, (hipStream_t)stream));
}

int moe_backward(const moe_desc *desc, const void *x, const moe_weights *w,
                 const moe_routing *r, const void *dy, float aux_scale,
                 float z_scale, const moe_grads *g, void *ws, size_t ws_bytes,
                 void *stream) {
    int st = check_grad_desc(desc);
    if (st != MOE_OK) return st;
    if (desc->expert_fp8) return MOE_ERR_UNSUPPORTED;
    if (!g) return MOE_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    if (desc->T == 0) return zero_grads(desc, g, s);
    if (!x || !dy) return MOE_ERR_INVALID_ARG;
    if ((st = check_router(desc, w, r, aux_scale)) != MOE_OK) return st;
    if ((st = check_ffn(desc, w, r)) != MOE_OK) return st;
    if (!aligned(x, dy) || !aligned_weights(w) || !aligned_grads(g))
        return MOE_ERR_INVALID_ARG;
    const GradLayout L = layout(desc);
    if (!ws || ws_bytes < L.total || !aligned(ws)) return MOE_ERR_WORKSPACE;
    if (clash({g->x, g->w_router, g->b_router, g->w1, g->b1, g->w2, g->b2, g->ws1,
               g->bs1, g->ws2, g->bs2, g->w3, g->b3, g->ws3, g->bs3},
              {x, dy, ws, w->w_router, w->b_router, w->expert_bias, w->w1, w->b1,
               w->w2, w->b2, w->ws1, w->bs1, w->ws2, w->bs2, w->w3, w->b3, w->ws3,
               w->bs3, r->topk_idx, r->topk_w, r->offsets, r->slot_of, r->f}))
        return MOE_ERR_INVALID_ARG;

    RowsParams rp = rows_params(desc, r);
    rp.tok = x;
    rp.tok2 = dy;
    rp.rows_out = at(ws, L.xs);
    rp.rows_out2 = at(ws, L.dys);
    rp.row_w = (float *)at(ws, L.row_w);
    rp.topk_idx = expert_choice(desc) ? nullptr : r->topk_idx;
    rp.offsets = r->offsets;
    rp.pad = (const int32_t *)at(ws, L.pad);
    rp.pad_slot = (int32_t *)at(ws, L.pad_slot);
    rp.shared_base = 0;

    PadParams pp;
    pp.offsets = r->offsets;
    pp.pad = (int32_t *)at(ws, L.pad);
    pp.xs = rp.rows_out;
    pp.dys = rp.rows_out2;
    pp.row_w = rp.row_w;
    pp.E = desc->E;
    pp.n_shared = desc->n_shared;
    pp.T = desc->T;
    pp.d = desc->d;

    FfnGradParams p = {};
    p.offsets = pp.pad;
    p.xs = at(ws, L.xs);
    p.dys = at(ws, L.dys);
    p.row_w = rp.row_w;
    p.w1 = w->w1;
    p.w2 = w->w2;
    p.w3 = w->w3;
    p.b1 = w->b1;
    p.b2 = w->b2;
    p.b3 = w->b3;
    if (desc->n_shared) {
        p.ws1 = w->ws1;
        p.ws2 = w->ws2;
        p.ws3 = w->ws3;
        p.bs1 = w->bs1;
        p.bs2 = w->bs2;
        p.bs3 = w->bs3;
        p.g_ws1 = g->ws1;
        p.g_ws2 = g->ws2;
        p.g_ws3 = g->ws3;
        p.g_bs1 = g->bs1;
        p.g_bs2 = g->bs2;
        p.g_bs3 = g->bs3;
    }
    p.h = at(ws, L.h);
    p.dz = at(ws, L.dz);
    p.du = at(ws, L.du);
    p.q = (float *)at(ws, L.q);
    p.dw_part = (float *)at(ws, L.dw_part);
    p.dw_tiles = L.dw_tiles + (p.b2 || p.bs2 ? 1 : 0);
    p.dxs = (float *)at(ws, L.dxs);
    p.g_w1 = g->w1;
    p.g_w2 = g->w2;
    p.g_b1 = g->b1;
    p.g_b2 = g->b2;
    if (desc->activation == MOE_ACT_SWIGLU) {
        p.g_w3 = g->w3;
        p.g_b3 = g->b3;
    } else {
        p.w3 = p.b3 = p.ws3 = p.bs3 = nullptr;
        p.g_ws3 = p.g_bs3 = nullptr;
    }
    p.E = desc->E;
    p.n_shared = desc->n_shared;
    p.T = (desc->T + MOE_GRAD_ROWS - 1) / MOE_GRAD_ROWS * MOE_GRAD_ROWS;
    p.d = desc->d;
    p.d_ff = desc->d_ff;
    p.act = desc->activation;
    p.rows = (int)L.rows;
    p.q_splits = L.q_splits;
    p.dx_splits = L.dx_splits;
    p.routed = (int)routed_rows(desc);

    const moe_grads absent = absent_grads(desc, g);
    if ((st = zero_grads(desc, &absent, s)) != MOE_OK) return st;
    const bool weights = p.g_w1 || p.g_w2 || p.g_w3 || p.g_ws1 || p.g_ws2 || p.g_ws3;
    const bool biases = p.g_b1 || p.g_b2 || p.g_b3 || p.g_bs1 || p.g_bs2 || p.g_bs3;
    const bool router = g->x || g->w_router || g->b_router;
    if (!weights && !biases && !router) return MOE_OK;
    const int dt = desc->dtype;
    if (launch_pad_groups(pp, dt, s) != hipSuccess) return MOE_ERR_HIP;
    if (launch_dispatch_rows(rp, dt, s) != hipSuccess) return MOE_ERR_HIP;
    if (launch_ffn_act_grad(p, dt, s) != hipSuccess) return MOE_ERR_HIP;
    if (g->x && launch_ffn_row_grad(p, dt, s) != hipSuccess) return MOE_ERR_HIP;
    if (weights && launch_ffn_weight_grad(p, dt, s) != hipSuccess)
        return MOE_ERR_HIP;
    if (biases && launch_ffn_bias_grad(p, dt, s) != hipSuccess) return MOE_ERR_HIP;
    if (router) {
        RouterGradParams q =
            router_params(desc, x, w, r, aux_scale, z_scale, g, ws, L);
        q.dw_part = p.dw_part;
        q.dw_tiles = p.dw_tiles;
        q.dxs = p.dxs;
        q.dx_splits = p.dx_splits;
        q.dx_plane = (size_t)p.rows * p.d;
        q.slot_of = rp.pad_slot;
        q.shared_base = 0;
        if (launch_router_grad(q, dt, s) != hipSuccess) return MOE_ERR_HIP;
    }
    return MOE_OK;
}

size_t moe_clip_workspace_size(int32_t n) {
    if (n < 0) return 0;
    const int tables = clip_tables(n);
    const size_t bytes = (size_t)tables * clip_blocks(tables) * sizeof(double);
    return align_up(bytes ? bytes : 1);
}

int moe_clip_grads(int32_t n, const moe_tensor *tensors, float max_norm,
                   float *norm, void *ws, size_t ws_bytes, void *stream) {
    if (n < 0 || (n > 0 && !tensors) || !norm || !(max_norm >= 0.0f) ||
        max_norm > 3.4028234e38f)
        return MOE_ERR_INVALID_ARG;
    bool write = false;
    for (int i = 0; i < n; ++i) {
        const moe_tensor &t = tensors[i];
        if (t.numel < 0 || (t.numel > 0 && !t.src)) return MOE_ERR_INVALID_ARG;
        if (t.dtype != MOE_F32 && t.dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
        const uintptr_t es = elem_bytes(t.dtype);
        if ((uintptr_t)t.src % es || (uintptr_t)t.dst % es)
            return MOE_ERR_INVALID_ARG;
        write = write || (t.dst && t.numel > 0);
        // chunk numbers are 32-bit within a launch
        if (t.numel > (1ll << 40)) return MOE_ERR_UNSUPPORTED;
    }
    if (!ws || ws_bytes < moe_clip_workspace_size(n) || !aligned(ws))
        return MOE_ERR_WORKSPACE;
    for (int i = 0; i < n; ++i)
        if (tensors[i].src == norm || tensors[i].dst == norm)
            return MOE_ERR_INVALID_ARG;
    if (ws == norm) return MOE_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    const int tables = clip_tables(n), most = clip_blocks(tables);
    double *part = (double *)ws;
    auto fill = [&](int k, ClipTable &tab) {
        tab = ClipTable{};
        const int i0 = k * MOE_CLIP_TENSORS;
        tab.count = n - i0 < MOE_CLIP_TENSORS ? n - i0 : MOE_CLIP_TENSORS;
        long long chunks = 0;
        for (int i = 0; i < tab.count; ++i) {
            const moe_tensor &t = tensors[i0 + i];
            const int f32 = t.dtype == MOE_F32;
            tab.t[i] = {t.src, t.dst, (long long)t.numel};
            tab.first[i] = (int32_t)chunks;
            if (f32) tab.f32[i >> 5] |= 1u << (i & 31);
            chunks += clip_chunks(t.numel, f32);
            if (chunks > 0x7fffffffll) return (long long)-1;
        }
        tab.first[tab.count] = (int32_t)chunks;
        return chunks;
    };
    ClipTable tab;
    int parts = 0;
    for (int k = 0; k < tables; ++k)
        if (fill(k, tab) < 0) return MOE_ERR_UNSUPPORTED;
    for (int k = 0; k < tables; ++k) {
        const long long chunks = fill(k, tab);
        if (chunks == 0) continue;
        const int grid = (int)(chunks < most ? chunks : most);
        if (launch_clip_norm(tab, part + parts, grid, s) != hipSuccess)
            return MOE_ERR_HIP;
        parts += grid;
    }
    float *out = norm;
    // backwards, as within a table: the last tensors are still cached
    for (int k = tables - 1; k >= 0 && write; --k) {
        const long long chunks = fill(k, tab);
        if (chunks == 0) continue;
        const int grid = (int)(chunks < kClipBlocks ? chunks : kClipBlocks);
        if (launch_clip_scale(tab, part, parts, max_norm, out, grid, s) != hipSuccess)
            return MOE_ERR_HIP;
        out = nullptr;
    }
    if (out) {                        // the norm alone
        tab = ClipTable{};
        if (launch_clip_scale(tab, part, parts, max_norm, out, 1, s) != hipSuccess)
            return MOE_ERR_HIP;
    }
    return MOE_OK;
}

}  // extern "C"
