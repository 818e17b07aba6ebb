// Host side of the dense layer's entry points of include/moe.h: argument
// checks, workspace layout and launches.
#include "../../include/moe.h"
#include "dense.h"
#include "grad.h"
#include "host.h"

using namespace moe_host;

namespace {

bool gated(int act) { return act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU; }

int check_sizes(int M, int N, int K, int dtype, int act) {
    if (M < 0 || N < 1 || K < 1 || act < MOE_ACT_GELU || act > MOE_ACT_GEGLU)
        return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    // 32-bit row offsets within a tile, and grids of row ranges
    if (N % 64 || K % 64 || N > (1 << 20) || K > (1 << 20) || M > (1 << 22))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int check_linear(const moe_linear_desc *d) {
    return d ? check_sizes(d->M, d->N, d->K, d->dtype, d->activation) : MOE_ERR_INVALID_ARG;
}
int check_dense(const moe_dense_desc *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->activation == MOE_ACT_NONE) return MOE_ERR_INVALID_ARG;
    return check_sizes(d->T, d->d_ff, d->d, d->dtype, d->activation);
}

size_t most(size_t a, size_t b) { return a > b ? a : b; }
size_t pad64(int M) { return ((size_t)M + 63) / 64 * 64; }

struct Take {
    size_t off = 0;
    size_t operator()(size_t bytes) {
        const size_t at = off;
        off += align_up(bytes);
        return at;
    }
};

size_t plane_bytes(const DensePlan &p, int M, int N, int panels) {
    return p.splits > 1 ? (size_t)p.splits * panels * M * N * 4 : 0;
}

// ------------------------------------------------------------ linear

DensePlan linear_plan(const moe_linear_desc *d) {
    return dense_rows_plan(d->dtype, d->M, d->N, d->K, gated(d->activation) ? 2 : 1, false, false);
}

size_t linear_bytes(const moe_linear_desc *d, const DensePlan &plan) {
    const size_t n = align_up(plane_bytes(plan, d->M, d->N, gated(d->activation) ? 2 : 1));
    return n ? n : kAlign;
}

struct LinearLayout {
    size_t dz, du, x_tail, dz_tail, plane, w_plane, sums, total;
    DensePlan up, dx;
    DenseWeights w;
};

// The weight gradients' operands, where they are wanted.
DenseWeights linear_weights(const moe_linear_desc *d, const void *x, const void *dz,
                            const void *du, const moe_linear_grads *g) {
    DenseWeights w = {};
    w.M = d->M;
    if (g->w) w.m[w.count++] = {dz, x, nullptr, nullptr, g->w, d->N, d->K};
    if (g->w3 && gated(d->activation))
        w.m[w.count++] = {du, x, nullptr, nullptr, g->w3, d->N, d->K};
    return w;
}

LinearLayout linear_layout(const moe_linear_desc *d) {
    LinearLayout L = {};
    const size_t es = elem_bytes(d->dtype);
    const bool two = gated(d->activation), none = d->activation == MOE_ACT_NONE;
    const size_t rows = pad64(d->M);
    Take take;
    L.up = linear_plan(d);
    L.dx = dense_rows_plan(d->dtype, d->M, d->K, d->N, 1, true, two);
    L.dz = take(none ? 0 : rows * d->N * es);
    L.du = take(two ? rows * d->N * es : 0);
    L.x_tail = take((size_t)64 * d->K * es);
    L.dz_tail = take(none ? (size_t)64 * d->N * es : 0);
    L.plane = take(most(none ? 0 : plane_bytes(L.up, d->M, d->N, two ? 2 : 1),
                        plane_bytes(L.dx, d->M, d->K, 1)));
    // (any number of the matrices' gradients may be wanted)
    size_t planes = 0;
    for (int k = 1; k <= (two ? 2 : 1); ++k) {
        DenseWeights w = {};
        w.M = d->M;
        w.count = k;
        for (int i = 0; i < k; ++i)
            w.m[i] = {nullptr, nullptr, nullptr, nullptr, nullptr, d->N, d->K};
        planes = most(planes, dense_weights_plan(w, d->dtype) * 4);
    }
    L.w_plane = take(planes);
    L.sums = take((size_t)dense_sum_ranges(d->M) * d->N * 4 * (two ? 2 : 1));
    L.total = take.off ? take.off : kAlign;
    return L;
}

int check_linear_weights(const moe_linear_desc *d, const moe_linear_weights *w) {
    if (!w || !w->w || (gated(d->activation) && !w->w3) || !aligned(w->w, w->b, w->w3, w->b3))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

DenseRows up_rows(int M, int N, int K, int act, const void *x, const void *w, const void *b,
                  const void *w3, const void *b3) {
    DenseRows p = {};
    p.a = x;
    p.b = w;
    p.M = M;
    p.N = N;
    p.K = K;
    p.act = act;
    p.bias = b;
    if (gated(act)) {
        p.b2 = w3;
        p.bias2 = b3;
    }
    return p;
}

// dx = add + dz W (+ du W3)
DenseRows down_rows(int M, int N, int K, const void *dz, const void *w, const void *du,
                    const void *w3, const void *add, void *dx) {
    DenseRows p = {};
    p.a = dz;
    p.b = w;
    p.a2 = du;
    p.b2 = w3;
    p.M = M;
    p.N = N;
    p.K = K;
    p.bk = true;
    p.two = du != nullptr;
    p.act = ACT_NONE;
    p.epilogue = DENSE_FORWARD;
    p.res = add;
    p.y = dx;
    return p;
}

// Adds the rows from M / 64 * 64 on of a bf16 operand of the weight
// gradients: a tensor of the caller's is copied beside zeros, one of the
// workspace (rows up to the next multiple of 64) gets zero rows.
struct Tails {
    int M;
    DenseTails &t;
    Tails(int M, DenseTails &t) : M(M), t(t) {}
    const void *of(const void *src, void *tail, int cols) {
        const int whole = M / 64 * 64;
        const char *from = (const char *)src + (size_t)whole * cols * 2;
        if (M == whole) return src;             // not read
        if (!tail) {
            t.t[t.count++] = {nullptr, (char *)src + (size_t)M * cols * 2, cols * 2, 0,
                              whole + 64 - M};
            return from;
        }
        t.t[t.count++] = {from, tail, cols * 2, M - whole, 64};
        return tail;
    }
};

int zero(void *p, size_t bytes, hipStream_t s) {
    return !p || launch_zero(p, bytes, s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_size(const moe_linear_desc *d) {
    return check_linear(d) == MOE_OK ? linear_bytes(d, linear_plan(d)) : 0;
}

int moe_linear(const moe_linear_desc *d, const void *x, const moe_linear_weights *w,
               const void *residual, void *y, void *ws, size_t ws_bytes, void *stream) {
    int st = check_linear(d);
    if (st != MOE_OK) return st;
    if (d->M == 0) return MOE_OK;
    if (!x || !y || !aligned(x, y, residual)) return MOE_ERR_INVALID_ARG;
    if ((st = check_linear_weights(d, w)) != MOE_OK) return st;
    const DensePlan plan = linear_plan(d);
    if (!ws || ws_bytes < linear_bytes(d, plan) || !aligned(ws)) return MOE_ERR_WORKSPACE;
    if (clash({y}, {x, w->w, w->b, w->w3, w->b3, residual, ws})) return MOE_ERR_INVALID_ARG;
    DenseRows p = up_rows(d->M, d->N, d->K, d->activation, x, w->w, w->b, w->w3, w->b3);
    p.epilogue = DENSE_FORWARD;
    p.res = residual;
    p.y = y;
    p.plane = (float *)ws;
    p.plan = plan;
    return to_status(launch_dense_rows(p, d->dtype, (hipStream_t)stream));
}

size_t moe_linear_grad_workspace_size(const moe_linear_desc *d) {
    return check_linear(d) == MOE_OK ? linear_layout(d).total : 0;
}

int moe_linear_grad(const moe_linear_desc *d, const void *x, const moe_linear_weights *w,
                    const void *dy, const void *dx_add, const moe_linear_grads *g, void *ws,
                    size_t ws_bytes, void *stream) {
    int st = check_linear(d);
    if (st != MOE_OK) return st;
    if (!g || !aligned(g->x, g->w, g->b, g->w3, g->b3)) return MOE_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    const bool two = gated(d->activation), none = d->activation == MOE_ACT_NONE;
    const size_t es = elem_bytes(d->dtype), mat = (size_t)d->N * d->K * es;
    if (clash({g->x, g->w, g->b, g->w3, g->b3},
              {x, dy, dx_add, ws, w ? w->w : nullptr, w ? w->b : nullptr, w ? w->w3 : nullptr,
               w ? w->b3 : nullptr}))
        return MOE_ERR_INVALID_ARG;
    LinearLayout L = {};
    if (d->M > 0) {
        if (!x || !dy || !aligned(x, dy, dx_add)) return MOE_ERR_INVALID_ARG;
        if ((st = check_linear_weights(d, w)) != MOE_OK) return st;
        L = linear_layout(d);
        if (!ws || ws_bytes < L.total || !aligned(ws)) return MOE_ERR_WORKSPACE;
    }
    // gradients of what the layer does not have, and of no rows
    if (!two || d->M == 0) {
        if ((st = zero(g->w3, mat, s)) != MOE_OK) return st;
        if ((st = zero(g->b3, d->N * es, s)) != MOE_OK) return st;
    }
    if (d->M == 0) {
        if ((st = zero(g->w, mat, s)) != MOE_OK) return st;
        return zero(g->b, d->N * es, s);
    }
    const void *dz = none ? dy : at(ws, L.dz), *du = two ? at(ws, L.du) : nullptr;
    float *plane = (float *)at(ws, L.plane);
    if (!g->x && !g->w && !g->b && !(two && (g->w3 || g->b3))) return MOE_OK;
    if (!none) {
        DenseRows p = up_rows(d->M, d->N, d->K, d->activation, x, w->w, w->b, w->w3, w->b3);
        p.epilogue = DENSE_GRAD;
        p.dy = dy;
        p.dz = (void *)dz;
        p.du = (void *)du;
        p.plane = plane;
        p.plan = L.up;
        if (launch_dense_rows(p, d->dtype, s) != hipSuccess) return MOE_ERR_HIP;
    }
    DenseBack back = {};
    if (g->x) {
        back.rows = true;
        back.dx = down_rows(d->M, d->K, d->N, dz, w->w, du, two ? w->w3 : nullptr, dx_add, g->x);
        back.dx.plane = plane;
        back.dx.plan = L.dx;
    }
    DenseSums &b = back.b;
    b.M = d->M;
    float *part = (float *)at(ws, L.sums);
    if (g->b) b.t[b.count++] = {dz, g->b, part, d->N};
    if (two && g->b3)
        b.t[b.count++] = {du, g->b3, part + (size_t)dense_sum_ranges(d->M) * d->N, d->N};
    DenseWeights &q = back.w;
    q = linear_weights(d, x, dz, du, g);
    if (q.count && d->dtype == MOE_BF16) {
        Tails tails(d->M, back.t);
        const void *xt = tails.of(x, at(ws, L.x_tail), d->K);
        for (int k = 0; k < q.count; ++k) {
            q.m[k].a2 = tails.of(q.m[k].a, none ? at(ws, L.dz_tail) : nullptr, d->N);
            q.m[k].b2 = xt;
        }
    }
    dense_weights_plan(q, d->dtype);
    q.plane = (float *)at(ws, L.w_plane);
    return to_status(launch_dense_back(back, d->dtype, s));
}

}  // extern "C"

// ------------------------------------------------------------- block

namespace {

struct DenseLayout {
    size_t h, plane, total;                       // forward
    size_t q, dz, du, x_tail, dy_tail, w_plane, sums;     // backward
    DensePlan up, down, qp, dx;
};

DenseLayout forward_layout(const moe_dense_desc *d) {
    DenseLayout L = {};
    const int panels = gated(d->activation) ? 2 : 1;
    Take take;
    L.up = dense_rows_plan(d->dtype, d->T, d->d_ff, d->d, panels, false, false);
    L.down = dense_rows_plan(d->dtype, d->T, d->d, d->d_ff, 1, false, false);
    L.h = take((size_t)d->T * d->d_ff * elem_bytes(d->dtype));
    L.plane = take(most(plane_bytes(L.up, d->T, d->d_ff, panels),
                        plane_bytes(L.down, d->T, d->d, 1)));
    L.total = take.off ? take.off : kAlign;
    return L;
}

DenseLayout backward_layout(const moe_dense_desc *d) {
    DenseLayout L = {};
    const bool two = gated(d->activation);
    const size_t es = elem_bytes(d->dtype), rows = pad64(d->T), F = d->d_ff;
    Take take;
    L.up = dense_rows_plan(d->dtype, d->T, d->d_ff, d->d, two ? 2 : 1, false, false);
    L.qp = dense_rows_plan(d->dtype, d->T, d->d_ff, d->d, 1, true, false);
    L.dx = dense_rows_plan(d->dtype, d->T, d->d, d->d_ff, 1, true, two);
    L.q = take((size_t)L.qp.splits * d->T * F * 4);
    L.h = take(rows * F * es);
    L.dz = take(rows * F * es);
    L.du = take(two ? rows * F * es : 0);
    L.x_tail = take((size_t)64 * d->d * es);
    L.dy_tail = take((size_t)64 * d->d * es);
    L.plane = take(most(plane_bytes(L.up, d->T, d->d_ff, two ? 2 : 1),
                        plane_bytes(L.dx, d->T, d->d, 1)));
    size_t planes = 0;
    // (any number of the matrices' gradients may be wanted)
    for (int k = 1; k <= (two ? 3 : 2); ++k) {
        DenseWeights w = {};
        w.M = d->T;
        w.count = k;
        for (int i = 0; i < k; ++i)
            w.m[i] = {nullptr, nullptr, nullptr, nullptr, nullptr, d->d_ff, d->d};
        planes = most(planes, dense_weights_plan(w, d->dtype) * 4);
    }
    L.w_plane = take(planes);
    L.sums = take((size_t)dense_sum_ranges(d->T) * (2 * F + d->d) * 4);
    L.total = take.off ? take.off : kAlign;
    return L;
}

int check_dense_weights(const moe_dense_desc *d, const moe_dense_weights *w) {
    if (!w || !w->w1 || !w->w2 || (gated(d->activation) && !w->w3) ||
        !aligned(w->w1, w->b1, w->w2, w->b2, w->w3, w->b3))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_dense_workspace_size(const moe_dense_desc *d) {
    return check_dense(d) == MOE_OK ? forward_layout(d).total : 0;
}

int moe_dense_forward(const moe_dense_desc *d, const void *x, const moe_dense_weights *w,
                      const void *residual, void *y, void *ws, size_t ws_bytes, void *stream) {
    int st = check_dense(d);
    if (st != MOE_OK) return st;
    if (d->T == 0) return MOE_OK;
    if (!x || !y || !aligned(x, y, residual)) return MOE_ERR_INVALID_ARG;
    if ((st = check_dense_weights(d, w)) != MOE_OK) return st;
    const DenseLayout L = forward_layout(d);
    if (!ws || ws_bytes < L.total || !aligned(ws)) return MOE_ERR_WORKSPACE;
    if (clash({y}, {x, w->w1, w->b1, w->w2, w->b2, w->w3, w->b3, residual, ws}))
        return MOE_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    DenseRows p = up_rows(d->T, d->d_ff, d->d, d->activation, x, w->w1, w->b1, w->w3, w->b3);
    p.epilogue = DENSE_FORWARD;
    p.y = at(ws, L.h);
    p.plane = (float *)at(ws, L.plane);
    p.plan = L.up;
    if (launch_dense_rows(p, d->dtype, s) != hipSuccess) return MOE_ERR_HIP;
    DenseRows q = up_rows(d->T, d->d, d->d_ff, ACT_NONE, p.y, w->w2, w->b2, nullptr, nullptr);
    q.epilogue = DENSE_FORWARD;
    q.res = residual;
    q.y = y;
    q.plane = p.plane;
    q.plan = L.down;
    return to_status(launch_dense_rows(q, d->dtype, s));
}

size_t moe_dense_grad_workspace_size(const moe_dense_desc *d) {
    return check_dense(d) == MOE_OK ? backward_layout(d).total : 0;
}

int moe_dense_backward(const moe_dense_desc *d, const void *x, const moe_dense_weights *w,
                       const void *dy, const void *dx_add, const moe_dense_grads *g, void *ws,
                       size_t ws_bytes, void *stream) {
    int st = check_dense(d);
    if (st != MOE_OK) return st;
    if (!g || !aligned(g->x, g->w1, g->b1, g->w2, g->b2, g->w3, g->b3)) return MOE_ERR_INVALID_ARG;
    if (clash({g->x, g->w1, g->b1, g->w2, g->b2, g->w3, g->b3},
              {x, dy, dx_add, ws, w ? w->w1 : nullptr, w ? w->b1 : nullptr, w ? w->w2 : nullptr,
               w ? w->b2 : nullptr, w ? w->w3 : nullptr, w ? w->b3 : nullptr}))
        return MOE_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    const bool two = gated(d->activation);
    const int T = d->T, F = d->d_ff, D = d->d, dt = d->dtype;
    const size_t es = elem_bytes(dt), mat = (size_t)F * D * es;
    DenseLayout L = {};
    if (T > 0) {
        if (!x || !dy || !aligned(x, dy, dx_add)) return MOE_ERR_INVALID_ARG;
        if ((st = check_dense_weights(d, w)) != MOE_OK) return st;
        L = backward_layout(d);
        if (!ws || ws_bytes < L.total || !aligned(ws)) return MOE_ERR_WORKSPACE;
    }
    if (!two || T == 0) {
        if ((st = zero(g->w3, mat, s)) != MOE_OK) return st;
        if ((st = zero(g->b3, F * es, s)) != MOE_OK) return st;
    }
    if (T == 0) {
        if ((st = zero(g->w1, mat, s)) != MOE_OK) return st;
        if ((st = zero(g->w2, mat, s)) != MOE_OK) return st;
        if ((st = zero(g->b1, F * es, s)) != MOE_OK) return st;
        return zero(g->b2, D * es, s);
    }
    float *plane = (float *)at(ws, L.plane);
    char *h = at(ws, L.h), *dz = at(ws, L.dz), *du = two ? at(ws, L.du) : nullptr;
    const bool w3 = two && g->w3, b3 = two && g->b3;
    if (g->x || g->w1 || g->w2 || w3 || g->b1 || b3) {
        // q = dy W2, then z (and u) again, and with q: h, dz, du
        DenseRows q = down_rows(T, F, D, dy, w->w2, nullptr, nullptr, nullptr, nullptr);
        q.epilogue = DENSE_PLANE;
        q.plane = (float *)at(ws, L.q);
        q.plan = L.qp;
        if (launch_dense_rows(q, dt, s) != hipSuccess) return MOE_ERR_HIP;
        DenseRows p = up_rows(T, F, D, d->activation, x, w->w1, w->b1, w->w3, w->b3);
        p.epilogue = DENSE_GRAD;
        p.q = q.plane;
        p.q_planes = L.qp.splits;
        p.h = g->w2 ? h : nullptr;
        p.dz = dz;
        p.du = du;
        p.plane = plane;
        p.plan = L.up;
        if (launch_dense_rows(p, dt, s) != hipSuccess) return MOE_ERR_HIP;
    }
    DenseBack back = {};
    if (g->x) {
        back.rows = true;
        back.dx = down_rows(T, D, F, dz, w->w1, du, two ? w->w3 : nullptr, dx_add, g->x);
        back.dx.plane = plane;
        back.dx.plan = L.dx;
    }
    DenseSums &b = back.b;
    b.M = T;
    float *part = (float *)at(ws, L.sums);
    const size_t ranges = dense_sum_ranges(T);
    if (g->b1) b.t[b.count++] = {dz, g->b1, part, F};
    if (b3) b.t[b.count++] = {du, g->b3, part + ranges * F, F};
    if (g->b2) b.t[b.count++] = {dy, g->b2, part + 2 * ranges * F, D};
    DenseWeights &q = back.w;
    q.M = T;
    if (g->w1) q.m[q.count++] = {dz, x, nullptr, nullptr, g->w1, F, D};
    if (w3) q.m[q.count++] = {du, x, nullptr, nullptr, g->w3, F, D};
    if (g->w2) q.m[q.count++] = {dy, h, nullptr, nullptr, g->w2, D, F};
    if (q.count && dt == MOE_BF16) {
        Tails tails(T, back.t);
        const void *xt = g->w1 || w3 ? tails.of(x, at(ws, L.x_tail), D) : nullptr;
        for (int k = 0; k < q.count; ++k) {
            DenseMat &m = q.m[k];
            const bool second = m.a == dy;
            m.a2 = tails.of(m.a, second ? at(ws, L.dy_tail) : nullptr, m.R);
            m.b2 = second ? tails.of(h, nullptr, F) : xt;
        }
    }
    dense_weights_plan(q, dt);
    q.plane = (float *)at(ws, L.w_plane);
    return to_status(launch_dense_back(back, dt, s));
}

}  // extern "C"
