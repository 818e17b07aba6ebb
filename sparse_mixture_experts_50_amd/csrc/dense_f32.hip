// The dense layer's products in single precision (tile product in
// f32_tile.h): 64 x 64 tiles, one a block, over ranges of K (the weight
// gradient: of the rows) where there are few.
#include "act.h"
#include "dense.h"
#include "f32_tile.h"

namespace {

// The block's tile: row tiles side by side, then columns, then ranges.
struct Tile {
    int m0, n0, split;
};
__device__ __forceinline__ Tile tile_at(int L, int mt, int nt) {
    Tile t;
    t.split = L / (mt * nt);
    const int local = L - t.split * (mt * nt);
    t.n0 = local / mt * f32t::BN;
    t.m0 = local % mt * f32t::BM;
    return t;
}

template <int PANELS, bool BK, bool TWO, int EPI, int ACT>
__global__ __launch_bounds__(256) void dense_rows_f32(DenseRows p) {
    __shared__ f32t::Stage st;
    const int M = p.M, N = p.N, K = p.K;
    const Tile t = tile_at(blockIdx.x, p.plan.mt, p.plan.nt);
    const int rows = min(f32t::BM, M - t.m0);
    const int k0 = t.split * p.plan.per * 64, k = min(p.plan.per * 64, K - k0);
    f32t::Acc acc[PANELS];
    auto product = [&](f32t::Acc &to, const void *a, const void *b) __attribute__((always_inline)) {
        f32t::product<true, !BK>(to, st, (const float *)a + (size_t)t.m0 * K + k0, K, rows,
                                 (const float *)b + (BK ? (size_t)k0 * N + t.n0
                                                        : (size_t)t.n0 * K + k0),
                                 BK ? N : K, BK ? k : f32t::BN, k);
    };
#pragma unroll
    for (int i = 0; i < PANELS; ++i) {
        f32t::clear(acc[i]);
        product(acc[i], p.a, i ? p.b2 : p.b);
    }
    if (TWO) product(acc[0], p.a2, p.b2);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = (wave >> 1) * 32 + 16 * i + (lane & 15);
        if (m >= rows) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = t.n0 + (wave & 1) * 32 + 16 * j + 4 * (lane >> 4);
            const size_t at = (size_t)(t.m0 + m) * N + c;
            floatx4 z = acc[0][i][j], u = acc[PANELS - 1][i][j];
            if constexpr (EPI == DENSE_PLANE) {
                float *plane = p.plane + (size_t)t.split * PANELS * M * N + at;
                *(floatx4 *)plane = z;
                if (PANELS > 1) *(floatx4 *)(plane + (size_t)M * N) = u;
                continue;
            }
            if (p.bias) z += *(const floatx4 *)((const float *)p.bias + c);
            if (PANELS > 1 && p.bias2) u += *(const floatx4 *)((const float *)p.bias2 + c);
            if constexpr (EPI == DENSE_FORWARD) {
                floatx4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = act_value<ACT, false>(z[e], u[e]);
                if (p.res) y += *(const floatx4 *)((const float *)p.res + at);
                *(floatx4 *)((float *)p.y + at) = y;
            } else {
                floatx4 q;
                if (p.dy) {
                    q = *(const floatx4 *)((const float *)p.dy + at);
                } else {
                    q = *(const floatx4 *)(p.q + at);
                    for (int s = 1; s < p.q_planes; ++s)
                        q += *(const floatx4 *)(p.q + (size_t)s * M * N + at);
                }
                floatx4 h, dz, du;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float hz, hu, v;
                    act_grad<ACT, false>(z[e], u[e], v, hz, hu);
                    h[e] = v;
                    dz[e] = q[e] * hz;
                    du[e] = q[e] * hu;
                }
                *(floatx4 *)((float *)p.dz + at) = dz;
                if (PANELS > 1) *(floatx4 *)((float *)p.du + at) = du;
                if (p.h) *(floatx4 *)((float *)p.h + at) = h;
            }
        }
    }
}

__global__ __launch_bounds__(256) void dense_weight_f32(DenseWeights p) {
    __shared__ f32t::Stage st;
    int L = blockIdx.x, i = 0;
    for (; i + 1 < p.count; ++i) {
        const int n = p.m[i].R / f32t::BM * (p.m[i].C / f32t::BN) * p.splits;
        if (L < n) break;
        L -= n;
    }
    const DenseMat &m = p.m[i];
    const Tile t = tile_at(L, m.R / f32t::BM, m.C / f32t::BN);
    const int r0 = t.split * p.per * 64, rows = min(p.per * 64, p.M - r0);
    f32t::Acc acc;
    f32t::clear(acc);
    f32t::product<false, false>(acc, st, (const float *)m.a + (size_t)r0 * m.R + t.m0, m.R, rows,
                                (const float *)m.b + (size_t)r0 * m.C + t.n0, m.C, rows, rows);
    float *out = p.splits > 1
                     ? p.plane + p.offset[i] + (size_t)t.split * m.R * m.C
                     : (float *)m.out;
    f32t::each(acc, [&](int r, int c, floatx4 v) {
        *(floatx4 *)(out + (size_t)(t.m0 + r) * m.C + t.n0 + c) = v;
    });
}

template <int PANELS, bool BK, bool TWO, int EPI, int ACT>
hipError_t launch(const DenseRows &p, hipStream_t s) {
    hipLaunchKernelGGL((dense_rows_f32<PANELS, BK, TWO, EPI, ACT>),
                       dim3(p.plan.mt * p.plan.nt * p.plan.splits), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int EPI> hipError_t by_act(const DenseRows &p, hipStream_t s) {
    switch (p.act) {
    case ACT_GELU: return launch<1, false, false, EPI, ACT_GELU>(p, s);
    case ACT_SILU: return launch<1, false, false, EPI, ACT_SILU>(p, s);
    case ACT_SWIGLU: return launch<2, false, false, EPI, ACT_SWIGLU>(p, s);
    case ACT_GEGLU: return launch<2, false, false, EPI, ACT_GEGLU>(p, s);
    default: return launch<1, false, false, EPI, ACT_NONE>(p, s);
    }
}

}  // namespace

hipError_t launch_dense_rows_f32(const DenseRows &p, hipStream_t s) {
    if (p.epilogue == DENSE_PLANE) {
        if (p.two) return launch<1, true, true, DENSE_PLANE, ACT_NONE>(p, s);
        if (p.bk) return launch<1, true, false, DENSE_PLANE, ACT_NONE>(p, s);
        return p.panels() == 2 ? launch<2, false, false, DENSE_PLANE, ACT_SWIGLU>(p, s)
                               : launch<1, false, false, DENSE_PLANE, ACT_NONE>(p, s);
    }
    if (p.two) return launch<1, true, true, DENSE_FORWARD, ACT_NONE>(p, s);
    if (p.bk) return launch<1, true, false, DENSE_FORWARD, ACT_NONE>(p, s);
    return p.epilogue == DENSE_FORWARD ? by_act<DENSE_FORWARD>(p, s) : by_act<DENSE_GRAD>(p, s);
}

hipError_t launch_dense_weights_f32(const DenseWeights &p, hipStream_t s) {
    long long tiles = 0;
    for (int k = 0; k < p.count; ++k)
        tiles += (long long)(p.m[k].R / f32t::BM) * (p.m[k].C / f32t::BN) * p.splits;
    hipLaunchKernelGGL(dense_weight_f32, dim3((unsigned)tiles), dim3(256), 0, s, p);
    return hipGetLastError();
}
