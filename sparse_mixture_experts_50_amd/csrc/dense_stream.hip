// Linear layers of few rows (M <= 64), both types: the weights are streamed
// once from memory straight into MFMA fragments.
//
// A block has 16 NB columns (of each panel) and all rows; its eight waves
// split K, and their sums are added through LDS in wave order before the
// epilogue.  In the fragments' layout a lane holds 16 consecutive bytes of a
// weight row and of an x row, four lanes a run of 64 bytes of the same row.
// (fp32: the four k of a lane go to four MFMAs; which k an MFMA adds up does
// not matter as long as both operands agree.)  Rows past M re-read the last.
// Bound by HBM: two batches of loads are in flight per wave.
#include "act.h"
#include "dense.h"

namespace {

constexpr int WAVES = 8;

template <typename T>
__device__ __forceinline__ void mac(floatx4 &acc, u32x4 w, u32x4 x) {
    if constexpr (sizeof(T) == 2) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), as_bf16x8(x), acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[e]),
                                                       __uint_as_float(x[e]), acc, 0, 0, 0);
    }
}

__device__ __forceinline__ floatx4 load4(const float *p) { return *(const floatx4 *)p; }
__device__ __forceinline__ floatx4 load4(const uint16_t *p) {
    const u32x2 v = *(const u32x2 *)p;
    return floatx4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}
__device__ __forceinline__ void store4(float *p, floatx4 v) { *(floatx4 *)p = v; }
__device__ __forceinline__ void store4(uint16_t *p, floatx4 v) {
    *(u32x2 *)p = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// The epilogue of 4 columns of a row, at element `at`.
template <typename T, int EPI, int ACT>
__device__ __forceinline__ void finish(const DenseRows &p, floatx4 z, floatx4 u, size_t at) {
    constexpr bool FAST = sizeof(T) == 2;
    if (EPI == DENSE_FORWARD) {
        floatx4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = act_value<ACT, FAST>(z[e], u[e]);
        if (p.res) y += load4((const T *)p.res + at);
        store4((T *)p.y + at, y);
        return;
    }
    floatx4 q;
    if (p.dy) {
        q = load4((const T *)p.dy + at);
    } else {
        q = load4(p.q + at);
        for (int s = 1; s < p.q_planes; ++s) q += load4(p.q + (size_t)s * p.M * p.N + at);
    }
    floatx4 h, dz, du;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float v, hz, hu;
        act_grad<ACT, FAST>(z[e], u[e], v, hz, hu);
        h[e] = v;
        dz[e] = q[e] * hz;
        du[e] = q[e] * hu;
    }
    store4((T *)p.dz + at, dz);
    if (act_gated(ACT)) store4((T *)p.du + at, du);
    if (p.h) store4((T *)p.h + at, h);
}

template <typename T, int EPI, int P, int MB, int NB>
__global__ __launch_bounds__(64 * WAVES) void dense_stream(DenseRows p) {
    constexpr int E = 16 / sizeof(T);           // elements of a lane's load
    constexpr int U = P * NB + MB <= 3 ? 4 : 2; // steps of a batch
    __shared__ floatx4 red[WAVES][MB * NB * P][64];
    const int M = p.M, N = p.N, K = p.K;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, hq = lane >> 4;
    const int n0 = blockIdx.x * 16 * NB;
    const T *w[P * NB], *x[MB];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int n = 0; n < NB; ++n)
            w[i * NB + n] = (const T *)(i ? p.b2 : p.b) + (size_t)(n0 + 16 * n + l16) * K + hq * E;
#pragma unroll
    for (int m = 0; m < MB; ++m) x[m] = (const T *)p.a + (size_t)min(16 * m + l16, M - 1) * K + hq * E;
    const int steps = K / (4 * E);
    const int s0 = steps * wave / WAVES, s1 = steps * (wave + 1) / WAVES;
    floatx4 acc[MB][P * NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < P * NB; ++n) acc[m][n] = floatx4{0.f, 0.f, 0.f, 0.f};
    u32x4 wv[2][U][P * NB], xv[2][U][MB];
    // (steps from s1 on re-read the last; they are not used)
    auto load = [&](int buf, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const size_t at = (size_t)min(s + u, s1 - 1) * (4 * E);
#pragma unroll
            for (int n = 0; n < P * NB; ++n) wv[buf][u][n] = *(const u32x4 *)(w[n] + at);
#pragma unroll
            for (int m = 0; m < MB; ++m) xv[buf][u][m] = *(const u32x4 *)(x[m] + at);
        }
    };
    auto compute = [&](int buf, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int n = 0; n < P * NB; ++n) mac<T>(acc[m][n], wv[buf][u][n], xv[buf][u][m]);
        }
    };
    if (s0 < s1) {
        load(0, s0);
        for (int s = s0; s < s1; s += 2 * U) {
            if (s + U < s1) load(1, s + U);
            __builtin_amdgcn_sched_barrier(0);
            compute(0, s);
            __builtin_amdgcn_sched_barrier(0);
            if (s + U >= s1) break;
            if (s + 2 * U < s1) load(0, s + 2 * U);
            __builtin_amdgcn_sched_barrier(0);
            compute(1, s + U);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < P; ++i) red[wave][(m * NB + n) * P + i][lane] = acc[m][i * NB + n];
    __syncthreads();
    for (int b = wave; b < MB * NB; b += WAVES) {
        const int m = b / NB * 16 + l16, c = n0 + b % NB * 16 + 4 * hq;
        floatx4 z = red[0][b * P][lane], u = red[0][b * P + P - 1][lane];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) {
            z += red[v][b * P][lane];
            if (P > 1) u += red[v][b * P + P - 1][lane];
        }
        if (m >= M) continue;
        if (p.bias) z += load4((const T *)p.bias + c);
        if (P > 1 && p.bias2) u += load4((const T *)p.bias2 + c);
        const size_t at = (size_t)m * N + c;
        if (P > 1) {
            if (p.act == ACT_SWIGLU) finish<T, EPI, ACT_SWIGLU>(p, z, u, at);
            else finish<T, EPI, ACT_GEGLU>(p, z, u, at);
        } else {
            if (p.act == ACT_GELU) finish<T, EPI, ACT_GELU>(p, z, u, at);
            else if (p.act == ACT_SILU) finish<T, EPI, ACT_SILU>(p, z, u, at);
            else finish<T, EPI, ACT_NONE>(p, z, u, at);
        }
    }
}

template <typename T, int EPI, int P, int MB, int NB>
void launch(const DenseRows &p, hipStream_t s) {
    hipLaunchKernelGGL((dense_stream<T, EPI, P, MB, NB>), dim3(p.N / (16 * NB)),
                       dim3(64 * WAVES), 0, s, p);
}
template <typename T, int EPI, int P, int MB> void by_columns(const DenseRows &p, hipStream_t s) {
    if constexpr (MB * P <= 2)
        if (p.plan.nb == 4) return launch<T, EPI, P, MB, 4>(p, s);
    if constexpr (MB * P <= 4)
        if (p.plan.nb >= 2) return launch<T, EPI, P, MB, 2>(p, s);
    launch<T, EPI, P, MB, 1>(p, s);
}
template <typename T, int EPI, int P> void by_rows(const DenseRows &p, hipStream_t s) {
    if (p.M <= 16) by_columns<T, EPI, P, 1>(p, s);
    else if (p.M <= 32) by_columns<T, EPI, P, 2>(p, s);
    else by_columns<T, EPI, P, 4>(p, s);
}
template <typename T> void by_form(const DenseRows &p, hipStream_t s) {
    if (p.epilogue == DENSE_FORWARD) {
        if (p.panels() == 2) by_rows<T, DENSE_FORWARD, 2>(p, s);
        else by_rows<T, DENSE_FORWARD, 1>(p, s);
    } else {
        if (p.panels() == 2) by_rows<T, DENSE_GRAD, 2>(p, s);
        else by_rows<T, DENSE_GRAD, 1>(p, s);
    }
}

}  // namespace

hipError_t launch_dense_stream(const DenseRows &p, int dtype, hipStream_t s) {
    if (dtype == 1) by_form<uint16_t>(p, s);
    else by_form<float>(p, s);
    return hipGetLastError();
}
