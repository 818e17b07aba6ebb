// Tokens into expert-sorted rows and back, and the gradients of both:
//   dispatch        xs[slot_of[t,j]] = x[t]                  (kept j)
//   its gradient    dx[t] = sum over kept j of dxs[slot_of[t,j]]
//   combine         y[t] = sum over kept j of w[t,j] ys[slot_of[t,j]]
//   its gradient    dys[slot_of[t,j]] = w[t,j] dy[t],
//                   dw[t,j] = <dy[t], ys[slot_of[t,j]]>      (0 if dropped)
// and, with a shared expert, row shared_base + t of weight 1.  ("MoE
// architecture deep dive", sec. 1.1 and 2.3; "AI-Research-SKILLs MoE
// training guide", sec. 3.1.)
//
// All four are bound by HBM: they read and write each row once and do at
// most two operations per element.  Every kernel walks tokens rather than
// rows, so that a token's row, which its k slots share, is read or written
// once; the k rows of a token lie in k different experts either way.  A wave
// takes one token and 1 to 4 KB of its columns: the token's slots sit one
// per lane, a ballot finds the kept ones, and readlane turns each into a
// scalar row address (no LDS, no barrier; k = E up to 256 for expert choice
// is four ballots).  Sums run in j order in fp32 and are rounded once, so
// results do not depend on scheduling; there are no atomics.
//
// Measured: dispatch of 8192 tokens of 7168 bf16 columns to 8 rows and the
// shared one (1.17 GB) 228 us, 5.2 TB/s; its gradient, 4095 x 4096, top-2
// under a capacity limit (67 MB, last-level cache) 10.4 us; combine, 1021 x
// 1984 f32, top-5 and the shared row (57 MB) 10.0 us; its gradient, 4096 x
// 4096, top-2 (168 MB) 34 us, 4.9 TB/s.  A copy of 4 GB reaches 4.7 TB/s.
#include "grad.h"

namespace {

constexpr int WAVES = 4;              // waves per block

template <typename T> struct Vec;     // 16 bytes of a row
template <> struct Vec<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(u32x4 q, float *v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(q[i]);
            v[2 * i + 1] = bf16_hi(q[i]);
        }
    }
    static __device__ __forceinline__ u32x4 put(const float *v) {
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        return q;
    }
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(u32x4 q, float *v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(q[i]);
    }
    static __device__ __forceinline__ u32x4 put(const float *v) {
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(v[i]);
        return q;
    }
};

__device__ __forceinline__ float lane_f(float v, int l) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l));
}

// Calls body(slot, weight, j) for the token's kept assignments, j ascending.
// W: whether the weights are needed.  PAD: slots of the padded space, which
// are also kept in pad_slot (by one wave of the token's: keep).
template <bool W, bool PAD = false, typename F>
__device__ __forceinline__ void each_kept(const RowsParams &p, int t, int lane,
                                          F body, bool keep = false) {
    const int32_t *so = p.slot_of + (size_t)t * p.k;
    const float *tw = W ? p.topk_w + (size_t)t * p.k : nullptr;
    for (int j0 = 0; j0 < p.k; j0 += 64) {
        const int j = j0 + lane;
        int s = j < p.k ? so[j] : -1;
        const float w = W && j < p.k ? tw[j] : 0.0f;
        if (PAD && j < p.k) {
            const int e = p.topk_idx ? p.topk_idx[(size_t)t * p.k + j] : j;
            if (s >= 0) s += p.pad[e] - p.offsets[e];
            if (keep) p.pad_slot[(size_t)t * p.k + j] = s;
        }
        unsigned long long m = __ballot(s >= 0);
        while (m) {
            const int l = __builtin_ctzll(m);
            m &= m - 1;
            body(__builtin_amdgcn_readlane(s, l), W ? lane_f(w, l) : 1.0f, j0 + l);
        }
    }
}

// Wave -> (token, first vector of its columns); false past the end.
template <int S>
__device__ __forceinline__ bool wave_span(const RowsParams &p, int nv, int &t,
                                          int &v0) {
    const int per = (nv + 64 * S - 1) / (64 * S);       // waves per token
    const long long w = (long long)blockIdx.x * WAVES + (threadIdx.x >> 6);
    t = __builtin_amdgcn_readfirstlane((int)(w / per));
    v0 = __builtin_amdgcn_readfirstlane((int)(w % per)) * 64 * S;
    return t < p.T;
}

// TWO: x and dy into the gradient's padded row space, with the row weights.
template <typename T, int S, bool TWO>
__global__ __launch_bounds__(WAVES * 64) void dispatch_rows(RowsParams p) {
    const int lane = threadIdx.x & 63;
    const int nv = p.d / Vec<T>::N;
    int t, v0;
    if (!wave_span<S>(p, nv, t, v0)) return;
    const u32x4 *a = (const u32x4 *)p.tok + (size_t)t * nv;
    const u32x4 *b = TWO ? (const u32x4 *)p.tok2 + (size_t)t * nv : nullptr;
    u32x4 qa[S], qb[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int v = v0 + i * 64 + lane;
        if (v < nv) {
            qa[i] = a[v];
            if (TWO) qb[i] = b[v];
        }
    }
    auto write = [&](int row, float w) __attribute__((always_inline)) {
        u32x4 *o = (u32x4 *)p.rows_out + (size_t)row * nv;
        u32x4 *o2 = TWO ? (u32x4 *)p.rows_out2 + (size_t)row * nv : nullptr;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int v = v0 + i * 64 + lane;
            if (v < nv) {
                o[v] = qa[i];
                if (TWO) o2[v] = qb[i];
            }
        }
        if (TWO && v0 == 0 && lane == 0) p.row_w[row] = w;
    };
    each_kept<TWO, TWO>(p, t, lane, [&](int s, float w, int) { write(s, w); }, v0 == 0);
    if (p.n_shared) write(p.shared_base + t, 1.0f);
}

// Rows come in pairs: two rows' loads are in flight per wave (and 8 to 32
// waves per CU), summed in j order.
template <typename T, int S, bool W>
__global__ __launch_bounds__(WAVES * 64) void sum_rows(RowsParams p) {
    constexpr int N = Vec<T>::N;
    const int lane = threadIdx.x & 63;
    const int nv = p.d / N;
    int t, v0;
    if (!wave_span<S>(p, nv, t, v0)) return;
    const u32x4 *in = (const u32x4 *)p.rows_in;
    float acc[S][N];
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) acc[i][e] = 0.0f;
    auto load = [&](int row, u32x4 (&q)[S]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int v = v0 + i * 64 + lane;
            q[i] = in[(size_t)row * nv + (v < nv ? v : nv - 1)];
        }
    };
    auto add = [&](float w, const u32x4 (&q)[S]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
            float f[N];
            Vec<T>::get(q[i], f);
#pragma unroll
            for (int e = 0; e < N; ++e)
                acc[i][e] = W ? fmaf(w, f[e], acc[i][e]) : acc[i][e] + f[e];
        }
    };
    int prev = -1;
    float pw = 0.0f;
    each_kept<W>(p, t, lane, [&](int s, float w, int) __attribute__((always_inline)) {
        if (prev < 0) {
            prev = s;
            pw = w;
            return;
        }
        u32x4 qa[S], qb[S];
        load(prev, qa);
        load(s, qb);
        add(pw, qa);
        add(w, qb);
        prev = -1;
    });
    if (prev >= 0) {
        u32x4 q[S];
        load(prev, q);
        add(pw, q);
    }
    if (p.n_shared) {
        u32x4 q[S];
        load(p.shared_base + t, q);
        add(1.0f, q);
    }
    u32x4 *out = (u32x4 *)p.tok_out + (size_t)t * nv;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int v = v0 + i * 64 + lane;
        if (v < nv) out[v] = Vec<T>::put(acc[i]);
    }
}

// One block per token, its waves side by side on the columns; a wave's
// part of each dot product goes to LDS and the block adds the parts in
// wave order.  Rows wider than the block's reach take several passes.
template <typename T, int S>
__global__ __launch_bounds__(WAVES * 64) void combine_rows_grad(RowsParams p) {
    constexpr int N = Vec<T>::N;
    __shared__ float part[WAVES][MOE_MAX_E];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int nv = p.d / N, t = blockIdx.x;
    for (int j = lane; j < p.k; j += 64) part[wave][j] = 0.0f;
    const u32x4 *dy = (const u32x4 *)p.tok + (size_t)t * nv;
    for (int v0 = wave * 64 * S; v0 < nv; v0 += waves * 64 * S) {
        u32x4 q[S];
        float g[S][N];
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int v = v0 + i * 64 + lane;
            q[i] = u32x4{0, 0, 0, 0};
            if (v < nv) q[i] = dy[v];
            Vec<T>::get(q[i], g[i]);
        }
        each_kept<true>(p, t, lane, [&](int s, float w, int j) __attribute__((always_inline)) {
            const u32x4 *ys = (const u32x4 *)p.rows_in + (size_t)s * nv;
            u32x4 *o = (u32x4 *)p.rows_out + (size_t)s * nv;
            u32x4 y[S];
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const int v = v0 + i * 64 + lane;
                y[i] = u32x4{0, 0, 0, 0};
                if (v < nv) y[i] = ys[v];
            }
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const int v = v0 + i * 64 + lane;
                float f[N], b[N];
                Vec<T>::get(y[i], f);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    dot = fmaf(g[i][e], f[e], dot);
                    b[e] = w * g[i][e];
                }
                if (v < nv) o[v] = Vec<T>::put(b);
            }
            dot = wave_sum(dot);
            if (lane == 0) part[wave][j] += dot;
        });
        if (p.n_shared) {
            u32x4 *o = (u32x4 *)p.rows_out + (size_t)(p.shared_base + t) * nv;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const int v = v0 + i * 64 + lane;
                if (v < nv) o[v] = q[i];
            }
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < p.k; j += blockDim.x) {
        float sum = part[0][j];
        for (int w = 1; w < waves; ++w) sum += part[w][j];
        p.dw[(size_t)t * p.k + j] = sum;
    }
}

// 16-byte vectors per lane: 1 while that leaves the chip short of waves
// (fewer than 8 per SIMD), then 2 and 4.
int span(const RowsParams &p, int nv) {
    const long long waves = (long long)p.T * ((nv + 63) / 64);
    return waves <= 8192 ? 1 : waves <= 32768 || nv <= 128 ? 2 : 4;
}

int grid_of(const RowsParams &p, int nv, int S) {
    const long long per = (nv + 64 * S - 1) / (64 * S);
    return (int)((p.T * per + WAVES - 1) / WAVES);
}

template <typename T, int S>
void dispatch_as(const RowsParams &p, int grid, hipStream_t s) {
    if (p.tok2)
        hipLaunchKernelGGL((dispatch_rows<T, S, true>), dim3(grid), dim3(WAVES * 64), 0, s, p);
    else
        hipLaunchKernelGGL((dispatch_rows<T, S, false>), dim3(grid), dim3(WAVES * 64), 0, s, p);
}
template <typename T>
void dispatch_type(const RowsParams &p, hipStream_t s) {
    const int nv = p.d / Vec<T>::N, S = span(p, nv), grid = grid_of(p, nv, S);
    if (S == 1) dispatch_as<T, 1>(p, grid, s);
    else if (S == 2) dispatch_as<T, 2>(p, grid, s);
    else dispatch_as<T, 4>(p, grid, s);
}

template <typename T, bool W>
void sum_type(const RowsParams &p, hipStream_t s) {
    const int nv = p.d / Vec<T>::N, S = span(p, nv), grid = grid_of(p, nv, S);
    if (S == 1)
        hipLaunchKernelGGL((sum_rows<T, 1, W>), dim3(grid), dim3(WAVES * 64), 0, s, p);
    else if (S == 2)
        hipLaunchKernelGGL((sum_rows<T, 2, W>), dim3(grid), dim3(WAVES * 64), 0, s, p);
    else
        hipLaunchKernelGGL((sum_rows<T, 4, W>), dim3(grid), dim3(WAVES * 64), 0, s, p);
}

template <typename T>
void combine_grad_type(const RowsParams &p, hipStream_t s) {
    const int nv = p.d / Vec<T>::N;
    const int S = nv <= 256 ? 1 : 2;
    int waves = (nv + 64 * S - 1) / (64 * S);
    if (waves > WAVES) waves = WAVES;
    if (S == 1)
        hipLaunchKernelGGL((combine_rows_grad<T, 1>), dim3(p.T), dim3(waves * 64), 0, s, p);
    else
        hipLaunchKernelGGL((combine_rows_grad<T, 2>), dim3(p.T), dim3(waves * 64), 0, s, p);
}

}  // namespace

hipError_t launch_dispatch_rows(const RowsParams &p, int dtype, hipStream_t s) {
    if (dtype == 1) dispatch_type<uint16_t>(p, s);
    else dispatch_type<float>(p, s);
    return hipGetLastError();
}

hipError_t launch_sum_rows(const RowsParams &p, int dtype, bool weighted,
                           hipStream_t s) {
    if (dtype == 1) {
        if (weighted) sum_type<uint16_t, true>(p, s);
        else sum_type<uint16_t, false>(p, s);
    } else {
        if (weighted) sum_type<float, true>(p, s);
        else sum_type<float, false>(p, s);
    }
    return hipGetLastError();
}

hipError_t launch_combine_rows_grad(const RowsParams &p, int dtype,
                                    hipStream_t s) {
    if (dtype == 1) combine_grad_type<uint16_t>(p, s);
    else combine_grad_type<float>(p, s);
    return hipGetLastError();
}
