// Gradient of the router.  With logits l, softmax p over all experts and
// the renormalised weights w of the k selected ones,
//   w_j = p_j / sum_S p = softmax of l over the selection S, so
//   dl_j += w_j (dw_j - sum_S w dw)                      (top-k)
//   dl_e += p_e (dp_e - sum p dp), dp_e = dw_e           (expert choice,
//                                           whose weight is p itself)
// and of the losses, the counts behind f being constants,
//   L_aux = alpha E sum_i f_i mean_t p[t,i]:  dp_e += alpha E f_e / T
//   z     = mean_t (log sum_e exp l)^2:       dl_e += 2 lse p_e / T.
// Then dx = dl Wr, dWr = dl^T x, db_router = sum_t dl.  ("MoE architecture
// deep dive", sec. 1.2-1.3 and 2.2; "AI-Research-SKILLs MoE training guide",
// sec. 4.2-4.3, give the router and its losses.)
//
// Without losses top-k routing needs no logits: dl depends on the k weights
// alone.
#include "grad.h"
#include "simt.h"

namespace {

template <typename T>
__global__ __launch_bounds__(256) void router_grad_logits(RouterGradParams p) {
    __shared__ simt::Stage st;
    const int t0 = blockIdx.x * simt::BM, e0 = blockIdx.y * simt::BN;
    float acc[4][4];
    simt::clear(acc);
    simt::product<true, true>(acc, st, (const T *)p.x + (size_t)t0 * p.d, p.d,
                              p.T - t0, (const T *)p.wr + (size_t)e0 * p.d,
                              p.d, p.E - e0, p.d);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + ty * 4 + i;
        if (t >= p.T) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = e0 + tx * 4 + j;
            if (e < p.E) {
                acc[i][j] += p.add ? p.add[e] : 0.0f;
                acc[i][j] -= p.sub ? p.sub[e] : 0.0f;
            }
        }
        simt::store4(p.logits + (size_t)t * p.ep + e0 + tx * 4, acc[i]);
    }
}

__device__ __forceinline__ float lane_f(float v, int l) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l));
}

// A wave per token, experts lane + 64 i.  Each block also leaves the column
// sums of its tokens for the bias gradient.
template <bool CHOICE>
__global__ __launch_bounds__(256) void router_grad_dlogits(RouterGradParams p) {
    constexpr int NE = MOE_MAX_E / 64;
    __shared__ float part[4][MOE_MAX_E];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool aux = p.aux != 0.0f, zl = p.z != 0.0f;
    const bool logits = zl || (aux && !CHOICE);
    float db[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) db[i] = 0.0f;
    for (int n = wave; n < MOE_ROUTER_GRAD_TOKENS; n += 4) {
        const int t = blockIdx.x * MOE_ROUTER_GRAD_TOKENS + n;
        if (t >= p.T) break;
        const size_t at = (size_t)t * p.k;
        // gradient and weight of assignment lane + 64 i
        float dw[NE], w[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int j = lane + 64 * i;
            dw[i] = w[i] = 0.0f;
            if (j < p.k) {
                w[i] = p.topk_w[at + j];
                if (p.dw) dw[i] = p.dw[at + j];
            }
        }
        if (!p.dw) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int j = lane + 64 * i;
                const int s = j < p.k ? p.slot_of[at + j] : -1;
                unsigned long long m = __ballot(s >= 0);
                while (m) {
                    const int l = __builtin_ctzll(m);
                    m &= m - 1;
                    const float *q = p.dw_part + (size_t)__builtin_amdgcn_readlane(s, l) * p.dw_tiles;
                    float sum = 0.0f;
                    for (int c = lane; c < p.dw_tiles; c += 64) sum += q[c];
                    sum = wave_sum(sum);
                    if (lane == l) dw[i] = sum;
                }
            }
        }
        float lse = 0.0f, pe[NE], dl[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) dl[i] = pe[i] = 0.0f;
        if (logits) {
            const float *q = p.logits + (size_t)t * p.ep;
            float l[NE], mx = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                l[i] = lane + 64 * i < p.E ? q[lane + 64 * i] : -INFINITY;
                mx = fmaxf(mx, l[i]);
            }
            mx = wave_max(mx);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                pe[i] = expf(l[i] - mx);
                sum += pe[i];
            }
            sum = wave_sum(sum);
            lse = mx + logf(sum);
            const float inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < NE; ++i) pe[i] *= inv;
        }
        if (CHOICE) {
#pragma unroll
            for (int i = 0; i < NE; ++i) pe[i] = w[i];
        } else {
            const float mean = wave_sum(w[0] * dw[0]);      // k <= 64
            const float v = w[0] * (dw[0] - mean);
            const int idx = lane < p.k ? p.topk_idx[at + lane] : 0;
            for (int j = 0; j < p.k; ++j) {
                const int e = __builtin_amdgcn_readlane(idx, j);
                const float vj = lane_f(v, j);
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    if (e == lane + 64 * i) dl[i] += vj;
            }
        }
        if (CHOICE || aux) {
            float dp[NE], dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 64 * i;
                dp[i] = CHOICE ? dw[i] : 0.0f;
                if (aux && e < p.E) dp[i] = fmaf(p.aux, p.f[e], dp[i]);
                dot = fmaf(pe[i], dp[i], dot);
            }
            dot = wave_sum(dot);
#pragma unroll
            for (int i = 0; i < NE; ++i) dl[i] = fmaf(pe[i], dp[i] - dot, dl[i]);
        }
        if (zl) {
            const float c = p.z * lse;
#pragma unroll
            for (int i = 0; i < NE; ++i) dl[i] = fmaf(c, pe[i], dl[i]);
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 64 * i;
            if (e < p.ep) p.dl[(size_t)t * p.ep + e] = dl[i];
            db[i] += dl[i];
        }
    }
    if (!p.db) return;
#pragma unroll
    for (int i = 0; i < NE; ++i) part[wave][lane + 64 * i] = db[i];
    __syncthreads();
    const int e = threadIdx.x;
    if (e < p.E)
        p.db_part[(size_t)blockIdx.x * p.E + e] =
            (part[0][e] + part[1][e]) + (part[2][e] + part[3][e]);
}

// db[e]: the blocks' partial sums, 64 lanes in a fixed order.
__global__ __launch_bounds__(64) void router_grad_bias(RouterGradParams p) {
    const int e = blockIdx.x;
    const int n = (p.T + MOE_ROUTER_GRAD_TOKENS - 1) / MOE_ROUTER_GRAD_TOKENS;
    float sum = 0.0f;
    for (int i = threadIdx.x; i < n; i += 64) sum += p.db_part[(size_t)i * p.E + e];
    sum = wave_sum(sum);
    if (threadIdx.x == 0) p.db[e] = sum;
}

// dx = dl Wr, plus what reaches the token through the experts: a given
// [T][d] tensor, or the fp32 row gradients of its slots in j order and of
// its shared row.
template <typename T>
__global__ __launch_bounds__(256) void router_grad_x(RouterGradParams p) {
    __shared__ simt::Stage st;
    const int t0 = blockIdx.x * simt::BM, c0 = blockIdx.y * simt::BN;
    float acc[4][4];
    simt::clear(acc);
    simt::product<true, false>(acc, st, p.dl + (size_t)t0 * p.ep, p.ep,
                               p.T - t0, (const T *)p.wr + c0, p.d, p.E, p.ep);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + ty * 4 + i;
        if (t >= p.T) continue;
        const int c = c0 + tx * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        auto add = [&](float4 q) __attribute__((always_inline)) {
            v[0] += q.x;
            v[1] += q.y;
            v[2] += q.z;
            v[3] += q.w;
        };
        if (p.dxs) {
            for (int j = 0; j < p.k; ++j) {
                const int s = p.slot_of[(size_t)t * p.k + j];
                if (s >= 0) add(simt::load4(p.dxs + (size_t)s * p.d + c));
            }
            if (p.n_shared)
                add(simt::load4(p.dxs + (size_t)(p.shared_base + t) * p.d + c));
        }
        if (p.dx_add)
            add(simt::load4((const T *)p.dx_add + (size_t)t * p.d + c));
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += acc[i][j];
        simt::store4((T *)p.dx + (size_t)t * p.d + c, v);
    }
}

// dWr over one token range (of p.splits), in fp32 or, undivided, rounded.
template <typename T>
__global__ __launch_bounds__(256) void router_grad_w(RouterGradParams p) {
    __shared__ simt::Stage st;
    const int e0 = blockIdx.x * simt::BM, c0 = blockIdx.y * simt::BN;
    const int per = (p.T + p.splits - 1) / p.splits;
    const int t0 = blockIdx.z * per;
    const int n = min(per, p.T - t0);       // may be <= 0: zeros
    float acc[4][4];
    simt::clear(acc);
    simt::product<false, false>(acc, st, p.dl + (size_t)t0 * p.ep + e0, p.ep, n,
                                (const T *)p.x + (size_t)t0 * p.d + c0, p.d, n,
                                n);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = e0 + ty * 4 + i;
        if (e >= p.E) continue;
        const size_t at = (size_t)e * p.d + c0 + tx * 4;
        if (p.splits > 1)
            simt::store4(p.wr_part + blockIdx.z * (size_t)p.E * p.d + at, acc[i]);
        else
            simt::store4((T *)p.dwr + at, acc[i]);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void router_grad_w_sum(RouterGradParams p) {
    const size_t n = (size_t)p.E * p.d;
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.splits; ++s) {
        const float4 q = simt::load4(p.wr_part + s * n + i);
        v[0] += q.x;
        v[1] += q.y;
        v[2] += q.z;
        v[3] += q.w;
    }
    simt::store4((T *)p.dwr + i, v);
}

__global__ __launch_bounds__(256) void zero_fill(uint16_t *p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n;
         i += (size_t)gridDim.x * 256)
        p[i] = 0;
}

template <typename T>
hipError_t router_grad(const RouterGradParams &p, hipStream_t s) {
    const int tt = (p.T + simt::BM - 1) / simt::BM;
    if (p.z != 0.0f || (p.aux != 0.0f && !p.choice))
        hipLaunchKernelGGL((router_grad_logits<T>), dim3(tt, p.ep / simt::BN),
                           dim3(256), 0, s, p);
    const int nb = (p.T + MOE_ROUTER_GRAD_TOKENS - 1) / MOE_ROUTER_GRAD_TOKENS;
    if (p.choice)
        hipLaunchKernelGGL((router_grad_dlogits<true>), dim3(nb), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((router_grad_dlogits<false>), dim3(nb), dim3(256), 0, s, p);
    if (p.db)
        hipLaunchKernelGGL(router_grad_bias, dim3(p.E), dim3(64), 0, s, p);
    if (p.dx)
        hipLaunchKernelGGL((router_grad_x<T>), dim3(tt, p.d / simt::BN), dim3(256), 0, s, p);
    if (p.dwr) {
        hipLaunchKernelGGL((router_grad_w<T>),
                           dim3(p.ep / simt::BM, p.d / simt::BN, p.splits),
                           dim3(256), 0, s, p);
        if (p.splits > 1)
            hipLaunchKernelGGL((router_grad_w_sum<T>),
                               dim3((unsigned)(((size_t)p.E * p.d / 4 + 255) / 256)),
                               dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace

// Enough ranges for two blocks per CU, of at least 128 tokens each.
int router_grad_splits(int T, int d, int E) {
    const long long tiles = (long long)((E + 63) / 64) * (d / simt::BN);
    long long n = (512 + tiles - 1) / tiles;
    const long long most = (T + 127) / 128;
    if (n > most) n = most;
    return (int)(n < 1 ? 1 : n);
}

hipError_t launch_router_grad(const RouterGradParams &p, int dtype,
                              hipStream_t s) {
    return dtype == 1 ? router_grad<uint16_t>(p, s) : router_grad<float>(p, s);
}

hipError_t launch_zero(void *dst, size_t n, hipStream_t s) {
    const size_t words = n / 2;
    const size_t nb = (words + 2047) / 2048;
    hipLaunchKernelGGL(zero_fill, dim3((unsigned)(nb < 4096 ? (nb ? nb : 1) : 4096)),
                       dim3(256), 0, s, (uint16_t *)dst, words);
    return hipGetLastError();
}
