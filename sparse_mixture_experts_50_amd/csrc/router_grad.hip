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
//
// Measured, 8192 tokens of 7168 columns, 256 experts, top-8, both losses (30
// GFLOP in the logits, twice that in dx and in dWr, whose dl has two parts):
// logits 47 us, dl 18, dx 77, dWr 60 and its sum 10.  With the experts' part
// dx is bound by HBM: 4096 tokens of 4096 with two fp32 rows each 67 us (of
// 2048 with six, 79 us).
#include "grad.h"
#include "kernels.h"
#include "f32_tile.h"
#include "mfma_tile.h"

namespace {

__global__ __launch_bounds__(256) void router_grad_logits_f32(RouterGradParams p) {
    __shared__ f32t::Stage st;
    const int t0 = blockIdx.x * f32t::BM, e0 = blockIdx.y * f32t::BN;
    f32t::Acc acc;
    f32t::clear(acc);
    f32t::product<true, true>(acc, st, (const float *)p.x + (size_t)t0 * p.d, p.d,
                              p.T - t0, (const float *)p.wr + (size_t)e0 * p.d, p.d,
                              p.E - e0, p.d);
    f32t::each(acc, [&](int m, int c, floatx4 v) {
        if (t0 + m >= p.T) return;
        for (int e = 0; e < 4; ++e)
            if (e0 + c + e < p.E)
                p.logits[(size_t)(t0 + m) * p.E + e0 + c + e] = v[e];
    });
}

__device__ __forceinline__ float lane_f(float v, int l) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l));
}

// dl of token t and expert e.  bf16: as the sum of two bf16 parts (2^-16), [T]
// [ep / 64][2][64], the second part what the first one's rounding leaves, and
// both are multiplied.  A single part would put an error of half a bf16 step
// of every token and expert into dx and dWr beside the rounding of their
// results, which with few experts a token nothing averages out.  (The sizes
// above with a single part: dx 52 us, dWr 55.)
__device__ __forceinline__ void store_dl(float *dl, const RouterGradParams &p, int t, int e,
                                         float v) {
    dl[(size_t)t * p.ep + e] = v;
}
__device__ __forceinline__ void store_dl(uint16_t *dl, const RouterGradParams &p, int t, int e,
                                         float v) {
    const uint16_t hi = (uint16_t)f32_to_bf16_bits(v);
    uint16_t *at = dl + (size_t)t * p.ep * 2 + (e >> 6) * 128 + (e & 63);
    at[0] = hi;
    const float left = v - bf16_lo(hi);         // (not a number if v is infinite)
    at[64] = (uint16_t)f32_to_bf16_bits(left == left ? left : 0.0f);
}

// A wave per token, experts lane + 64 i.  Each block also leaves the column
// sums of its tokens for the bias gradient (of dl in fp32).  A token per wave: the kernel
// waits for a few dependent loads and reductions a token.
template <typename T, bool CHOICE>
__global__ __launch_bounds__(1024) void router_grad_dlogits(RouterGradParams p) {
    constexpr int NE = MOE_MAX_E / 64, WAVES = 16;
    __shared__ float part[WAVES][MOE_MAX_E];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool aux = p.aux != 0.0f, zl = p.z != 0.0f;
    const bool logits = zl || (aux && !CHOICE);
    float db[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) db[i] = 0.0f;
    for (int n = wave; n < MOE_ROUTER_GRAD_TOKENS; n += WAVES) {
        const int t = blockIdx.x * MOE_ROUTER_GRAD_TOKENS + n;
        if (t >= p.T) break;
        const size_t at = (size_t)t * p.k;
        // the token's logits, summed over the depth ranges
        float l[NE];
        if (logits) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 64 * i;
                l[i] = -INFINITY;
                if (e < p.E) {
                    const float *q = p.logits + (size_t)t * p.E + e;
                    const size_t plane = (size_t)p.T * p.E;
                    // every load issued before the in-order sum
                    float part[MOE_ROUTER_MAX_SPLITS];
#pragma unroll
                    for (int s = 0; s < MOE_ROUTER_MAX_SPLITS; ++s)
                        part[s] = s < p.logit_splits ? q[s * plane] : 0.0f;
                    float a = part[0];
#pragma unroll
                    for (int s = 1; s < MOE_ROUTER_MAX_SPLITS; ++s)
                        if (s < p.logit_splits) a += part[s];
                    if (p.add) a += p.add[e];
                    if (p.sub) a -= p.sub[e];
                    l[i] = a;
                }
            }
        }
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
            // four rows' partial sums in flight
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int j = lane + 64 * i;
                const int s = j < p.k ? p.slot_of[at + j] : -1;
                unsigned long long m = __ballot(s >= 0);
                while (m) {
                    int who[4];
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    const float *q[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        who[u] = m ? __builtin_ctzll(m) : who[0];
                        m &= m - 1;
                        q[u] = p.dw_part +
                               (size_t)__builtin_amdgcn_readlane(s, who[u]) * p.dw_tiles;
                    }
                    for (int c = lane; c < p.dw_tiles; c += 64) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) sum[u] += q[u][c];
                    }
#pragma unroll
                    for (int u = 3; u >= 0; --u) {
                        const float v = wave_sum(sum[u]);
                        if (lane == who[u]) dw[i] = v;
                    }
                }
            }
        }
        float lse = 0.0f, pe[NE], dl[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) dl[i] = pe[i] = 0.0f;
        if (logits) {
            float mx = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NE; ++i) mx = fmaxf(mx, l[i]);
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
            if (e < p.ep) store_dl((T *)p.dl, p, t, e, dl[i]);
            db[i] += dl[i];
        }
    }
    if (!p.db) return;
#pragma unroll
    for (int i = 0; i < NE; ++i) part[wave][lane + 64 * i] = db[i];
    __syncthreads();
    const int e = threadIdx.x;
    if (e >= p.E) return;
    float sum = part[0][e];
    for (int i = 1; i < WAVES; ++i) sum += part[i][e];
    p.db_part[(size_t)blockIdx.x * p.E + e] = sum;
}

// db[e]: the blocks' partial sums, the 64 lanes of a wave in a fixed order.
__device__ __forceinline__ void bias_sum(const RouterGradParams &p, int e) {
    if (e >= p.E) return;
    const int lane = threadIdx.x & 63;
    const int n = (p.T + MOE_ROUTER_GRAD_TOKENS - 1) / MOE_ROUTER_GRAD_TOKENS;
    float sum = 0.0f;
    for (int i = lane; i < n; i += 64) sum += p.db_part[(size_t)i * p.E + e];
    sum = wave_sum(sum);
    if (lane == 0) p.db[e] = sum;
}
__global__ __launch_bounds__(256) void router_grad_bias(RouterGradParams p) {
    bias_sum(p, blockIdx.x * 4 + (threadIdx.x >> 6));
}

__device__ __forceinline__ floatx4 load4(const float *p) { return *(const floatx4 *)p; }
__device__ __forceinline__ floatx4 load4(const uint16_t *p) {
    const u32x2 q = *(const u32x2 *)p;
    return floatx4{bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
}
__device__ __forceinline__ void store4(float *p, floatx4 v) { *(floatx4 *)p = v; }
__device__ __forceinline__ void store4(uint16_t *p, floatx4 v) {
    u32x2 q;
    q.x = pack_bf16x2(v[0], v[1]);
    q.y = pack_bf16x2(v[2], v[3]);
    *(u32x2 *)p = q;
}

// What reaches token t through the experts, NB runs of 4 columns, 16
// columns apart from c on: the fp32 row gradients of its slots in j order
// and of its shared row, or a given [T][d] tensor.
template <typename T, int NB>
__device__ __forceinline__ void expert_part(const RouterGradParams &p, int t, int c,
                                            floatx4 (&v)[NB]) {
#pragma unroll
    for (int b = 0; b < NB; ++b) v[b] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (p.dxs) {
        const int32_t *so = p.slot_of + (size_t)t * p.k;
        // four rows in flight: a slot that has none re-reads the first one
        // that has, and drops it
        auto add4 = [&](const int (&s)[4]) __attribute__((always_inline)) {
            const int any = max(max(s[0], s[1]), max(s[2], s[3]));
            if (any < 0) return;
            const float *q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                q[u] = p.dxs + (size_t)(s[u] < 0 ? any : s[u]) * p.d + c;
            for (int i = 0; i < p.dx_splits; ++i) {
                floatx4 x[4][NB];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int b = 0; b < NB; ++b) x[u][b] = load4(q[u] + 16 * b);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    q[u] += p.dx_plane;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        if (s[u] >= 0) v[b] += x[u][b];
                }
            }
        };
        for (int j = 0; j < p.k; j += 4) {
            int s[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] = j + u < p.k ? so[j + u] : -1;
            add4(s);
        }
        if (p.n_shared) {
            const int s[4] = {p.shared_base + t, -1, -1, -1};
            add4(s);
        }
    }
    if (p.dx_add) {
        const T *q = (const T *)p.dx_add + (size_t)t * p.d + c;
#pragma unroll
        for (int b = 0; b < NB; ++b) v[b] += load4(q + 16 * b);
    }
}

// dx = dl Wr + what comes through the experts, 64 tokens x 64 columns.
__global__ __launch_bounds__(256) void router_grad_x_f32(RouterGradParams p) {
    __shared__ f32t::Stage st;
    const int t0 = blockIdx.x * f32t::BM, c0 = blockIdx.y * f32t::BN;
    f32t::Acc acc;
    f32t::clear(acc);
    f32t::product<true, false>(acc, st, (const float *)p.dl + (size_t)t0 * p.ep, p.ep,
                               p.T - t0, (const float *)p.wr + c0, p.d, p.E, p.ep);
    f32t::each(acc, [&](int m, int c, floatx4 a) {
        if (t0 + m >= p.T) return;
        floatx4 v[1];
        expert_part<float, 1>(p, t0 + m, c0 + c, v);
        store4((float *)p.dx + (size_t)(t0 + m) * p.d + c0 + c, v[0] + a);
    });
}

// The same for bf16 layers, 16 tokens per wave: dl's fragments straight from
// memory, the router rows of the 64 columns staged in LDS (zeros past E) and
// transposed on the way to the MFMAs.  The rows of dx through the experts,
// k fp32 rows a token, are what takes its time.
template <int KS, bool ROWS>                  // KS 64-deep stages: ep / 64
__global__ __launch_bounds__(256) void router_grad_x_bf16(RouterGradParams p) {
    typedef mt::Loader<true, 64, 1, 0> LB;
    __shared__ u32x4 slot[KS * LB::UNITS];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t0 = blockIdx.x * 64 + wave * 16, c0 = blockIdx.y * 64;
    LB lb;
    mt::Reader<true, 64, 0, 4> b;
    b.init(0, lane);
    // (rows past E, where dl is zero: the router's first again)
    {
        const uint64_t wr = (uint64_t)((const uint16_t *)p.wr + c0);
        lb.init(p.d * 2, 64, wave, lane);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int q = 0; q < LB::LOADS; ++q) {
                const int e = s * 64 + (wave * 64 + lane) / 8 + 32 * q;
                const uint32_t back = e < p.E ? 0 : (uint32_t)e * (uint32_t)p.d * 2;
                mt::dma16(wr, lb.at(q) + (uint32_t)s * 128u * (uint32_t)p.d - back,
                          slot + s * LB::UNITS + (q * 4 + wave) * 64);
            }
    }
    const int t = t0 + (lane & 15);
    const uint16_t *dl = (const uint16_t *)p.dl + (size_t)min(t, p.T - 1) * p.ep * 2 +
                         8 * (lane >> 4);
    bf16x8 fa[2][2 * KS];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 2 * KS; ++k)
            fa[h][k] = as_bf16x8(*(const u32x4 *)(dl + 64 * ((k >> 1) * 2 + h) + 32 * (k & 1)));
    const int c = c0 + 4 * (lane >> 4);
    floatx4 v[4];
    if (ROWS) expert_part<uint16_t, 4>(p, min(t, p.T - 1), c, v);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    floatx4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2 * KS; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bf16x8 fb = {};
            b.read(fb, slot + (k >> 1) * LB::UNITS, k & 1, j, 0, 0);
            b.read(fb, slot + (k >> 1) * LB::UNITS, k & 1, j, 0, 1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb, fa[h][k], acc[j], 0, 0, 0);
        }
    if (t >= p.T) return;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        store4((uint16_t *)p.dx + (size_t)t * p.d + c + 16 * j, ROWS ? v[j] + acc[j] : acc[j]);
}

// dx without the experts' part in 256 x 256 tiles: the sum of two products of
// K = E, of dl's two parts (every second block of 64 columns each).
__global__ __launch_bounds__(256) void router_grad_x_tiles(RouterGradParams p) {
    typedef mt::Tiles<256, 256, 2, 2, 1, false, true, true> P;
    constexpr int RB = 8, TN = P::TN;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE], scr[4 * 32 * TN];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mtiles = (p.T + 255) / 256, total = mtiles * ((p.d + 255) / 256);
    auto place = [&](int L, int &t0, int &c0) __attribute__((always_inline)) {
        const int ni = L / mtiles;
        t0 = mt::tile_start(L - ni * mtiles, 256, p.T);
        c0 = mt::tile_start(ni, 256, p.d);
    };
    auto source = [&](int t0, int c0) __attribute__((always_inline)) {
        typename P::Source s;
        s.a = (uint64_t)((const uint16_t *)p.dl + (size_t)t0 * p.ep * 2);
        s.a2 = s.a + mt::SK * 2;
        s.b = s.b2 = (uint64_t)((const uint16_t *)p.wr + c0);
        s.kt = p.ep / mt::SK * 2;
        s.s0 = 0;
        return s;
    };
    int L = mt::tile_of(0);
    if (L >= total) return;
    typename P::Lanes ln;
    ln.init(p.ep * 4, 256, p.d * 2, 256, wave, threadIdx.x & 63);
    ln.step_a = mt::SK * 4;
    ln.split = p.ep / mt::SK;
    int t0, c0;
    place(L, t0, c0);
    typename P::Source src = source(t0, c0);
    P::load_stage(src, ln, 0, slot0, wave);
    P::load_stage(src, ln, 1, slot1, wave);
    mt::wait_loads<0>();
    for (int r = 1;; ++r) {
        const int lane = mt::tile_lane();
        L = mt::tile_of(r);
        const bool more = L < total;
        int tn = t0, cn = c0;
        if (more) place(L, tn, cn);
        const typename P::Source next = source(tn, cn);
        floatx4 acc[RB][TN];
        mt::clear(acc);
        P::template run<RB, RB, mt::EVEN>(acc, src, ln, next, ln, slot0, slot1, wave, lane);
        uint16_t *out = (uint16_t *)p.dx + (size_t)(t0 + wave / 2 * RB * 16) * p.d + c0 +
                        wave % 2 * TN * 16;
        mt::RowStore<TN> rows[2];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            float v[TN][4];
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j][e] = acc[i][j][e];
            rows[i & 1].turn(scr, wave * 32 * TN, v, lane);
            if (i > 0) rows[(i - 1) & 1].store(out + (size_t)(i - 1) * 16 * p.d, p.d, lane);
            if (i == RB - 1) rows[i & 1].store(out + (size_t)i * 16 * p.d, p.d, lane);
            __builtin_amdgcn_sched_barrier(0);
        }
        // the next tile's loads, ahead of the stores, have landed
        mt::wait_loads<RB * TN / 2>();
        if (!more) break;
        t0 = tn;
        c0 = cn;
        src = next;
    }
    __builtin_amdgcn_s_waitcnt(0);
}

// dWr over one token range (of p.splits), in fp32 or, undivided, rounded.
__global__ __launch_bounds__(256) void router_grad_w_f32(RouterGradParams p) {
    __shared__ f32t::Stage st;
    const int e0 = blockIdx.x * f32t::BM, c0 = blockIdx.y * f32t::BN;
    const int per = (p.T + p.splits - 1) / p.splits;
    const int t0 = blockIdx.z * per;
    const int n = min(per, p.T - t0);       // may be <= 0: zeros
    f32t::Acc acc;
    f32t::clear(acc);
    f32t::product<false, false>(acc, st, (const float *)p.dl + (size_t)t0 * p.ep + e0,
                                p.ep, n, (const float *)p.x + (size_t)t0 * p.d + c0,
                                p.d, n, n);
    float *out = p.splits > 1 ? p.wr_part + blockIdx.z * (size_t)p.E * p.d
                              : (float *)p.dwr;
    f32t::each(acc, [&](int m, int c, floatx4 v) {
        if (e0 + m < p.E) store4(out + (size_t)(e0 + m) * p.d + c0 + c, v);
    });
}

static __device__ __align__(1024) const char zero_line[1024] = {};

// EXPERTS (64 or 128, see dw_wide) x 256 columns on the matrix cores, both
// operands along tokens, dl's two parts side by side: of each wave's row
// blocks the first half are the first parts of 64 experts, the others the
// second parts of the same, added at the end.  With 128 experts and E = 256
// every column of x is read by two tiles instead of four.
template <int EXPERTS>
__global__ __launch_bounds__(256) void router_grad_w_bf16(RouterGradParams p) {
    constexpr int BM = 2 * EXPERTS, WM = BM / 128, WN = 4 / WM, RB = 8;
    typedef mt::Tiles<BM, 256, WM, WN, 1, true, true> P;
    constexpr int TN = P::TN, LOADS = BM / 32;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e0 = blockIdx.x * EXPERTS, c0 = blockIdx.y * 256;
    const int lda = p.ep * 2, a0 = e0 * 2;
    const int per = (p.T + p.splits - 1) / p.splits;
    const int t0 = blockIdx.z * per;
    const int n = max(0, min(per, p.T - t0));       // may be 0: zeros
    // stage 0 holds what the whole stages of 64 tokens leave over
    const int over = n % mt::SK, head = over ? over : min(n, mt::SK);
    const uint16_t *A = (const uint16_t *)p.dl + (size_t)t0 * lda + a0;
    const uint16_t *B = (const uint16_t *)p.x + (size_t)t0 * p.d + c0;
    typename P::Source src;
    src.a = src.a2 = (uint64_t)A + ((int64_t)head - mt::SK) * lda * 2;
    src.b = src.b2 = (uint64_t)B + ((int64_t)head - mt::SK) * p.d * 2;
    src.kt = (n + mt::SK - 1) / mt::SK;
    src.s0 = 0;
    typename P::Lanes ln;
    ln.init(lda * 2, min(BM, lda - a0), p.d * 2, min(256, p.d - c0), wave, lane);
    ln.split = 0;
    auto head_load = [&](const void *base, uint32_t off, int k, u32x4 *to) __attribute__((always_inline)) {
        const char *from = (const char *)base + off;
        if (k >= head) from = zero_line + lane * 16;
        mt::dma16_lanes(from, to);
    };
#pragma unroll
    for (int q = 0; q < LOADS; ++q)
        head_load(A, ln.a.at(q), (wave * 64 + lane) / (BM / 8) + 256 / (BM / 8) * q,
                  slot0 + (q * 4 + wave) * 64);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        head_load(B, ln.b.at(q), (wave * 64 + lane) / 32 + 8 * q,
                  slot0 + (P::LA::UNITS + (q * 4 + wave) * 64));
    // no stage after the last: every lane a zeroed line (x may end anywhere)
    typename P::Source none;
    none.a = none.a2 = none.b = none.b2 = (uint64_t)zero_line;
    none.kt = none.s0 = 0;
    typename P::Lanes still = {};
    if (src.kt > 1) P::load_stage(src, ln, 1, slot1, wave);
    else P::load_stage(none, still, 1, slot1, wave);
    mt::wait_loads<0>();
    const int wm = wave / WN, wn = wave % WN;
    const int c = c0 + wn * TN * 16 + 4 * (lane >> 4);
    P::by_stages(src.kt, [&](auto kind) __attribute__((always_inline)) {
        floatx4 acc[RB][TN];
        mt::clear(acc);
        P::template run<RB, LOADS, decltype(kind)::value>(acc, src, ln, none, still, slot0,
                                                         slot1, wave, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + (wm * 4 + i) * 16 + (lane & 15);
            if (e >= p.E) continue;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                if (c + 16 * j >= p.d) continue;
                const size_t at = (size_t)e * p.d + c + 16 * j;
                const floatx4 v = acc[i][j] + acc[4 + i][j];
                if (p.splits > 1)
                    store4(p.wr_part + blockIdx.z * (size_t)p.E * p.d + at, v);
                else
                    store4((uint16_t *)p.dwr + at, v);
            }
        }
    });
    __builtin_amdgcn_s_waitcnt(0);
}

// dWr of the token ranges added up in `blocks` blocks, db in the others.
template <typename T>
__global__ __launch_bounds__(256) void router_grad_w_sum(RouterGradParams p, int blocks) {
    if ((int)blockIdx.x >= blocks) {
        bias_sum(p, (blockIdx.x - blocks) * 4 + (threadIdx.x >> 6));
        return;
    }
    const size_t n = (size_t)p.E * p.d;
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    floatx4 v = load4(p.wr_part + i);
#pragma unroll 4
    for (int s = 1; s < p.splits; ++s) v += load4(p.wr_part + s * n + i);
    store4((T *)p.dwr + i, v);
}

__global__ __launch_bounds__(256) void zero_fill(uint16_t *p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n;
         i += (size_t)gridDim.x * 256)
        p[i] = 0;
}

// Whether dWr's token ranges are added up by a kernel, which then does db too.
bool sums_w(const RouterGradParams &p) { return p.dwr && p.splits > 1; }

template <typename T> void dlogits(const RouterGradParams &p, hipStream_t s) {
    const int nb = (p.T + MOE_ROUTER_GRAD_TOKENS - 1) / MOE_ROUTER_GRAD_TOKENS;
    if (p.choice)
        hipLaunchKernelGGL((router_grad_dlogits<T, true>), dim3(nb), dim3(1024), 0, s, p);
    else
        hipLaunchKernelGGL((router_grad_dlogits<T, false>), dim3(nb), dim3(1024), 0, s, p);
    if (p.db && !sums_w(p))
        hipLaunchKernelGGL(router_grad_bias, dim3((p.E + 3) / 4), dim3(256), 0, s, p);
}

template <typename T> void sum_splits(const RouterGradParams &p, hipStream_t s) {
    if (!sums_w(p)) return;
    const int blocks = (int)(((size_t)p.E * p.d / 4 + 255) / 256);
    hipLaunchKernelGGL((router_grad_w_sum<T>), dim3(blocks + (p.db ? (p.E + 3) / 4 : 0)),
                       dim3(256), 0, s, p, blocks);
}

bool need_logits(const RouterGradParams &p) {
    return p.z != 0.0f || (p.aux != 0.0f && !p.choice);
}

void router_grad_f32(const RouterGradParams &p, hipStream_t s) {
    const int tt = (p.T + f32t::BM - 1) / f32t::BM;
    if (need_logits(p))
        hipLaunchKernelGGL(router_grad_logits_f32, dim3(tt, p.ep / f32t::BN), dim3(256),
                           0, s, p);
    dlogits<float>(p, s);
    if (p.dx)
        hipLaunchKernelGGL(router_grad_x_f32, dim3(tt, p.d / f32t::BN), dim3(256), 0, s, p);
    if (p.dwr) {
        hipLaunchKernelGGL(router_grad_w_f32,
                           dim3(p.ep / f32t::BM, p.d / f32t::BN, p.splits), dim3(256), 0,
                           s, p);
        sum_splits<float>(p, s);
    }
}

template <bool ROWS> void dx_rows(const RouterGradParams &p, hipStream_t s) {
    const dim3 grid((p.T + 63) / 64, p.d / 64), block(256);
    switch (p.ep / 64) {
    case 1: hipLaunchKernelGGL((router_grad_x_bf16<1, ROWS>), grid, block, 0, s, p); break;
    case 2: hipLaunchKernelGGL((router_grad_x_bf16<2, ROWS>), grid, block, 0, s, p); break;
    case 3: hipLaunchKernelGGL((router_grad_x_bf16<3, ROWS>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((router_grad_x_bf16<4, ROWS>), grid, block, 0, s, p); break;
    }
}

// dx alone by large tiles: whole 64s of experts (a stage's depth) and a tile
// for half of the CUs.  The whole router gradient with them and with a block
// per 64 x 64: 8192 x 7168, 256 experts (896 tiles) 189 and 246 us; 2048 x
// 7168, 256 experts (224) 81 and 98; 4096 x 2048, 64 experts (128) 45.6 and
// 46.4; 1536 x 4096, 64 experts (96) 39.7 and 38.5; 512 x 4096, 64 experts (32)
// 31.7 and 27.5.
bool dx_tiles(int T, int d, int E) {
    return E % 64 == 0 && T >= 256 && d >= 256 &&
           (long long)((T + 255) / 256) * ((d + 255) / 256) >= 128;
}

// dWr by 128-expert tiles: more than 64 experts, and tokens for a block on
// every CU.  The whole gradient with them and with 64-expert tiles: 8192 x
// 7168, 256 experts 189 and 253 us; 1024 x 4096, 256 experts 59 and 65; 512 x
// 4096, 128 experts 39 and 36; 300 x 2048, 256 experts 40 and 37.
bool dw_wide(int T, int d, int E) {
    return E > 64 &&
           (long long)((E + 127) / 128) * ((d + 255) / 256) * ((T + 127) / 128) >= 256;
}

hipError_t router_grad_bf16(const RouterGradParams &p, hipStream_t s) {
    if (need_logits(p)) {
        // the forward's partial logits
        RouterParams q = {};
        q.x = p.x;
        q.wr = p.wr;
        q.part = p.logits;
        q.S = p.logit_splits;
        q.kc = p.logit_depth;
        q.T = p.T;
        q.d = p.d;
        q.E = p.E;
        const hipError_t e = launch_router_logits(q, s);
        if (e != hipSuccess) return e;
    }
    dlogits<uint16_t>(p, s);
    if (p.dx) {
        if (p.dxs || p.dx_add) {
            dx_rows<true>(p, s);
        } else if (dx_tiles(p.T, p.d, p.E)) {
            const int grid = mt::grid_for((long long)((p.T + 255) / 256) * ((p.d + 255) / 256), 1);
            hipLaunchKernelGGL(router_grad_x_tiles, dim3(grid), dim3(256), 0, s, p);
        } else {
            dx_rows<false>(p, s);
        }
    }
    if (p.dwr) {
        const int ny = (p.d + 255) / 256;
        if (dw_wide(p.T, p.d, p.E))
            hipLaunchKernelGGL((router_grad_w_bf16<128>), dim3((p.E + 127) / 128, ny, p.splits),
                               dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL((router_grad_w_bf16<64>), dim3((p.E + 63) / 64, ny, p.splits),
                               dim3(256), 0, s, p);
        sum_splits<uint16_t>(p, s);
    }
    return hipSuccess;
}

}  // namespace

// Enough ranges for the blocks that the CUs hold at once (bf16: one per CU), of
// at least 128 tokens each.  bf16 with twice as many: 8192 x 4096, 64 experts
// 95 us instead of 86, 4096 x 4096, 8 experts 52 instead of 49.
int router_grad_splits(int dtype, int T, int d, int E) {
    const bool bf16 = dtype == 1, wide = bf16 && dw_wide(T, d, E);
    const int bm = wide ? 128 : 64, bn = bf16 ? 256 : f32t::BN;
    const long long tiles = (long long)((E + bm - 1) / bm) * ((d + bn - 1) / bn);
    const long long want = bf16 ? 256 : 512;
    // (rounded up to a block over, the wide tiles would need a second round)
    long long n = wide ? want / tiles : (want + tiles - 1) / tiles;
    const long long most = (T + 127) / 128;
    if (n > most) n = most;
    return (int)(n < 1 ? 1 : n);
}

hipError_t launch_router_grad(const RouterGradParams &p, int dtype, hipStream_t s) {
    if (dtype == 1) {
        const hipError_t e = router_grad_bf16(p, s);
        if (e != hipSuccess) return e;
    } else {
        router_grad_f32(p, s);
    }
    return hipGetLastError();
}

hipError_t launch_zero(void *dst, size_t n, hipStream_t s) {
    const size_t words = n / 2;
    const size_t nb = (words + 2047) / 2048;
    hipLaunchKernelGGL(zero_fill, dim3((unsigned)(nb < 4096 ? (nb ? nb : 1) : 4096)),
                       dim3(256), 0, s, (uint16_t *)dst, words);
    return hipGetLastError();
}
