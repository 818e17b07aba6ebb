// The dense layer's products in single precision: fp32 MFMAs (16x16x4) on
// B x B tiles (128, or 64 where those are few), four waves of B/2 x B/2, over
// ranges of K (the weight gradient: of the rows) where there are few tiles.
//
// A stage is 32 k of both operands, of either memory order, and lies in LDS as
// in memory; two stages, one barrier each.  k contiguous: rows of eight
// 16-byte chunks, XOR-swizzled by the row; a lane reads a chunk, and its four
// k go to four MFMAs (which k an MFMA adds up does not matter as long as both
// operands agree).  Rows contiguous: the same four k by four 4-byte reads, the
// columns XOR-swizzled by 16 so that the four k groups fall on different
// banks.  Sums run over 64 k at a time and are then added to the total, which
// keeps their error near one rounding's.
// Bound by the MFMAs (157 TFLOP/s).
#include "dense_parts.h"

namespace {

constexpr int BK_ = 32;                  // stage depth
constexpr int CHAIN = 64;                // k added up before joining the total

// B x B tiles of 2 x WN waves.
template <int B, int WN> struct Tiles {
    static constexpr int THREADS = 128 * WN;
    // 16 x 16 blocks a wave
    static constexpr int NI = B / 32, NJ = B / 16 / WN;
    static constexpr int LOADS = B * BK_ / 4 / THREADS;   // of a thread and operand
    struct Stage {
        float a[2][B * BK_], b[2][B * BK_];
    };
    // Wave w: rows B/2 (w / WN), columns B/WN (w % WN); block (i, j); the
    // lane's element e: row l % 16, column 4 (l / 16) + e.
    typedef floatx4 Acc[NI][NJ];
    static __device__ __forceinline__ int row(int i) {
        return (threadIdx.x >> 6) / WN * (B / 2) + 16 * i + (threadIdx.x & 15);
    }

    // One operand's stage.  KC: element (r, k) at p[r * ld + k], else at
    // p[k * ld + r]; r from `rows` and k from `depth` on read as 0.  PAIR (of
    // KC): 16 rows of p and 16 of p2 in turn, so that both panels' columns
    // come to the same lanes.
    template <bool KC, bool PAIR = false> struct Part {
        floatx4 v[LOADS];
        __device__ __forceinline__ void fetch(const float *p, const float *p2, size_t ld,
                                              int rows, int k0, int depth) {
#pragma unroll
            for (int h = 0; h < LOADS; ++h) {
                const int i = threadIdx.x + THREADS * h;
                int r = KC ? i >> 3 : i % (B / 4) * 4;
                const int k = k0 + (KC ? (i & 7) * 4 : i / (B / 4));
                const float *from = PAIR && (r & 16) ? p2 : p;
                if (PAIR) r = (r >> 5) * 16 + (r & 15);
                v[h] = r < rows && k < depth
                           ? *(const floatx4 *)(KC ? from + r * ld + k : from + k * ld + r)
                           : floatx4{0.f, 0.f, 0.f, 0.f};
            }
        }
        __device__ __forceinline__ void put(float *s) const {
#pragma unroll
            for (int h = 0; h < LOADS; ++h) {
                const int i = threadIdx.x + THREADS * h;
                if (KC) {
                    const int r = i >> 3, c = i & 7;
                    *(floatx4 *)(s + r * BK_ + ((c ^ (r & 7)) * 4)) = v[h];
                } else {
                    const int k = i / (B / 4), r = i % (B / 4) * 4;
                    *(floatx4 *)(s + k * B + (r ^ (((k >> 2) & 3) * 16))) = v[h];
                }
            }
        }
    };
    // Row r, k 16 kk + 4 b + e of a stage.
    template <bool KC>
    static __device__ __forceinline__ floatx4 fragment(const float *s, int r, int kk, int b) {
        if (KC) return *(const floatx4 *)(s + r * BK_ + (((kk * 4 + b) ^ (r & 7)) * 4));
        floatx4 f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = s[(kk * 16 + 4 * b + e) * B + (r ^ (b * 16))];
        return f;
    }
    static __device__ __forceinline__ void clear(Acc &acc) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    // acc += the sum over k < depth.  Begins and ends with the stages free.
    template <bool AK, bool BKC, bool PAIR = false>
    static __device__ __forceinline__ void product(Acc &acc, Stage &st, const float *pa,
                                                   size_t lda, int rows, const float *pb,
                                                   size_t ldb, int columns, int depth,
                                                   const float *pb2 = nullptr) {
        if (depth <= 0) return;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int l16 = lane & 15, b = lane >> 4;
        const int r0 = wave / WN * (B / 2) + l16, c0 = wave % WN * (B / WN) + l16;
        Part<AK> fa;
        Part<BKC, PAIR> fb;
        fa.fetch(pa, nullptr, lda, rows, 0, depth);
        fb.fetch(pb, pb2, ldb, columns, 0, depth);
        fa.put(st.a[0]);
        fb.put(st.b[0]);
        Acc part;
        clear(part);
        int cur = 0;
        for (int k0 = 0; k0 < depth; k0 += BK_) {
            const bool more = k0 + BK_ < depth;
            if (more) {
                fa.fetch(pa, nullptr, lda, rows, k0 + BK_, depth);
                fb.fetch(pb, pb2, ldb, columns, k0 + BK_, depth);
            }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < BK_ / 16; ++kk) {
                floatx4 x[NI], y[NJ];
#pragma unroll
                for (int i = 0; i < NI; ++i) x[i] = fragment<AK>(st.a[cur], r0 + 16 * i, kk, b);
#pragma unroll
                for (int j = 0; j < NJ; ++j) y[j] = fragment<BKC>(st.b[cur], c0 + 16 * j, kk, b);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
                            part[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                y[j][e], x[i][e], part[i][j], 0, 0, 0);
                // (one half's fragments in registers at a time)
                if (B == 128) __builtin_amdgcn_sched_barrier(0);
            }
            if (more) {
                // (last read before the barrier above)
                fa.put(st.a[cur ^ 1]);
                fb.put(st.b[cur ^ 1]);
                cur ^= 1;
            }
            if (!more || (k0 + BK_) % CHAIN == 0) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) acc[i][j] += part[i][j];
                clear(part);
            }
        }
        __syncthreads();
    }
};

// The block's tile: row tiles side by side, then columns, then ranges.
struct Tile {
    int m0, n0, split;
};
__device__ __forceinline__ Tile tile_at(int L, int mt, int nt, int bm, int bn) {
    Tile t;
    t.split = L / (mt * nt);
    const int local = L - t.split * (mt * nt);
    t.n0 = local / mt * bn;
    t.m0 = local % mt * bm;
    return t;
}

template <int B, int WN, int PANELS, bool BK, bool TWO, int EPI, int ACT>
__device__ __forceinline__ void rows_tile(const DenseRows &p, int L,
                                          typename Tiles<B, WN>::Stage &st) {
    typedef Tiles<B, WN> P;
    constexpr int BN = B / PANELS, NJ = P::NJ / PANELS;
    const int M = p.M, N = p.N, K = p.K;
    const Tile t = tile_at(L, p.plan.mt, p.plan.nt, B, BN);
    const int rows = min(B, M - t.m0), columns = min(BN, N - t.n0);
    const int k0 = t.split * p.plan.per * 64, k = min(p.plan.per * 64, K - k0);
    const size_t bat = BK ? (size_t)k0 * N + t.n0 : (size_t)t.n0 * K + k0;
    typename P::Acc acc;
    P::clear(acc);
    P::template product<true, !BK, PANELS == 2>(
        acc, st, (const float *)p.a + (size_t)t.m0 * K + k0, K, rows, (const float *)p.b + bat,
        BK ? N : K, columns, k, PANELS == 2 ? (const float *)p.b2 + bat : nullptr);
    if (TWO)
        P::template product<true, !BK>(acc, st, (const float *)p.a2 + (size_t)t.m0 * K + k0, K,
                                       rows, (const float *)p.b2 + bat, N, columns, k);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < P::NI; ++i) {
        const int m = P::row(i);
        if (m >= rows) continue;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int in = wave % WN * (BN / WN) + 16 * j + 4 * (lane >> 4), c = t.n0 + in;
            if (in >= columns) continue;
            const size_t at = (size_t)(t.m0 + m) * N + c;
            floatx4 z = acc[i][j * PANELS], u = acc[i][j * PANELS + PANELS - 1];
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

template <int B, int WN, int PANELS, bool BK, bool TWO, int EPI, int ACT>
__global__ __launch_bounds__(128 * WN, 4) void dense_rows_f32(DenseRows p) {
    __shared__ typename Tiles<B, WN>::Stage st;
    rows_tile<B, WN, PANELS, BK, TWO, EPI, ACT>(p, blockIdx.x, st);
}

__device__ __forceinline__ void weight_tile(const DenseWeights &p, int L, Tiles<64, 2>::Stage &st) {
    constexpr int B = 64, WN = 2;
    typedef Tiles<B, WN> P;
    auto tiles = [&](int n) { return (n + B - 1) / B; };
    int k = 0;
    for (; k + 1 < p.count; ++k) {
        const int n = tiles(p.m[k].R) * tiles(p.m[k].C) * p.splits;
        if (L < n) break;
        L -= n;
    }
    const DenseMat &m = p.m[k];
    const Tile t = tile_at(L, tiles(m.R), tiles(m.C), B, B);
    const int r0 = t.split * p.per * 64, depth = min(p.per * 64, p.M - r0);
    const int rows = min(B, m.R - t.m0), columns = min(B, m.C - t.n0);
    typename P::Acc acc;
    P::clear(acc);
    P::template product<false, false>(acc, st, (const float *)m.a + (size_t)r0 * m.R + t.m0, m.R,
                                      rows, (const float *)m.b + (size_t)r0 * m.C + t.n0, m.C,
                                      columns, depth);
    float *out = p.splits > 1
                     ? p.plane + p.offset[k] + (size_t)t.split * m.R * m.C
                     : (float *)m.out;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < P::NI; ++i) {
        const int r = P::row(i);
        if (r >= rows) continue;
#pragma unroll
        for (int j = 0; j < P::NJ; ++j) {
            const int c = wave % WN * (B / WN) + 16 * j + 4 * (lane >> 4);
            if (c < columns)
                *(floatx4 *)(out + (size_t)(t.m0 + r) * m.C + t.n0 + c) = acc[i][j];
        }
    }
}

// The rows' gradient (blocks up to `rows`), the weights' (up to `weights`
// more) and the column sums: nothing here waits for another.
template <bool TWO, int EPI>
__global__ __launch_bounds__(256, 4) void dense_back_f32(DenseBack p, int rows, int weights) {
    __shared__ Tiles<64, 2>::Stage st;
    static_assert(sizeof(st) >= dense_parts::SUMS_LDS, "sums in a stage");
    int block = blockIdx.x;
    if (block < rows) {
        rows_tile<64, 2, 1, true, TWO, EPI, ACT_NONE>(p.dx, block, st);
    } else if ((block -= rows) < weights) {
        weight_tile(p.w, block, st);
    } else {
        dense_parts::sums_and_tails<float>(p.b, p.t, block - weights, (float *)&st);
    }
}

template <int PANELS, bool BK, int EPI, int ACT>
hipError_t launch_large(const DenseRows &p, hipStream_t s) {
    hipLaunchKernelGGL((dense_rows_f32<128, 4, PANELS, BK, false, EPI, ACT>),
                       dim3(p.plan.mt * p.plan.nt), dim3(512), 0, s, p);
    return hipGetLastError();
}
template <int PANELS, bool BK, int EPI, int ACT>
hipError_t launch(const DenseRows &p, hipStream_t s) {
    if (!p.plan.small) return launch_large<PANELS, BK, EPI, ACT>(p, s);
    hipLaunchKernelGGL((dense_rows_f32<64, 2, PANELS, BK, false, EPI, ACT>),
                       dim3(p.plan.mt * p.plan.nt * p.plan.splits), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int EPI> hipError_t by_act(const DenseRows &p, hipStream_t s) {
    switch (p.act) {
    case ACT_GELU: return launch<1, false, EPI, ACT_GELU>(p, s);
    case ACT_SILU: return launch<1, false, EPI, ACT_SILU>(p, s);
    case ACT_SWIGLU: return launch<2, false, EPI, ACT_SWIGLU>(p, s);
    case ACT_GEGLU: return launch<2, false, EPI, ACT_GEGLU>(p, s);
    default: return launch<1, false, EPI, ACT_NONE>(p, s);
    }
}

}  // namespace

hipError_t launch_dense_rows_f32(const DenseRows &p, hipStream_t s) {
    if (p.epilogue == DENSE_PLANE) {
        if (p.bk) return launch<1, true, DENSE_PLANE, ACT_NONE>(p, s);
        return p.panels() == 2 ? launch<2, false, DENSE_PLANE, ACT_SWIGLU>(p, s)
                               : launch<1, false, DENSE_PLANE, ACT_NONE>(p, s);
    }
    // (with small tiles a part of the backward pass's launch)
    if (p.bk) return launch_large<1, true, DENSE_FORWARD, ACT_NONE>(p, s);
    return p.epilogue == DENSE_FORWARD ? by_act<DENSE_FORWARD>(p, s) : by_act<DENSE_GRAD>(p, s);
}

hipError_t launch_dense_back_f32(const DenseBack &p, hipStream_t s) {
    constexpr int b = 64;
    long long weights = 0;
    for (int k = 0; k < p.w.count; ++k)
        weights += (long long)((p.w.m[k].R + b - 1) / b) * ((p.w.m[k].C + b - 1) / b) * p.w.splits;
    const int rows = p.rows ? p.dx.plan.mt * p.dx.plan.nt * p.dx.plan.splits : 0;
    const int sums = dense_parts::sums_blocks(p.b, p.t, 128);
    if (rows + weights + sums == 0) return hipSuccess;
    const dim3 grid((unsigned)(rows + weights + sums));
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, p, rows, (int)weights);
        return hipGetLastError();
    };
    if (p.rows && p.dx.plan.splits > 1)
        return p.dx.two ? run(dense_back_f32<true, DENSE_PLANE>)
                        : run(dense_back_f32<false, DENSE_PLANE>);
    return p.rows && p.dx.two ? run(dense_back_f32<true, DENSE_FORWARD>)
                              : run(dense_back_f32<false, DENSE_FORWARD>);
}
