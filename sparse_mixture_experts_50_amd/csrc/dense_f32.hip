// The dense layer's products in single precision: fp32 MFMAs (16x16x4) on
// B x B tiles (128, or 64 where those are few), over ranges of K (the weight
// gradient: of the rows) where there are few tiles.
//
// A stage is 32 k of both operands, of either memory order, and goes from
// memory to LDS as it lies there; two slots, one barrier a stage.  k
// contiguous: rows of eight 16-byte chunks, XOR-swizzled by the row; a lane
// reads a chunk, and its four k go to four MFMAs (which k an MFMA adds up does
// not matter as long as both operands agree).  Rows contiguous: the same four k
// by four 4-byte reads, the columns XOR-swizzled by 16 so that the four k
// groups fall on different banks.  Sums run over 64 k at a time and are then
// added to the total, which keeps their error near one rounding's.
//
// Bound by the MFMAs (157 TFLOP/s at 2.4 GHz): 4096 x 4096 x 4096 944 us, 146
// TFLOP/s, with the 64 tiles 962; by way of registers instead of straight to
// LDS, 1074 and 1199 (fewer of them left for waves, and the clock lower: 2.15
// GHz).  Four waves of 64 x 64 instead of eight of 64 x 32: 982.
#include "dense_parts.h"

namespace {

constexpr int BK_ = 32;                  // stage depth
constexpr int CHAIN = 2 * BK_;           // k added up before joining the total

// 64 lanes' 16 bytes at base + off (the lane's) to LDS, 0 from base + bytes on.
__device__ __forceinline__ void dma16(uint64_t base, int bytes, uint32_t off, u32x4 *lds) {
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, bytes, 0x00020000),
        (__attribute__((address_space(3))) void *)lds, 16, off, 0, 0, 0);
#endif
}

// B x B tiles of 2 x WN waves.
template <int B, int WN> struct Tiles {
    static constexpr int THREADS = 128 * WN, BLOCKS = B == 64 ? 4 : 2;
    static constexpr int WAVES = THREADS / 256 * BLOCKS;  // of a SIMD
    // 16 x 16 blocks a wave
    static constexpr int NI = B / 32, NJ = B / 16 / WN;
    static constexpr int LOADS = B * BK_ / 4 / THREADS;   // of a wave and operand
    static constexpr int SLOT = 2 * B * BK_ / 4;          // 16-byte chunks of a stage
    // Wave w: rows B/2 (w / WN), columns B/WN (w % WN); block (i, j); the
    // lane's element e: row l % 16, column 4 (l / 16) + e.
    typedef floatx4 Acc[NI][NJ];
    static __device__ __forceinline__ int row(int i) {
        return (threadIdx.x >> 6) / WN * (B / 2) + 16 * i + (threadIdx.x & 15);
    }

    // One operand.  KC: element (r, k) at p[r * ld + k], else at p[k * ld +
    // r]; what r >= rows reads is of no matter, k >= depth reads as 0 (past
    // the end of a buffer).  PAIR (of KC): 16 rows of p and 16 of p2 in turn,
    // so that both panels' columns come to the same lanes.
    template <bool KC, bool PAIR = false> struct Operand {
        const float *p, *p2;
        size_t ld;
        int skip, depth;          // !KC: elements of a row before p
        uint32_t off[LOADS];      // of the lane's chunks, in bytes
        __device__ __forceinline__ Operand(const float *p, const float *p2, size_t ld, int rows,
                                           int skip, int depth)
            : p(p), p2(p2), ld(ld), skip(skip), depth(depth) {
#pragma unroll
            for (int h = 0; h < LOADS; ++h) {
                const int i = threadIdx.x + THREADS * h;
                if (KC) {
                    int r = i >> 3;
                    const int c = (i & 7) ^ (r & 7);
                    if (PAIR) r = (r >> 5) * 16 + (r & 15);
                    off[h] = (uint32_t)min(r, rows - 1) * (uint32_t)(ld * 4) + c * 16;
                } else {
                    const int k = i / (B / 4), r = i % (B / 4) * 4 ^ ((k >> 2) & 3) * 16;
                    off[h] = (uint32_t)k * (uint32_t)(ld * 4) + r * 4;
                }
            }
        }
        // Stage k0 to `to`.
        __device__ __forceinline__ void load(u32x4 *to, int k0) const {
            const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            long long left = k0 < depth ? 0x7FFFFFFF : 0;
            if (!KC) left = max(0ll, min(left, ((depth - k0) * (long long)ld - skip) * 4));
#pragma unroll
            for (int h = 0; h < LOADS; ++h) {
                const int first = wave * 64 + THREADS * h;
                uint64_t from = (uint64_t)(p + (KC ? (size_t)k0 : k0 * ld));
                if (PAIR) from += (first & 128) ? (uint64_t)p2 - (uint64_t)p : 0;
                dma16(from, (int)left, off[h], to + first);
            }
        }
    };
    // Row r, k 16 kk + 4 b + e of a stage.
    template <bool KC>
    static __device__ __forceinline__ floatx4 fragment(const u32x4 *slot, int r, int kk, int b) {
        const float *s = (const float *)slot;
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
    // acc += the stage's products.
    template <bool AK, bool BKC>
    static __device__ __forceinline__ void stage(Acc &acc, const u32x4 *slot) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int l16 = lane & 15, b = lane >> 4;
        const int r0 = wave / WN * (B / 2) + l16, c0 = wave % WN * (B / WN) + l16;
#pragma unroll
        for (int kk = 0; kk < BK_ / 16; ++kk) {
            floatx4 x[NI], y[NJ];
#pragma unroll
            for (int i = 0; i < NI; ++i) x[i] = fragment<AK>(slot, r0 + 16 * i, kk, b);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                y[j] = fragment<BKC>(slot + SLOT / 2, c0 + 16 * j, kk, b);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(y[j][e], x[i][e],
                                                                         acc[i][j], 0, 0, 0);
            // (one half's fragments in registers at a time)
            if (B == 128) __builtin_amdgcn_sched_barrier(0);
        }
    }
    // acc += the sum over k < depth.  Begins and ends with the slots free.
    template <bool AK, bool BKC, bool PAIR = false>
    static __device__ __forceinline__ void product(Acc &acc, u32x4 *slot0, u32x4 *slot1,
                                                   const Operand<AK> &fa,
                                                   const Operand<BKC, PAIR> &fb, int depth) {
        if (depth <= 0) return;
        auto load = [&](u32x4 *slot, int k0) __attribute__((always_inline)) {
            fa.load(slot, k0);
            fb.load(slot + SLOT / 2, k0);
        };
        load(slot0, 0);
        for (int k0 = 0; k0 < depth; k0 += CHAIN) {
            Acc part;
            clear(part);
            __syncthreads();
            load(slot1, k0 + BK_);
            stage<AK, BKC>(part, slot0);
            __syncthreads();
            load(slot0, k0 + CHAIN);
            if (AK || k0 + BK_ < depth) stage<AK, BKC>(part, slot1);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] += part[i][j];
        }
        __syncthreads();
    }
};

constexpr int LARGE_WN = 4;
typedef Tiles<128, LARGE_WN> Large;

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
__device__ __forceinline__ void rows_tile(const DenseRows &p, int L, u32x4 *slot0, u32x4 *slot1) {
    typedef Tiles<B, WN> P;
    constexpr int BN = B / PANELS, NJ = P::NJ / PANELS;
    const int M = p.M, N = p.N, K = p.K;
    const Tile t = tile_at(L, p.plan.mt, p.plan.nt, B, BN);
    const int rows = min(B, M - t.m0), columns = min(BN, N - t.n0);
    const int k0 = t.split * p.plan.per * 64, k = min(p.plan.per * 64, K - k0);
    const size_t bat = BK ? (size_t)k0 * N + t.n0 : (size_t)t.n0 * K + k0;
    typename P::Acc acc;
    P::clear(acc);
    const size_t aat = (size_t)t.m0 * K + k0, ld = BK ? N : K;
    P::template product<true, !BK, PANELS == 2>(
        acc, slot0, slot1, {(const float *)p.a + aat, nullptr, (size_t)K, rows, 0, k},
        {(const float *)p.b + bat, PANELS == 2 ? (const float *)p.b2 + bat : nullptr, ld, columns,
         t.n0, k},
        k);
    if (TWO)
        P::template product<true, !BK>(
            acc, slot0, slot1, {(const float *)p.a2 + aat, nullptr, (size_t)K, rows, 0, k},
            {(const float *)p.b2 + bat, nullptr, ld, columns, t.n0, k}, k);
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
__global__ __launch_bounds__(128 * WN, (Tiles<B, WN>::WAVES)) void dense_rows_f32(DenseRows p) {
    __shared__ u32x4 slot0[Tiles<B, WN>::SLOT], slot1[Tiles<B, WN>::SLOT];
    rows_tile<B, WN, PANELS, BK, TWO, EPI, ACT>(p, blockIdx.x, slot0, slot1);
}

template <int B, int WN>
__device__ __forceinline__ void weight_tile(const DenseWeights &p, int L, u32x4 *slot0,
                                            u32x4 *slot1) {
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
    P::template product<false, false>(
        acc, slot0, slot1,
        {(const float *)m.a + (size_t)r0 * m.R + t.m0, nullptr, (size_t)m.R, rows, t.m0, depth},
        {(const float *)m.b + (size_t)r0 * m.C + t.n0, nullptr, (size_t)m.C, columns, t.n0, depth},
        depth);
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

__global__ __launch_bounds__(Large::THREADS, Large::WAVES) void dense_weight_f32(DenseWeights p) {
    __shared__ u32x4 slot0[Large::SLOT], slot1[Large::SLOT];
    weight_tile<128, LARGE_WN>(p, blockIdx.x, slot0, slot1);
}

// The rows' gradient (blocks up to `rows`), the weights' (up to `weights`
// more) and the column sums: nothing here waits for another.
template <bool TWO, int EPI>
__global__ __launch_bounds__(256, 4) void dense_back_f32(DenseBack p, int rows, int weights) {
    __shared__ u32x4 slot0[Tiles<64, 2>::SLOT], slot1[Tiles<64, 2>::SLOT];
    static_assert(sizeof(slot0) >= dense_parts::SUMS_LDS, "sums in a slot");
    int block = blockIdx.x;
    if (block < rows) {
        rows_tile<64, 2, 1, true, TWO, EPI, ACT_NONE>(p.dx, block, slot0, slot1);
    } else if ((block -= rows) < weights) {
        weight_tile<64, 2>(p.w, block, slot0, slot1);
    } else {
        dense_parts::sums_and_tails<float>(p.b, p.t, block - weights, (float *)slot0);
    }
}

template <int PANELS, bool BK, int EPI, int ACT, bool TWO = false>
hipError_t launch_large(const DenseRows &p, hipStream_t s) {
    hipLaunchKernelGGL((dense_rows_f32<128, LARGE_WN, PANELS, BK, TWO, EPI, ACT>),
                       dim3(p.plan.mt * p.plan.nt * p.plan.splits), dim3(Large::THREADS), 0, s, p);
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
    }
    // (a layer without an activation has no pre-activation's gradient)
    return launch<1, false, DENSE_FORWARD, ACT_NONE>(p, s);
}

}  // namespace

hipError_t launch_dense_rows_f32(const DenseRows &p, hipStream_t s) {
    if (p.epilogue == DENSE_PLANE) {
        if (p.two) return launch_large<1, true, DENSE_PLANE, ACT_NONE, true>(p, s);
        if (p.bk) return launch<1, true, DENSE_PLANE, ACT_NONE>(p, s);
        return p.panels() == 2 ? launch<2, false, DENSE_PLANE, ACT_SWIGLU>(p, s)
                               : launch<1, false, DENSE_PLANE, ACT_NONE>(p, s);
    }
    // (with small tiles a part of the backward pass's launch)
    if (p.bk)
        return p.two ? launch_large<1, true, DENSE_FORWARD, ACT_NONE, true>(p, s)
                     : launch_large<1, true, DENSE_FORWARD, ACT_NONE>(p, s);
    return p.epilogue == DENSE_FORWARD ? by_act<DENSE_FORWARD>(p, s) : by_act<DENSE_GRAD>(p, s);
}

hipError_t launch_dense_back_f32(const DenseBack &p, hipStream_t s) {
    auto tiles = [&](int b) {
        long long n = 0;
        for (int k = 0; k < p.w.count; ++k)
            n += (long long)((p.w.m[k].R + b - 1) / b) * ((p.w.m[k].C + b - 1) / b) * p.w.splits;
        return (int)n;
    };
    const bool together = p.rows && p.dx.plan.small;
    const int rows = together ? p.dx.plan.mt * p.dx.plan.nt * p.dx.plan.splits : 0;
    const int weights = p.w.small ? tiles(64) : 0;
    const int sums = dense_parts::sums_blocks(p.b, p.t, 128);
    if (rows + weights + sums > 0) {
        auto run = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(rows + weights + sums), dim3(256), 0, s, p, rows,
                               weights);
            return hipGetLastError();
        };
        const hipError_t e =
            together && p.dx.plan.splits > 1
                ? p.dx.two ? run(dense_back_f32<true, DENSE_PLANE>)
                           : run(dense_back_f32<false, DENSE_PLANE>)
                : together && p.dx.two ? run(dense_back_f32<true, DENSE_FORWARD>)
                                       : run(dense_back_f32<false, DENSE_FORWARD>);
        if (e != hipSuccess) return e;
    }
    if (p.rows && !together) {
        const hipError_t e = launch_dense_product(p.dx, 0, s);
        if (e != hipSuccess) return e;
    }
    if (p.w.count && !p.w.small) {
        hipLaunchKernelGGL(dense_weight_f32, dim3(tiles(128)), dim3(Large::THREADS), 0, s, p.w);
        return hipGetLastError();
    }
    return hipSuccess;
}
