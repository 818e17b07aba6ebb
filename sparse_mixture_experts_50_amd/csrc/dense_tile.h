// The bf16 products of rows on the matrix cores (tile product in
// mfma_tile.h), with the dense layer's epilogues.
//
// A tile's rows and columns end with their axes: the last of several starts
// where it ends with the axis, and what it shares with the one before is
// computed, and written with the same bits, twice.  An axis shorter than a
// tile: rows (columns) past its end re-read its first, so their results are
// the first row's and are stored over it with the same bits; columns past the
// end are not stored.  So no operand is read out of range and, in the large
// tiles, no store is a branch.
//
// Bound by the matrix cores, and in long products by the power that they draw:
// 4096 x 4096 to 14336 gated 700 to 720 us (best of 40 calls 653 to 689, by the
// card), 1.34 to 1.37 PFLOP/s, cores busy 75 % at 1.71 GHz; the same with the
// gradient's epilogue 750 to 770.  Short K: 8192 x 2048 to 7168 with a residual
// 213 to 223, 1.1 PFLOP/s: while a tile's epilogue reads and writes 128 KB its
// matrix cores wait.  Tiles of one height, 896 of them or 3.5 rounds of the CUs:
// 227 where two took 218.  The first of the residual fetched ahead of the
// product: 1 % more.
#pragma once

#include "act.h"
#include "dense.h"
#include "mfma_tile.h"

namespace dn {

typedef uint16_t bf16;

// Tiles and slots.  SMALL: for few rows or tiles, several blocks per CU and
// more loads in flight.
template <bool SMALL> struct Shape {
    static constexpr int BM = SMALL ? 64 : 256, BN = SMALL ? 128 : 256;
    static constexpr int SLOTS = SMALL ? 3 : 2, BLOCKS = SMALL ? 2 : 1;
};

struct Tile {
    int mi, ni, split;
};
// Tiles go in strips of 8 row tiles, so that the 32 consecutive tiles of an
// XCD's round are 8 x 4 and read 12 operand panels.
__device__ __forceinline__ Tile tile_at(int L, int mt, int nt) {
    // (divisions are done by vector instructions)
    auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    Tile t;
    t.split = uniform(L / (mt * nt));
    const int local = L - t.split * (mt * nt);
    const int strip = uniform(local / (8 * nt)), in = local - strip * (8 * nt);
    const int sm = min(mt - strip * 8, 8);
    t.ni = sm == 8 ? in >> 3 : uniform(in / sm);
    t.mi = strip * 8 + in - t.ni * sm;
    return t;
}

// mt::tile_of(0) for block `block` of `blocks` (multiples of 8).
__device__ __forceinline__ int first_tile(int block, int blocks) {
    return (block & 7) * (blocks >> 3) + (block >> 3);
}

// f(integral_constant<rb>).  PARTS: 8 and 4.
template <bool SMALL, bool PARTS, typename F>
__device__ __forceinline__ void by_height(int rb, F f) {
    if (SMALL) f(std::integral_constant<int, 2>{});
    else if (rb == 8) f(std::integral_constant<int, 8>{});
    else if (PARTS) f(std::integral_constant<int, 4>{});
    else if (rb == 7) f(std::integral_constant<int, 7>{});
    else if (rb == 6) f(std::integral_constant<int, 6>{});
    else f(std::integral_constant<int, 4>{});
}

// 16 rows of a wave's TN column blocks, columns lo..hi of them, as bf16 to
// `to` (the lane's row): exchanging every second row of 16 lanes with the
// next column block gives a lane 8 columns.
template <int TN>
__device__ __forceinline__ void store_pieces(const float (&v)[TN][4], bf16 *to, int lo, int hi,
                                             int lane) {
    static_assert(TN % 2 == 0, "pairs of column blocks");
    const int hq = lane >> 4, c = (hq & 1) * 16 + (hq >> 1) * 8;
#pragma unroll
    for (int j = 0; j < TN; j += 2) {
        const auto x = __builtin_amdgcn_permlane16_swap(pack_bf16x2(v[j][0], v[j][1]),
                                                        pack_bf16x2(v[j + 1][0], v[j + 1][1]),
                                                        false, false);
        const auto y = __builtin_amdgcn_permlane16_swap(pack_bf16x2(v[j][2], v[j][3]),
                                                        pack_bf16x2(v[j + 1][2], v[j + 1][3]),
                                                        false, false);
        const u32x4 q = {x[0], y[0], x[1], y[1]};
        if (16 * j + c >= lo && 16 * j + c < hi) *(u32x4 *)(to + 16 * j + c) = q;
    }
}

// Stores what rows.turn() read: rows lr0.. of the tile at `out`.
template <int TN>
__device__ __forceinline__ void store_rows(const mt::RowStore<TN> &rows, bf16 *out, size_t ld,
                                           int lr0, int valid, int lane) {
    constexpr int CPR = mt::RowStore<TN>::CPR;
#pragma unroll
    for (int i = 0; i < CPR / 4; ++i) {
        const int r = lr0 + i * (64 / CPR) + lane / CPR;
        *(u32x4 *)(out + (size_t)(r < valid ? r : 0) * ld + lane % CPR * 8) = rows.q[i];
    }
}

__device__ __forceinline__ floatx4 unpack4(u32x2 v) {
    return floatx4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}

// The tile product of rows.
template <int PANELS, bool BK, bool TWO, bool SMALL>
using RowTiles = mt::Tiles<Shape<SMALL>::BM, Shape<SMALL>::BN / PANELS, 2, 2, PANELS, false, BK,
                           TWO>;

// The tiles of one block.  slot2: SMALL; scr: 128 TN vectors, large tiles that
// leave no plane.
template <int PANELS, bool BK, bool TWO, int EPI, int ACT, bool RES, mt::Stages KIND, bool SMALL,
          bool PARTS = false>
__device__ __forceinline__ void rows_work(const DenseRows &p, int block, int blocks, u32x4 *slot0,
                                          u32x4 *slot1, u32x4 *slot2, u32x4 *scr) {
    constexpr int BN = Shape<SMALL>::BN / PANELS;
    typedef RowTiles<PANELS, BK, TWO, SMALL> P;
    constexpr int TN = P::TN;
    const int M = p.M, N = p.N, K = p.K;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / 2, wn = wave % 2;
    const int kt = (TWO ? 2 : 1) * K / mt::SK, per = p.plan.per;
    // Tiles L, L + blocks, ... of mt_ x nt x splits that are rb high, from
    // column ni0 on.
    auto tiles = [&](int rb, int mt_, int nt, int ni0, int L) __attribute__((always_inline)) {
        const int total = mt_ * nt * (ni0 ? 1 : p.plan.splits);
        if (L >= total) return;
        by_height<SMALL, PARTS>(rb, [&](auto height) __attribute__((always_inline)) {
            constexpr int RB = decltype(height)::value;
            // rows from here on re-read the first (also those that a lower tile
            // does not use but may load)
            const int valid = min(M, 32 * RB);
            auto row0_of = [&](const Tile &t) __attribute__((always_inline)) {
                return mt::tile_start(t.mi, 32 * RB, M);
            };
            auto source = [&](const Tile &t) __attribute__((always_inline)) {
                const size_t at = (size_t)row0_of(t) * K;
                const size_t n0 = mt::tile_start(t.ni, BN, N), bat = BK ? n0 : n0 * K;
                typename P::Source s;
                s.a = (uint64_t)((const bf16 *)p.a + at);
                s.a2 = TWO ? (uint64_t)((const bf16 *)p.a2 + at) : s.a;
                s.b = (uint64_t)((const bf16 *)p.b + bat);
                s.b2 = TWO || PANELS > 1 ? (uint64_t)((const bf16 *)p.b2 + bat) : s.b;
                s.s0 = t.split * per;
                s.kt = min(per, kt - s.s0);
                return s;
            };
            typename P::Lanes ln;
            ln.init(K * 2, valid, (BK ? N : K) * 2, min(N, BN), wave, threadIdx.x & 63);
            ln.split = K / mt::SK;
            auto tile = [&](int at) __attribute__((always_inline)) {
                Tile t = tile_at(at, mt_, nt);
                t.ni += ni0;
                return t;
            };
            Tile t = tile(L);
            typename P::Source src = source(t);
            P::load_stage(src, ln, 0, slot0, wave);
            P::load_stage(src, ln, 1, slot1, wave);
            if (SMALL) P::load_stage(src, ln, 2, slot2, wave);
            mt::wait_loads<0>();
            for (;;) {
                const int lane = mt::tile_lane();
                L += blocks;
                const bool more = L < total;
                const Tile tn = more ? tile(L) : t;
                const typename P::Source next = source(tn);
                const int l16 = lane & 15;
                const int c0 = mt::tile_start(t.ni, BN, N) + wn * TN * 16;
                // this wave's columns of the tile's own, from c0: lo..hi
                const int lo = t.ni * BN - c0, hi = N - c0;
                const int cq = c0 + 4 * (lane >> 4);
                const int row0 = row0_of(t);
                // the lane's row of row block i, and whether column block j is
                // stored
                auto row_of = [&](int i) __attribute__((always_inline)) {
                    const int lr = (wm * RB + i) * 16 + l16;
                    return (size_t)(row0 + (lr < valid ? lr : 0));
                };
                auto own = [&](int j) __attribute__((always_inline)) {
                    return !SMALL || (16 * j >= lo && 16 * j < hi);
                };
                floatx4 acc[RB][TN * PANELS];
                mt::clear(acc);
                if (EPI != DENSE_PLANE) {
                    // the sums start from the biases
    #pragma unroll
                    for (int k = 0; k < PANELS; ++k) {
                        const bf16 *bias = (const bf16 *)(k ? p.bias2 : p.bias);
                        if (!bias) continue;
    #pragma unroll
                        for (int j = 0; j < TN; ++j) {
                            if (16 * j >= hi) continue;      // whole blocks: N % 64 == 0
                            const floatx4 f = unpack4(*(const u32x2 *)(bias + cq + 16 * j));
    #pragma unroll
                            for (int i = 0; i < RB; ++i) acc[i][k * TN + j] = f;
                        }
                    }
                }
                if constexpr (SMALL) {
                    u32x4 *const slot[3] = {slot0, slot1, slot2};
                    P::template run_ring<RB, 3>(acc, src, ln, next, ln, slot, wave, lane);
                } else {
                    P::template run<RB, RB, KIND>(acc, src, ln, next, ln, slot0, slot1, wave, lane);
                }
                if constexpr (EPI == DENSE_PLANE) {
    #pragma unroll
                    for (int k = 0; k < PANELS; ++k) {
                        float *plane = p.plane + ((size_t)t.split * PANELS + k) * M * N;
    #pragma unroll
                        for (int i = 0; i < RB; ++i) {
                            float *out = plane + row_of(i) * N + cq;
    #pragma unroll
                            for (int j = 0; j < TN; ++j)
                                if (own(j)) *(floatx4 *)(out + 16 * j) = acc[i][k * TN + j];
                        }
                    }
                    // the next tile's loads, ahead of the stores, have landed
                    mt::wait_loads<SMALL ? 0 : RB * TN * PANELS>();
                } else if constexpr (EPI == DENSE_FORWARD) {
                    auto fetch = [&](int i, u32x2 (&q)[TN]) __attribute__((always_inline)) {
                        const bf16 *rp = (const bf16 *)p.res + row_of(i) * N + cq;
    #pragma unroll
                        for (int j = 0; j < TN; ++j)
                            q[j] = own(j) ? *(const u32x2 *)(rp + 16 * j) : u32x2{0, 0};
                    };
                    // the next row block's part of res is on the way while one is
                    // worked on
                    u32x2 q[2][TN];
                    if (RES) fetch(0, q[0]);
                    P::pin(acc);
    #pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        if (RES && i + 1 < RB) fetch(i + 1, q[(i + 1) & 1]);
                        __builtin_amdgcn_sched_barrier(0);
                        float v[TN][4];
    #pragma unroll
                        for (int j = 0; j < TN; ++j) {
                            const floatx4 add = RES ? unpack4(q[i & 1][j]) : floatx4{};
    #pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                v[j][e] = act_value<ACT, true>(acc[i][j][e],
                                                               acc[i][j + TN * (PANELS - 1)][e]);
                                if (RES) v[j][e] += add[e];
                            }
                        }
                        const int lr = (wm * RB + i) * 16;
                        if constexpr (SMALL) {
                            store_pieces<TN>(v, (bf16 *)p.y + row_of(i) * N + c0, lo, hi, lane);
                        } else {
                            mt::RowStore<TN> rows;
                            rows.turn(scr, wave * 32 * TN, v, lane);
                            store_rows<TN>(rows, (bf16 *)p.y + (size_t)row0 * N + c0, N, lr, valid,
                                           lane);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    mt::wait_loads<SMALL ? 0 : RB * TN / 2>();
                } else {
                    auto fetch = [&](int i, floatx4 (&q)[TN]) __attribute__((always_inline)) {
                        const size_t at = row_of(i) * N + cq;
                        if (p.dy) {
    #pragma unroll
                            for (int j = 0; j < TN; ++j)
                                q[j] = own(j) ? unpack4(*(const u32x2 *)((const bf16 *)p.dy + at +
                                                                         16 * j))
                                              : floatx4{0.f, 0.f, 0.f, 0.f};
                            return;
                        }
    #pragma unroll
                        for (int j = 0; j < TN; ++j)
                            q[j] = own(j) ? *(const floatx4 *)(p.q + at + 16 * j)
                                          : floatx4{0.f, 0.f, 0.f, 0.f};
                        for (int s = 1; s < p.q_planes; ++s) {
                            const float *qs = p.q + (size_t)s * M * N + at;
    #pragma unroll
                            for (int j = 0; j < TN; ++j)
                                if (own(j)) q[j] += *(const floatx4 *)(qs + 16 * j);
                        }
                    };
                    floatx4 q[2][TN];
                    fetch(0, q[0]);
                    P::pin(acc);
    #pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        if (i + 1 < RB) fetch(i + 1, q[(i + 1) & 1]);
                        __builtin_amdgcn_sched_barrier(0);
                        float vh[TN][4], vz[TN][4], vu[TN][4];
    #pragma unroll
                        for (int j = 0; j < TN; ++j)
    #pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float hz, hu;
                                act_grad<ACT, true>(acc[i][j][e],
                                                    acc[i][j + TN * (PANELS - 1)][e], vh[j][e],
                                                    hz, hu);
                                const float qq = q[i & 1][j][e];
                                vz[j][e] = qq * hz;
                                vu[j][e] = qq * hu;
                            }
                        const int lr = (wm * RB + i) * 16;
                        const size_t at = (size_t)row0 * N + c0;
                        auto put = [&](void *out, const float (&v)[TN][4])
                                       __attribute__((always_inline)) {
                            if constexpr (SMALL) {
                                store_pieces<TN>(v, (bf16 *)out + row_of(i) * N + c0, lo, hi, lane);
                            } else {
                                mt::RowStore<TN> rows;
                                rows.turn(scr, wave * 32 * TN, v, lane);
                                store_rows<TN>(rows, (bf16 *)out + at, N, lr, valid, lane);
                            }
                        };
                        put(p.dz, vz);
                        if (PANELS > 1) put(p.du, vu);
                        if (p.h) put(p.h, vh);
                        // one row block at a time: the accumulators are read as
                        // they are used, not all at once
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    // (the last fetch, waited for above, came behind the next
                    // tile's loads: what is outstanding are the last stores)
                    mt::wait_loads<SMALL ? 0 : TN / 2>();
                }
                if (!more) break;
                t = tn;
                src = next;
            }
        });
    };
    int L = first_tile(block, blocks);
    if (!PARTS) {
        tiles(p.plan.rb, p.plan.mt, p.plan.nt, 0, L);
    } else {
        // one copy of the code for both; the blocks that had one tile less
        // take the first of the lower ones
        const int whole = p.plan.nt - p.plan.nt2;
        for (int part = 0; part < 2; ++part) {
            tiles(part ? p.plan.rb2 : p.plan.rb, part ? p.plan.mt2 : p.plan.mt,
                  part ? p.plan.nt2 : whole, part ? whole : 0, L);
            // (what the last tile loaded ahead, and the slots)
            mt::wait_loads<0>();
            __builtin_amdgcn_s_barrier();
            L -= p.plan.mt * whole % blocks;
            if (L < 0) L += blocks;
        }
    }
    __builtin_amdgcn_s_waitcnt(0);
}

template <int PANELS, bool BK, bool TWO, int EPI, int ACT, bool RES, mt::Stages KIND, bool SMALL,
          bool PARTS>
__global__ __launch_bounds__(256, Shape<SMALL>::BLOCKS) void dense_rows(DenseRows p) {
    typedef RowTiles<PANELS, BK, TWO, SMALL> P;
    constexpr bool TURN = !SMALL && EPI != DENSE_PLANE;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE], slot2[SMALL ? P::STAGE : 1];
    __shared__ u32x4 scr[TURN ? 128 * P::TN : 1];
    rows_work<PANELS, BK, TWO, EPI, ACT, RES, KIND, SMALL, PARTS>(p, blockIdx.x, gridDim.x, slot0,
                                                                 slot1, slot2, scr);
}

template <int PANELS, bool BK, bool TWO, int EPI, int ACT, bool RES, mt::Stages KIND, bool SMALL,
          bool PARTS = false>
hipError_t launch_as(const DenseRows &p, hipStream_t s) {
    const dim3 grid(mt::grid_for(p.plan.tiles(), Shape<SMALL>::BLOCKS));
    hipLaunchKernelGGL((dense_rows<PANELS, BK, TWO, EPI, ACT, RES, KIND, SMALL, PARTS>), grid,
                       dim3(256), 0, s, p);
    return hipGetLastError();
}

// By the parity of a tile's stages, and the tiles' size.
template <int PANELS, bool BK, bool TWO, int EPI, int ACT, bool RES>
hipError_t launch_large(const DenseRows &p, hipStream_t s) {
    // planes of ranges of K, which are even and of one height (all of K in one
    // plane: the gradient of h alone)
    if constexpr (EPI == DENSE_PLANE && (TWO || !BK))
        return launch_as<PANELS, BK, TWO, EPI, ACT, RES, mt::EVEN, false>(p, s);
    auto launch = [&](auto kind) {
        constexpr mt::Stages KIND = decltype(kind)::value;
        return p.plan.nt2 ? launch_as<PANELS, BK, TWO, EPI, ACT, RES, KIND, false, true>(p, s)
                          : launch_as<PANELS, BK, TWO, EPI, ACT, RES, KIND, false>(p, s);
    };
    if constexpr (!TWO)
        if (p.plan.per & 1) return launch(std::integral_constant<mt::Stages, mt::ODD>{});
    return launch(std::integral_constant<mt::Stages, mt::EVEN>{});
}
template <int PANELS, bool BK, bool TWO, int EPI, int ACT, bool RES>
hipError_t launch_by_plan(const DenseRows &p, hipStream_t s) {
    return p.plan.small ? launch_as<PANELS, BK, TWO, EPI, ACT, RES, mt::EVEN, true>(p, s)
                        : launch_large<PANELS, BK, TWO, EPI, ACT, RES>(p, s);
}

// The forward's epilogue, with or without a residual.
template <int PANELS, int ACT> hipError_t launch_forward(const DenseRows &p, hipStream_t s) {
    return p.res ? launch_by_plan<PANELS, false, false, DENSE_FORWARD, ACT, true>(p, s)
                 : launch_by_plan<PANELS, false, false, DENSE_FORWARD, ACT, false>(p, s);
}

}  // namespace dn
