// Weight gradients of the dense layer, bf16: out[R][C] = A^T B over M rows
// (A [M][R], B [M][C]), up to three matrices in one launch, on the matrix
// cores (tile product in mfma_tile.h; both operands are transposed on their
// way from LDS).  The rows after the last whole stage of 64 come from a
// buffer of 64 rows that is zero from M on, as a second product.
// Few tiles: the rows go in ranges, each to an fp32 plane of its own.
//
// Bound by the matrix cores: 4096 rows, 4096 x 4096 106 us in long runs, 1.30
// PFLOP/s (best call 100, in runs of 40 calls 120); three of 4096 x 14336 in one
// launch 1095 to 1120 us, 1.3 (busy 67 % at 1.86 GHz).
// Tails of zeros instead of masks: with a mask on the rows the loads could not
// go straight to LDS.
#include "dense_parts.h"
#include "dense_tile.h"

namespace {

using dn::bf16;

struct WeightTile {
    int k, mi, ni, split;
};

template <bool SMALL>
using WeightTiles = mt::Tiles<SMALL ? 128 : 256, SMALL ? 128 : 256, 2, 2, 1, true, true, true>;

// The tiles of one block.  scr: 128 TN vectors, large tiles that leave no
// plane.
template <bool SMALL, bool PLANE>
__device__ __forceinline__ void weight_work(const DenseWeights &p, int block, int blocks,
                                            u32x4 *slot0, u32x4 *slot1, u32x4 *scr) {
    constexpr int B = SMALL ? 128 : 256;
    typedef WeightTiles<SMALL> P;
    constexpr int TN = P::TN, RB = B / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / 2, wn = wave % 2;
    const int stages = (p.M + mt::SK - 1) / mt::SK;
    auto tiles = [&](int k) __attribute__((always_inline)) {
        return (p.m[k].R + B - 1) / B * ((p.m[k].C + B - 1) / B);
    };
    int total = 0;
    for (int k = 0; k < p.count; ++k) total += tiles(k) * p.splits;
    auto tile_at = [&](int L) __attribute__((always_inline)) {
        WeightTile t;
        t.k = 0;
        for (; t.k + 1 < p.count && L >= tiles(t.k) * p.splits; ++t.k) L -= tiles(t.k) * p.splits;
        const dn::Tile at = dn::tile_at(L, (p.m[t.k].R + B - 1) / B, (p.m[t.k].C + B - 1) / B);
        t.mi = at.mi;
        t.ni = at.ni;
        t.split = at.split;
        return t;
    };
    auto source = [&](const WeightTile &t) __attribute__((always_inline)) {
        const DenseMat &m = p.m[t.k];
        const int m0 = mt::tile_start(t.mi, B, m.R), n0 = mt::tile_start(t.ni, B, m.C);
        typename P::Source s;
        s.a = (uint64_t)((const bf16 *)m.a + m0);
        s.b = (uint64_t)((const bf16 *)m.b + n0);
        s.a2 = (uint64_t)((const bf16 *)m.a2 + m0);
        s.b2 = (uint64_t)((const bf16 *)m.b2 + n0);
        s.s0 = t.split * p.per;
        s.kt = min(p.per, stages - s.s0);
        return s;
    };
    auto lanes = [&](const WeightTile &t, int lane) __attribute__((always_inline)) {
        const int R = p.m[t.k].R, C = p.m[t.k].C;
        typename P::Lanes ln;
        ln.init(R * 2, min(R, B), C * 2, min(C, B), wave, lane);
        ln.split = p.M / mt::SK;
        return ln;
    };
    int L = dn::first_tile(block, blocks);
    if (L >= total) return;
    WeightTile t = tile_at(L);
    typename P::Source src = source(t);
    typename P::Lanes ln = lanes(t, threadIdx.x & 63);
    P::load_stage(src, ln, 0, slot0, wave);
    P::load_stage(src, ln, 1, slot1, wave);
    mt::wait_loads<0>();
    for (;;) {
        const int lane = mt::tile_lane();
        L += blocks;
        const bool more = L < total;
        const WeightTile tn = more ? tile_at(L) : t;
        const typename P::Source next = source(tn);
        const typename P::Lanes lnext = lanes(tn, lane);
        const int R = p.m[t.k].R, C = p.m[t.k].C;
        const int m0 = mt::tile_start(t.mi, B, R) + wm * RB * 16;
        const int c0 = mt::tile_start(t.ni, B, C) + wn * TN * 16;
        auto work = [&](auto kind) __attribute__((always_inline)) {
            floatx4 acc[RB][TN];
            mt::clear(acc);
            // its first stages, ahead of the last tile's stores, have landed
            mt::wait_loads<SMALL ? 0 : PLANE ? RB * TN : RB * TN / 2>();
            P::template run<RB, RB, decltype(kind)::value>(acc, src, ln, next, lnext, slot0, slot1,
                                                           wave, lane);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const int mi = m0 + i * 16;
                if (SMALL && (mi < t.mi * B || mi >= R)) continue;
                if constexpr (PLANE) {
                    float *out = p.plane + p.offset[t.k] + (size_t)t.split * R * C +
                                 (size_t)(mi + (lane & 15)) * C + c0 + 4 * (lane >> 4);
                    const int lo = t.ni * B - c0, hi = C - c0;
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        if (!SMALL || (16 * j >= lo && 16 * j < hi))
                            *(floatx4 *)(out + 16 * j) = acc[i][j];
                } else {
                    float v[TN][4];
#pragma unroll
                    for (int j = 0; j < TN; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[j][e] = acc[i][j][e];
                    bf16 *row = (bf16 *)p.m[t.k].out + (size_t)mi * C + c0;
                    if constexpr (SMALL) {
                        dn::store_pieces<TN>(v, row + (size_t)(lane & 15) * C, t.ni * B - c0,
                                             C - c0, lane);
                    } else {
                        mt::RowStore<TN> rows;
                        rows.turn(scr, wave * 32 * TN, v, lane);
                        rows.store(row, C, lane);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (src.kt & 1) work(std::integral_constant<mt::Stages, mt::ODD>{});
        else work(std::integral_constant<mt::Stages, mt::EVEN>{});
        if (!more) break;
        t = tn;
        src = next;
        ln = lnext;
    }
    __builtin_amdgcn_s_waitcnt(0);
}

template <bool PLANE>
__global__ __launch_bounds__(256, 1) void dense_weight(DenseWeights p) {
    typedef WeightTiles<false> P;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE], scr[PLANE ? 1 : 128 * P::TN];
    weight_work<false, PLANE>(p, blockIdx.x, gridDim.x, slot0, slot1, scr);
}

// The first `tiles` blocks; the others join.
template <bool PLANE>
__global__ __launch_bounds__(256, 2) void dense_weight_joins(DenseWeights p, DenseRows dx,
                                                             DenseSums b, int tiles, int rows) {
    typedef WeightTiles<true> P;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE];
    const int block = blockIdx.x;
    if (block < tiles)
        weight_work<true, PLANE>(p, block, tiles, slot0, slot1, nullptr);
    else
        dense_parts::join<bf16>(dx, p, b, block - tiles, rows, 0, (float *)slot0);
}

int blocks_of(const DenseWeights &p, int B, int per_cu) {
    long long tiles = 0;
    for (int k = 0; k < p.count; ++k)
        tiles += (long long)((p.m[k].R + B - 1) / B) * ((p.m[k].C + B - 1) / B) * p.splits;
    return mt::grid_for(tiles, per_cu);
}

}  // namespace

hipError_t launch_dense_weights_mfma(const DenseWeights &p, hipStream_t s) {
    const dim3 grid(blocks_of(p, 256, 1));
    if (p.splits > 1) hipLaunchKernelGGL(dense_weight<true>, grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL(dense_weight<false>, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_dense_weights_joins(const DenseWeights &p, const DenseRows &dx,
                                      const DenseSums &b, int rows, int sums, hipStream_t s) {
    const int tiles = blocks_of(p, 128, 2);
    const dim3 grid(tiles + rows + sums);
    if (p.splits > 1)
        hipLaunchKernelGGL(dense_weight_joins<true>, grid, dim3(256), 0, s, p, dx, b, tiles, rows);
    else
        hipLaunchKernelGGL(dense_weight_joins<false>, grid, dim3(256), 0, s, p, dx, b, tiles, rows);
    return hipGetLastError();
}
