// The bf16 layer's gradient GEMMs on the matrix cores (formulas in
// ffn_grad.hip, the tile product in mfma_tile.h):
//   rows by weights  q = dy W2 (fp32), and at the end dx = dz W1 + du W3
//   act grad     z = x W1^T and u = x W3^T on one output tile, then with q
//                r h, dz, du and the parts of <q, h> from the accumulators
//   weight grad  dW1 = dz^T x, dW3 = du^T x, dW2 = dy^T (r h) over the rows
//                of a group
// r h, dz and du are operands of bf16 products and rounded to bf16 once: the
// gradients they enter are then off by 0.0023 of their norm, where the rounding
// of the result alone is 0.0017.  (In two parts each, as the router's dl, dx and
// all weight gradients would take twice the MFMAs.)
// q passes through memory in fp32 (4 bytes a value, written and read once:
// 0.2 ms of the Mixtral-shaped 4096-token gradient) so that every product
// has a 256 x 256 tile: with z and q accumulated side by side a block's
// tile is 256 x 128, whose fragment reads take longer than its MFMAs.
// Bound by the matrix cores.  Measured, Mixtral-shaped (4096 tokens, 8 experts
// of 4096 x 14336, top-2, 1.92 TFLOP of weight gradients and half of that in
// each other product): q 0.89 ms, act grad 1.05, dx 0.99, weight grad 1.73,
// 0.9 to 1.1 PFLOP/s, the matrix cores busy 47 to 57 %; a large plain product
// runs at 1.1 to 1.4.  Fine-grained (4096 tokens, 64 gated experts of
// 2048 x 1408, top-6, and the shared one): q 0.26 ms, act grad 0.44, dx 0.40,
// weight grad 0.73, 0.6 to 0.8 PFLOP/s: with 7 stages a tile, the tile's
// start, its epilogue and the burst of its stores, which all CUs come to
// together, take a third of the time.
// All three are persistent: one block per CU, whose tiles of a round lie
// side by side in each XCD (consecutive tile numbers), where they share
// operand panels through that XCD's L2.
#include "ffn_grad.h"
#include "mfma_tile.h"

namespace {

typedef uint16_t bf16;

// h, dh/dz and dh/du, with the fast forms of common.h: gelu_erf's erfc and
// silu_f's exponential (relative errors of a few 1e-7).
template <int ACT>
__device__ __forceinline__ void act_grad(float z, float u, float &h, float &hz,
                                         float &hu) {
    hu = 0.0f;
    if (ACT == ACT_GELU) {
        h = gelu_erf(z);
        // Phi + z phi; Phi = h / z loses nothing but its value at 0
        const float pdf = 0.39894228f * __builtin_amdgcn_exp2f(z * z * -0.72134752f);
        const float az = fabsf(z);
        const float cdf = az > 1e-3f ? h * __builtin_amdgcn_rcpf(z)
                                     : fmaf(0.39894228f, z, 0.5f);
        hz = fmaf(z, pdf, cdf);
    } else {
        const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
        const float a = z * sg;
        const float da = fmaf(a, 1.0f - sg, sg);
        if (ACT == ACT_SILU) {
            h = a;
            hz = da;
        } else {
            h = a * u;
            hz = da * u;
            hu = a;
        }
    }
}

// Stores 16 rows of a wave's TN column blocks, columns lo..hi of them, as
// bf16 and straight from the registers: exchanging every second row of 16
// lanes with the next column block gives a lane 8 columns.
template <int TN>
__device__ __forceinline__ void store_pieces(const float (&v)[TN][4], bf16 *out, size_t ld,
                                             int lo, int hi, int lane) {
    static_assert(TN % 2 == 0, "pairs of column blocks");
    const int hq = lane >> 4, c = (hq & 1) * 16 + (hq >> 1) * 8;
    bf16 *to = out + (size_t)(lane & 15) * ld + c;
#pragma unroll
    for (int j = 0; j < TN; j += 2) {
        const auto x = __builtin_amdgcn_permlane16_swap(pack_bf16x2(v[j][0], v[j][1]),
                                                        pack_bf16x2(v[j + 1][0], v[j + 1][1]),
                                                        false, false);
        const auto y = __builtin_amdgcn_permlane16_swap(pack_bf16x2(v[j][2], v[j][3]),
                                                        pack_bf16x2(v[j + 1][2], v[j + 1][3]),
                                                        false, false);
        const u32x4 q = {x[0], y[0], x[1], y[1]};
        if (16 * j + c >= lo && 16 * j + c < hi) *(u32x4 *)(to + 16 * j) = q;
    }
}

// (Groups are padded to 64 rows, see pad_groups.)
// A group's rows in ceil(rows / 256) tiles of one height, 32 rb rows: rb
// (16-row blocks per wave) is what an even split needs, rounded up to 2, 4,
// 6, 7 or 8.  (Whole tiles of every group first and one of the 64 to 192 rows
// left over after them: fine-grained act grad 0.53 ms instead of 0.44, dx 0.45
// instead of 0.40, Mixtral-shaped q 0.96 instead of 0.91 and dx 0.97 instead
// of 1.01; a stage of a low tile takes nearly as long as a whole one's.)  The
// last tile of several ends with the group: rows that it shares with the one before are
// computed, and written with the same bits, twice, so that every tile is
// whole and no store is a branch.
__device__ __forceinline__ int split_blocks(int rows) {
    const int m = (rows + 255) >> 8;
    const int rb = ((rows + m - 1) / m + 31) >> 5;
    return rb <= 6 ? (rb + 1) & ~1 : rb;
}

struct RowTile {
    int g, row0, rb, n_tile;
};
template <bool SMALL>
__device__ __forceinline__ RowTile row_tile(const TileTable &tt, int G, int L) {
    RowTile r;
    r.g = __builtin_amdgcn_readfirstlane(find_group(tt, G, L));
    const int local = L - __builtin_amdgcn_readfirstlane(tt.base[r.g]);
    const int mt = __builtin_amdgcn_readfirstlane(tt.mt[r.g]);
    const int rows = __builtin_amdgcn_readfirstlane(tt.rows[r.g]);
    r.rb = SMALL ? 2 : split_blocks(rows);
    r.n_tile = local / mt;
    const int m = local - r.n_tile * mt;
    r.row0 = __builtin_amdgcn_readfirstlane(tt.start[r.g]) +
             min(m * 32 * r.rb, rows - 32 * r.rb);
    return r;
}

// f(integral_constant<rb>)
template <bool SMALL, typename F> __device__ __forceinline__ void by_height(int rb, F f) {
    if (SMALL) f(std::integral_constant<int, 2>{});
    else if (rb == 8) f(std::integral_constant<int, 8>{});
    else if (rb == 7) f(std::integral_constant<int, 7>{});
    else if (rb == 6) f(std::integral_constant<int, 6>{});
    else if (rb == 4) f(std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, 2>{});
}

// Tiles and slots of the kernels below.  SMALL: for groups of few rows, whose
// products stream the weights once: small tiles, several blocks per CU, more
// loads in flight.
template <bool SMALL> struct Shape {
    static constexpr int BM = SMALL ? 64 : 256, BN = SMALL ? 128 : 256;
    static constexpr int SLOTS = SMALL ? 3 : 2, BLOCKS = SMALL ? 2 : 1;
};

// Keeps the slots' first stages coming: run() through two slots, run_ring()
// through three.
template <typename P, bool SMALL, int RB, mt::Stages KIND, int NC>
__device__ __forceinline__ void run_tile(floatx4 (&acc)[RB][NC], const typename P::Source &src,
                                         const typename P::Source &next,
                                         const typename P::Lanes &ln, u32x4 *slot0,
                                         u32x4 *slot1, u32x4 *slot2, int wave, int lane) {
    if constexpr (SMALL) {
        u32x4 *const slot[3] = {slot0, slot1, slot2};
        P::template run_ring<RB, 3>(acc, src, ln, next, ln, slot, wave, lane);
    } else {
        P::template run<RB, RB, KIND>(acc, src, ln, next, ln, slot0, slot1, wave, lane);
    }
}

// out[rows][N] (fp32) = the sum of one or two products A B of a group's rows
// with its weights, stored along K.  Q: q = dy W2; else dx = dz W1 + du W3
// (GATED).  SMALL: over one of `splits` ranges of K, each to a plane of its
// own.
template <bool Q, bool GATED, mt::Stages KIND, bool SMALL>
__global__ __launch_bounds__(256, Shape<SMALL>::BLOCKS) void ffn_rows_by_weights(FfnGradParams p) {
    constexpr int BM = Shape<SMALL>::BM, BN = Shape<SMALL>::BN;
    typedef mt::Tiles<BM, BN, 2, 2, 1, false, true, GATED> P;
    constexpr int TN = P::TN;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE], slot2[SMALL ? P::STAGE : 1];
    __shared__ TileTable tt;
    const int G = p.E + p.n_shared;
    const int N = Q ? p.d_ff : p.d, K = Q ? p.d : p.d_ff;
    build_tile_table(tt, p.offsets, p.E, p.n_shared, 0, p.T, BM, (N + BN - 1) / BN);
    const int splits = !SMALL ? 1 : Q ? p.q_splits : p.dx_splits;
    const int tiles = __builtin_amdgcn_readfirstlane(tt.base[G]), total = tiles * splits;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / 2, wn = wave % 2;
    const int kt = (GATED ? 2 : 1) * K / mt::SK, per = (kt + splits - 1) / splits;
    const size_t mat = (size_t)p.d_ff * p.d;
    auto source = [&](const RowTile &t, int split) __attribute__((always_inline)) {
        const int n0 = mt::tile_start(t.n_tile, BN, N);
        const size_t at = (size_t)t.row0 * K;
        typename P::Source s;
        s.a = (uint64_t)((const bf16 *)(Q ? p.dys : p.dz) + at);
        s.b = (uint64_t)(of_group<bf16>(Q ? p.w2 : p.w1, Q ? p.ws2 : p.ws1, t.g, p.E, mat) + n0);
        s.a2 = GATED ? (uint64_t)((const bf16 *)p.du + at) : s.a;
        s.b2 = GATED ? (uint64_t)(of_group<bf16>(p.w3, p.ws3, t.g, p.E, mat) + n0) : s.b;
        s.s0 = SMALL ? split * per : 0;
        s.kt = SMALL ? min(per, kt - s.s0) : kt;
        return s;
    };
    int L = mt::tile_of(0);
    if (L >= total) return;
    typename P::Lanes ln;
    ln.init(K * 2, BM, N * 2, min(N, BN), wave, threadIdx.x & 63);
    ln.split = K / mt::SK;
    int split = SMALL ? L / tiles : 0;
    RowTile t = row_tile<SMALL>(tt, G, L - split * tiles);
    typename P::Source src = source(t, split);
    P::load_stage(src, ln, 0, slot0, wave);
    P::load_stage(src, ln, 1, slot1, wave);
    if (SMALL) P::load_stage(src, ln, 2, slot2, wave);
    mt::wait_loads<0>();
    for (int r = 1;; ++r) {
        const int lane = mt::tile_lane();
        L = mt::tile_of(r);
        const bool more = L < total;
        const int nsplit = SMALL && more ? L / tiles : split;
        const RowTile tn = more ? row_tile<SMALL>(tt, G, L - nsplit * tiles) : t;
        const typename P::Source next = source(tn, nsplit);
        by_height<SMALL>(t.rb, [&](auto height) __attribute__((always_inline)) {
            constexpr int RB = decltype(height)::value;
            floatx4 acc[RB][TN];
            mt::clear(acc);
            run_tile<P, SMALL, RB, KIND>(acc, src, next, ln, slot0, slot1, slot2, wave, lane);
            const int lo = t.n_tile * BN;
            const int c0 = mt::tile_start(t.n_tile, BN, N) + wn * TN * 16;
            float *plane = (Q ? p.q : p.dxs) + (size_t)split * p.rows * N;
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                float *out = plane + (size_t)(t.row0 + (wm * RB + i) * 16 + (lane & 15)) * N +
                             c0 + 4 * (lane >> 4);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    if (!SMALL || (c0 + 16 * j >= lo && c0 + 16 * j < N))
                        *(floatx4 *)(out + 16 * j) = acc[i][j];
            }
            // the next tile's loads, ahead of the stores, have landed
            mt::wait_loads<SMALL ? 0 : RB * TN>();
        });
        if (!more) break;
        t = tn;
        src = next;
        split = nsplit;
    }
    __builtin_amdgcn_s_waitcnt(0);
}

// z (and u) of a tile, then with q: r h, dz, du and the parts of <q, h>.  A
// gated tile has half the columns, of z and of u.
template <int ACT, mt::Stages KIND, bool SMALL>
__global__ __launch_bounds__(256, Shape<SMALL>::BLOCKS) void ffn_act_grad(FfnGradParams p) {
    constexpr int PANELS = ACT == ACT_SWIGLU ? 2 : 1;
    constexpr int BM = Shape<SMALL>::BM, BN = Shape<SMALL>::BN / PANELS;
    typedef mt::Tiles<BM, BN, 2, 2, PANELS, false, false> P;
    constexpr int TN = P::TN;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE], slot2[SMALL ? P::STAGE : 1];
    __shared__ u32x4 scr[SMALL ? 1 : 4 * 32 * TN];
    __shared__ TileTable tt;
    const int G = p.E + p.n_shared, d = p.d, F = p.d_ff;
    build_tile_table(tt, p.offsets, p.E, p.n_shared, 0, p.T, BM, (F + BN - 1) / BN);
    const int total = __builtin_amdgcn_readfirstlane(tt.base[G]);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / 2, wn = wave % 2;
    const int kt = d / mt::SK;
    const size_t mat = (size_t)F * d;
    auto source = [&](const RowTile &t) __attribute__((always_inline)) {
        const size_t at = (size_t)mt::tile_start(t.n_tile, BN, F) * d;
        typename P::Source s;
        s.a = s.a2 = (uint64_t)((const bf16 *)p.xs + (size_t)t.row0 * d);
        s.b = (uint64_t)(of_group<bf16>(p.w1, p.ws1, t.g, p.E, mat) + at);
        s.b2 = PANELS > 1 ? (uint64_t)(of_group<bf16>(p.w3, p.ws3, t.g, p.E, mat) + at) : s.b;
        s.kt = kt;
        s.s0 = 0;
        return s;
    };
    int L = mt::tile_of(0);
    if (L >= total) return;
    typename P::Lanes ln;
    ln.init(d * 2, BM, d * 2, min(F, BN), wave, threadIdx.x & 63);
    ln.split = kt;
    RowTile t = row_tile<SMALL>(tt, G, L);
    typename P::Source src = source(t);
    P::load_stage(src, ln, 0, slot0, wave);
    P::load_stage(src, ln, 1, slot1, wave);
    if (SMALL) P::load_stage(src, ln, 2, slot2, wave);
    mt::wait_loads<0>();
    for (int r = 1;; ++r) {
        const int lane = mt::tile_lane();
        L = mt::tile_of(r);
        const bool more = L < total;
        const RowTile tn = more ? row_tile<SMALL>(tt, G, L) : t;
        const typename P::Source next = source(tn);
        const int l16 = lane & 15;
        const int c0 = mt::tile_start(t.n_tile, BN, F) + wn * TN * 16;
        // this wave's columns of the tile's own, from c0: lo..hi
        const int lo = t.n_tile * BN - c0, hi = F - c0;
        const int cq = c0 + 4 * (lane >> 4);
        const bf16 *bias[2] = {of_group<bf16>(p.b1, p.bs1, t.g, p.E, F),
                               PANELS > 1 ? of_group<bf16>(p.b3, p.bs3, t.g, p.E, F) : nullptr};
        by_height<SMALL>(t.rb, [&](auto height) __attribute__((always_inline)) {
            constexpr int RB = decltype(height)::value;
            // the sums start from the biases
            floatx4 z[RB][TN * PANELS];
            mt::clear(z);
#pragma unroll
            for (int k = 0; k < PANELS; ++k)
                if (bias[k]) {
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        if (16 * j >= hi) continue;      // whole blocks: F % 64 == 0
                        const u32x2 v = *(const u32x2 *)(bias[k] + cq + 16 * j);
                        const floatx4 f = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y),
                                           bf16_hi(v.y)};
#pragma unroll
                        for (int i = 0; i < RB; ++i) z[i][k * TN + j] = f;
                    }
                }
            run_tile<P, SMALL, RB, KIND>(z, src, next, ln, slot0, slot1, slot2, wave, lane);
            // q and the routing weight of row block i
            auto fetch = [&](int i, floatx4 (&q)[TN], float &w) __attribute__((always_inline)) {
                const int row = t.row0 + (wm * RB + i) * 16 + l16;
                const float *qp = p.q + (size_t)row * F + cq;
                w = p.row_w[row];
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    q[j] = !SMALL || (16 * j >= lo && 16 * j < hi)
                               ? *(const floatx4 *)(qp + 16 * j)
                               : floatx4{0.f, 0.f, 0.f, 0.f};
                if (SMALL) {
                    for (int s = 1; s < p.q_splits; ++s) {
                        const float *qs = qp + (size_t)s * p.rows * F;
#pragma unroll
                        for (int j = 0; j < TN; ++j)
                            if (16 * j >= lo && 16 * j < hi) q[j] += *(const floatx4 *)(qs + 16 * j);
                    }
                }
            };
            // The next row block's q is on the way while one is worked on.
            floatx4 q[2][TN];
            float rw[2];
            fetch(0, q[0], rw[0]);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                if (i + 1 < RB) fetch(i + 1, q[(i + 1) & 1], rw[(i + 1) & 1]);
                __builtin_amdgcn_sched_barrier(0);
                const int m0 = (wm * RB + i) * 16;
                const int row = t.row0 + m0 + l16;
                const float w = rw[i & 1];
                float vh[TN][4], vz[TN][4], vu[TN][4], dot = 0.0f;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    float part = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float h, hz, hu;
                        act_grad<ACT>(z[i][j][e],
                                      PANELS > 1 ? z[i][j + TN * (PANELS - 1)][e] : 0.0f,
                                      h, hz, hu);
                        const float qq = q[i & 1][j][e];
                        part = fmaf(qq, h, part);
                        vh[j][e] = w * h;
                        vz[j][e] = w * qq * hz;
                        if (PANELS > 1) vu[j][e] = w * qq * hu;
                    }
                    // columns shared with the tile before count there
                    dot += 16 * j >= lo ? part : 0.0f;
                }
                dot += __shfl_xor(dot, 16, 64);
                dot += __shfl_xor(dot, 32, 64);
                if (lane < 16) p.dw_part[(size_t)row * p.dw_tiles + t.n_tile * 2 + wn] = dot;
                const size_t at = (size_t)(t.row0 + m0) * F + c0;
                bf16 *h = (bf16 *)p.h + at, *dz = (bf16 *)p.dz + at;
                bf16 *du = PANELS > 1 ? (bf16 *)p.du + at : nullptr;
                if (SMALL) {
                    store_pieces<TN>(vh, h, F, lo, hi, lane);
                    store_pieces<TN>(vz, dz, F, lo, hi, lane);
                    if (PANELS > 1) store_pieces<TN>(vu, du, F, lo, hi, lane);
                } else {
                    const int u0 = wave * 32 * TN;
                    mt::RowStore<TN> sh, sz, su;
                    sh.turn(scr, u0, vh, lane);
                    sz.turn(scr, u0, vz, lane);
                    if (PANELS > 1) su.turn(scr, u0, vu, lane);
                    sh.store(h, F, lane);
                    sz.store(dz, F, lane);
                    if (PANELS > 1) su.store(du, F, lane);
                }
                // one row block at a time: the accumulators are read as they
                // are used, not all at once
                __builtin_amdgcn_sched_barrier(0);
            }
            // (the last q, waited for above, came behind the next tile's loads:
            // these have landed; what is outstanding are the last stores)
            mt::wait_loads<SMALL ? 0 : PANELS * TN>();
        });
        if (!more) break;
        t = tn;
        src = next;
    }
    __builtin_amdgcn_s_waitcnt(0);
}

// Tiles of one matrix's gradient go in strips of 8 row tiles, so that the 32
// consecutive tiles of an XCD's round are 8 x 4 and read 12 operand panels.
// Groups are whole stages of rows, their last rows zero.
// SMALL: 128 x 128 tiles, two blocks per CU, for groups of few rows, whose
// time is the stores'.
struct WeightTile {
    int g, which, mi, ni;                // which: 0 dW1, 1 dW2, 2 dW3
};

template <bool SMALL>
__global__ __launch_bounds__(256, SMALL ? 2 : 1) void ffn_weight_grad(FfnGradParams p) {
    constexpr int B = SMALL ? 128 : 256;
    typedef mt::Tiles<B, B, 2, 2, 1, true, true> P;
    constexpr int TN = P::TN, RB = B / 32;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE], scr[SMALL ? 1 : 4 * 32 * TN];
    const int G = p.E + p.n_shared, d = p.d, F = p.d_ff;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / 2, wn = wave % 2;
    const int mats = p.act == ACT_SWIGLU ? 3 : 2;
    const int tiles = (F + B - 1) / B * ((d + B - 1) / B);      // of a matrix
    const int per_group = tiles * mats;
    const size_t mat = (size_t)F * d;
    auto tile = [&](int g, int local) __attribute__((always_inline)) {
        WeightTile t;
        t.g = g;
        int k = 0;                           // dW1, dW3, dW2
        for (; local >= tiles; local -= tiles) ++k;
        t.which = k == mats - 1 ? 1 : 2 * k;
        const int M = t.which == 1 ? d : F, N = t.which == 1 ? F : d;
        const int mtiles = (M + B - 1) / B, strip_tiles = 8 * ((N + B - 1) / B);
        const int strip = local / strip_tiles;
        const int in = local - strip * strip_tiles, sm = mtiles - strip * 8;
        t.ni = sm >= 8 ? in >> 3 : in / sm;
        t.mi = strip * 8 + in - t.ni * (sm >= 8 ? 8 : sm);
        return t;
    };
    auto result = [&](const WeightTile &t) __attribute__((always_inline)) {
        return t.which == 0 ? of_group<bf16>(p.g_w1, p.g_ws1, t.g, p.E, mat)
               : t.which == 1 ? of_group<bf16>(p.g_w2, p.g_ws2, t.g, p.E, mat)
                              : of_group<bf16>(p.g_w3, p.g_ws3, t.g, p.E, mat);
    };
    // The rounds' tiles: tile `local` of group g.  (A step adds the grid's
    // blocks, a few groups at most, without a division.)
    int g = mt::tile_of(0) / per_group, local = mt::tile_of(0) - g * per_group;
    // the first wanted tile from the one at hand on (left after it); false:
    // none
    auto find = [&](WeightTile &t) __attribute__((always_inline)) {
        while (g < G) {
            t = tile(g, local);
            local += gridDim.x;
            while (local >= per_group) {
                local -= per_group;
                ++g;
            }
            if (result(t)) return true;
        }
        return false;
    };
    auto source = [&](const WeightTile &t) __attribute__((always_inline)) {
        const int M = t.which == 1 ? d : F, N = t.which == 1 ? F : d;
        const bf16 *a = (const bf16 *)(t.which == 0 ? p.dz : t.which == 1 ? p.dys : p.du);
        const bf16 *b = (const bf16 *)(t.which == 1 ? p.h : p.xs);
        int start, rows;
        group_rows(p, t.g, start, rows);
        typename P::Source s;
        s.a = s.a2 = (uint64_t)(a + (size_t)start * M + mt::tile_start(t.mi, B, M));
        s.b = s.b2 = (uint64_t)(b + (size_t)start * N + mt::tile_start(t.ni, B, N));
        s.kt = rows / mt::SK;
        s.s0 = 0;
        return s;
    };
    auto lanes = [&](const WeightTile &t, int lane) __attribute__((always_inline)) {
        const int M = t.which == 1 ? d : F, N = t.which == 1 ? F : d;
        typename P::Lanes ln;
        ln.init(M * 2, min(M, B), N * 2, min(N, B), wave, lane);
        ln.split = 0;
        return ln;
    };
    WeightTile t;
    if (!find(t)) return;
    typename P::Source src = source(t);
    typename P::Lanes ln = lanes(t, threadIdx.x & 63);
    P::load_stage(src, ln, 0, slot0, wave);
    P::load_stage(src, ln, 1, slot1, wave);
    mt::wait_loads<0>();
    for (;;) {
        const int lane = mt::tile_lane();
        WeightTile tn = t;
        const bool more = find(tn);
        if (!more) tn = t;
        const typename P::Source next = source(tn);
        const typename P::Lanes lnext = lanes(tn, lane);
        const int M = t.which == 1 ? d : F, N = t.which == 1 ? F : d;
        bf16 *out = result(t);
        const int m0 = mt::tile_start(t.mi, B, M) + wm * RB * 16;
        const int c0 = mt::tile_start(t.ni, B, N) + wn * TN * 16;
        P::by_stages(src.kt, [&](auto kind) __attribute__((always_inline)) {
            floatx4 acc[RB][TN];
            mt::clear(acc);
            // its first stages, ahead of the last tile's stores, have landed
            mt::wait_loads<SMALL ? 0 : RB * TN / 2>();
            P::template run<RB, RB, decltype(kind)::value>(acc, src, ln, next, lnext, slot0, slot1,
                                                           wave, lane);
            mt::RowStore<SMALL ? 2 : TN> rows[2];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const int mi = m0 + i * 16;
                if (SMALL && (mi < t.mi * B || mi >= M)) continue;
                float v[TN][4];
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[j][e] = acc[i][j][e];
                bf16 *row = out + (size_t)mi * N + c0;
                if constexpr (SMALL) {
                    store_pieces<TN>(v, row, N, t.ni * B - c0, N - c0, lane);
                } else {
                    rows[i & 1].turn(scr, wave * 32 * TN, v, lane);
                    if (i > 0) rows[(i - 1) & 1].store(row - (size_t)16 * N, N, lane);
                    if (i == RB - 1) rows[i & 1].store(row, N, lane);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        });
        if (!more) break;
        t = tn;
        src = next;
        ln = lnext;
    }
    __builtin_amdgcn_s_waitcnt(0);
}

bool few_rows(const FfnGradParams &p) { return mfma_few_rows(p.routed, p.E, p.d, p.d_ff); }

// Row tiles by n columns in tiles of bn.
template <bool SMALL> int row_grid(const FfnGradParams &p, int n, int bn, int splits = 1) {
    return mt::grid_for(ffn_row_tiles(p, Shape<SMALL>::BM) * ((n + bn - 1) / bn) * splits,
                    Shape<SMALL>::BLOCKS);
}

template <bool Q, bool GATED, bool SMALL> void rows_as(const FfnGradParams &p, hipStream_t s) {
    const dim3 grid(row_grid<SMALL>(p, Q ? p.d_ff : p.d, Shape<SMALL>::BN,
                                    Q ? p.q_splits : p.dx_splits));
    if (!GATED && ((Q ? p.d : p.d_ff) / mt::SK & 1))
        hipLaunchKernelGGL((ffn_rows_by_weights<Q, GATED, GATED ? mt::EVEN : mt::ODD, SMALL>),
                           grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((ffn_rows_by_weights<Q, GATED, mt::EVEN, SMALL>), grid, dim3(256), 0,
                           s, p);
}
template <bool Q, bool GATED> void rows_by_weights(const FfnGradParams &p, hipStream_t s) {
    if (few_rows(p)) rows_as<Q, GATED, true>(p, s);
    else rows_as<Q, GATED, false>(p, s);
}

template <int ACT, bool SMALL> void act_as(const FfnGradParams &p, hipStream_t s) {
    constexpr int BN = Shape<SMALL>::BN / (ACT == ACT_SWIGLU ? 2 : 1);
    const dim3 grid(row_grid<SMALL>(p, p.d_ff, BN));
    if (p.d / mt::SK & 1)
        hipLaunchKernelGGL((ffn_act_grad<ACT, mt::ODD, SMALL>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((ffn_act_grad<ACT, mt::EVEN, SMALL>), grid, dim3(256), 0, s, p);
}
template <int ACT> void act_grad_as(const FfnGradParams &p, hipStream_t s) {
    if (few_rows(p)) act_as<ACT, true>(p, s);
    else act_as<ACT, false>(p, s);
}

}  // namespace

// Groups of at most 48 rows on average: one 64-row tile holds most of them.
// The whole gradient with the small and with the large tiles, at 48 and 64
// rows a group: 16 experts of 1024 x 2816 170 and 190 us, 187 and 203; 8 of
// 4096 x 14336 1137 and 1213, 1348 and 1292; 64 gated of 2048 x 1408 853 and
// 820, 945 and 877.  So 48 is a middle: small layers would gain from small
// tiles beyond 64 rows, many gated experts lose 4 % to them at 48.  The average
// is that of the routed groups; the shared expert's rows take the same tiles.
// And layers with an axis shorter than a large tile.
bool mfma_few_rows(long long routed, int E, int d, int d_ff) {
    return routed <= 48ll * E || d < Shape<false>::BN || d_ff < Shape<false>::BN;
}

// Ranges of K for N columns: as many as give two blocks per CU (of 256) a
// tile, each of 8 stages or more.  A split product's planes are added by
// the kernel that reads them.
int mfma_splits(long long routed, int E, int shared_rows, int N, int K) {
    if (!mfma_few_rows(routed, E, N, K)) return 1;
    const long long tiles = ((routed < E ? routed : E) + (shared_rows + 63) / 64) *
                            ((N + 127) / 128);
    long long s = tiles > 0 ? 512 / tiles : 1;
    if (s > K / (8 * mt::SK)) s = K / (8 * mt::SK);
    return (int)(s < 1 ? 1 : s > 8 ? 8 : s);
}

// Two waves side by side in each column tile of the activation gradient.
int mfma_dw_tiles(int d_ff, int act, bool few) {
    const int bn = (few ? 128 : 256) / (act == ACT_SWIGLU ? 2 : 1);
    return (d_ff + bn - 1) / bn * 2;
}

hipError_t launch_act_grad_mfma(const FfnGradParams &p, hipStream_t s) {
    rows_by_weights<true, false>(p, s);
    if (p.act == ACT_GELU) act_grad_as<ACT_GELU>(p, s);
    else if (p.act == ACT_SILU) act_grad_as<ACT_SILU>(p, s);
    else act_grad_as<ACT_SWIGLU>(p, s);
    return hipGetLastError();
}

hipError_t launch_row_grad_mfma(const FfnGradParams &p, hipStream_t s) {
    if (p.act == ACT_SWIGLU) rows_by_weights<false, true>(p, s);
    else rows_by_weights<false, false>(p, s);
    return hipGetLastError();
}

hipError_t launch_weight_grad_mfma(const FfnGradParams &p, hipStream_t s) {
    const bool few = few_rows(p);
    const int b = few ? 128 : 256;
    const long long tiles = (long long)((p.d_ff + b - 1) / b) * ((p.d + b - 1) / b);
    const int grid = mt::grid_for(tiles * (p.E + p.n_shared) * (p.act == ACT_SWIGLU ? 3 : 2),
                              few ? 2 : 1);
    if (few) hipLaunchKernelGGL(ffn_weight_grad<true>, dim3(grid), dim3(256), 0, s, p);
    else hipLaunchKernelGGL(ffn_weight_grad<false>, dim3(grid), dim3(256), 0, s, p);
    return hipGetLastError();
}
