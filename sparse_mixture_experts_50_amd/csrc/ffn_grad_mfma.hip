// The bf16 layer's gradient GEMMs on the matrix cores (formulas in
// ffn_grad.hip, the tile product in mfma_tile.h):
//   rows by weights  q = dy W2 (fp32), and at the end dx = dz W1 + du W3
//   act grad     z = x W1^T and u = x W3^T on one output tile, then with q
//                r h, dz, du and the parts of <q, h> from the accumulators
//   weight grad  dW1 = dz^T x, dW3 = du^T x, dW2 = dy^T (r h) over the rows
//                of a group
// q passes through memory in fp32 (4 bytes a value, written and read once:
// 0.2 ms of the Mixtral-shaped 4096-token gradient) so that every product
// has a 256 x 256 tile: with z and q accumulated side by side a block's
// tile is 256 x 128, whose fragment reads take longer than its MFMAs.
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

// Writes 16 rows of a wave's TN column blocks as bf16, whole rows of
// 32 TN bytes at a time: the MFMA layout (lane: row l % 16, 4 columns from
// 4 (l / 16)) goes through the wave's own 512 TN bytes of LDS.
template <int TN>
__device__ __forceinline__ void store_rows(char *scr, const float (&v)[TN][4],
                                           bf16 *out, size_t ld, int rows,
                                           int cols, int lane) {
    constexpr int CPR = TN * 2;                  // 16-byte chunks per row
    const int l16 = lane & 15, hq = lane >> 4;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int c = (j * 2 + (hq >> 1)) ^ (l16 & (CPR - 1));
        u32x2 o;
        o.x = pack_bf16x2(v[j][0], v[j][1]);
        o.y = pack_bf16x2(v[j][2], v[j][3]);
        *(u32x2 *)(scr + l16 * (CPR * 16) + c * 16 + (hq & 1) * 8) = o;
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < CPR / 4; ++i) {
        const int r = i * (64 / CPR) + lane / CPR, c = lane % CPR;
        const u32x4 q = *(const u32x4 *)(scr + r * (CPR * 16) + ((c ^ (r & (CPR - 1))) * 16));
        if (r < rows && c * 8 < cols) *(u32x4 *)(out + (size_t)r * ld + c * 8) = q;
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// The tile of round r: persistent blocks, each XCD (block index mod 8)
// taking consecutive tiles.
__device__ __forceinline__ int tile_of(int r) {
    const int nb = gridDim.x, per = nb >> 3;
    return r * nb + (blockIdx.x & 7) * per + (blockIdx.x >> 3);
}

struct RowTile {
    int g, row0, nrows, n_tile;
};
template <int BM>
__device__ __forceinline__ RowTile row_tile(const TileTable &tt, int G, int L) {
    RowTile r;
    r.g = __builtin_amdgcn_readfirstlane(find_group(tt, G, L));
    const int local = L - __builtin_amdgcn_readfirstlane(tt.base[r.g]);
    const int mt = __builtin_amdgcn_readfirstlane(tt.mt[r.g]);
    r.n_tile = local / mt;
    const int m = local - r.n_tile * mt;
    r.row0 = __builtin_amdgcn_readfirstlane(tt.start[r.g]) + m * BM;
    r.nrows = min(BM, __builtin_amdgcn_readfirstlane(tt.rows[r.g]) - m * BM);
    return r;
}

// out[rows][N] (fp32) = the sum of one or two products A B of a group's rows
// with its weights, stored along K.  Q: q = dy W2; else dx = dz W1 + du W3.
template <int RB, int TN, int WM, int WN, bool Q, bool ODD>
__global__ __launch_bounds__(256, 1) void ffn_rows_by_weights(FfnGradParams p) {
    typedef mt::Product<RB, TN, WM, WN, 1, false, true, false, ODD> P;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE];
    __shared__ TileTable tt;
    const int G = p.E + p.n_shared;
    const int N = Q ? p.d_ff : p.d, K = Q ? p.d : p.d_ff;
    build_tile_table(tt, p.offsets, p.E, p.n_shared, p.shared_base, p.T, P::BM,
                     (N + P::BN - 1) / P::BN);
    const int total = __builtin_amdgcn_readfirstlane(tt.base[G]);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    for (int r = 0;; ++r) {
        const int L = tile_of(r);
        if (L >= total) break;
        // opaque, so that per-lane addresses are not kept across tiles
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63;
        const RowTile t = row_tile<P::BM>(tt, G, L);
        const int n0 = t.n_tile * P::BN;
        const size_t mat = (size_t)p.d_ff * p.d, at = (size_t)t.row0 * K;
        mt::Operand a = {(const char *)((const bf16 *)(Q ? p.dys : p.dz) + at), nullptr,
                         (size_t)K * 2, t.nrows, 0};
        mt::Operand b = {(const char *)(of_group<bf16>(Q ? p.w2 : p.w1, Q ? p.ws2 : p.ws1,
                                                       t.g, p.E, mat) + n0),
                         nullptr, (size_t)N * 2, min(P::BN, N - n0), 0};
        floatx4 acc[RB][TN];
        mt::clear(acc);
        P::run(acc, a, b, slot0, slot1, K / mt::SK, wave, lane);
        if (!Q && p.act == ACT_SWIGLU) {
            a.base = (const char *)((const bf16 *)p.du + at);
            b.base = (const char *)(of_group<bf16>(p.w3, p.ws3, t.g, p.E, mat) + n0);
            P::run(acc, a, b, slot0, slot1, K / mt::SK, wave, lane);
        }
        const int l16 = lane & 15, c0 = n0 + wn * TN * 16;
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int m = (wm * RB + i) * 16 + l16;
            if (m >= t.nrows) continue;
            float *out = (Q ? p.q : p.dxs) + (size_t)(t.row0 + m) * N + c0 + 4 * (lane >> 4);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                if (c0 + 16 * j < N) *(floatx4 *)(out + 16 * j) = acc[i][j];
        }
    }
}

// z (and u) of a tile, then with q: r h, dz, du and the parts of <q, h>.  A
// gated tile has TN column blocks of z and the same TN of u per wave.
template <int RB, int TN, int WM, int WN, int ACT, bool ODD>
__global__ __launch_bounds__(256, 1) void ffn_act_grad(FfnGradParams p) {
    constexpr int PANELS = ACT == ACT_SWIGLU ? 2 : 1;
    typedef mt::Product<RB, TN, WM, WN, PANELS, false, false, false, ODD> P;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE];
    __shared__ TileTable tt;
    const int G = p.E + p.n_shared, d = p.d, F = p.d_ff;
    build_tile_table(tt, p.offsets, p.E, p.n_shared, p.shared_base, p.T, P::BM,
                     (F + P::BN - 1) / P::BN);
    const int total = __builtin_amdgcn_readfirstlane(tt.base[G]);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    for (int r = 0;; ++r) {
        const int L = tile_of(r);
        if (L >= total) break;
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63;
        const RowTile t = row_tile<P::BM>(tt, G, L);
        const int n0 = t.n_tile * P::BN;
        const size_t mat = (size_t)F * d;
        const bf16 *w1 = of_group<bf16>(p.w1, p.ws1, t.g, p.E, mat);
        const bf16 *w3 = PANELS > 1 ? of_group<bf16>(p.w3, p.ws3, t.g, p.E, mat) : w1;
        const mt::Operand a = {(const char *)((const bf16 *)p.xs + (size_t)t.row0 * d),
                               nullptr, (size_t)d * 2, t.nrows, 0};
        const mt::Operand b = {(const char *)(w1 + (size_t)n0 * d),
                               (const char *)(w3 + (size_t)n0 * d), (size_t)d * 2,
                               min(P::BN, F - n0), 0};
        const int l16 = lane & 15, c0 = n0 + wn * TN * 16;
        const int cols = F - c0;             // columns of this wave
        const int cq = c0 + 4 * (lane >> 4);
        // the sums start from the biases
        floatx4 z[RB][TN * PANELS];
        mt::clear(z);
        const bf16 *bias[2] = {of_group<bf16>(p.b1, p.bs1, t.g, p.E, F),
                               PANELS > 1 ? of_group<bf16>(p.b3, p.bs3, t.g, p.E, F) : nullptr};
#pragma unroll
        for (int k = 0; k < PANELS; ++k)
            if (bias[k]) {
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    if (16 * j >= cols) continue;    // whole blocks: F % 64 == 0
                    const u32x2 v = *(const u32x2 *)(bias[k] + cq + 16 * j);
                    const floatx4 f = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
#pragma unroll
                    for (int i = 0; i < RB; ++i) z[i][k * TN + j] = f;
                }
            }
        P::run(z, a, b, slot0, slot1, d / mt::SK, wave, lane);
        __builtin_amdgcn_s_waitcnt(0);
        __builtin_amdgcn_s_barrier();        // the slots are free
        if (cols <= 0) continue;
        char *scr = (char *)slot0 + wave * (TN * 512);
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int m0 = (wm * RB + i) * 16;
            const int rows = t.nrows - m0;
            if (rows <= 0) continue;
            // rows past the group's end read its last row and store nothing
            const int row = t.row0 + m0 + min(l16, rows - 1);
            const float w = p.row_w[row];
            const float *qp = p.q + (size_t)row * F + cq;
            floatx4 q[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j)
                q[j] = *(const floatx4 *)(qp + (16 * j < cols ? 16 * j : 0));
            float vh[TN][4], vz[TN][4], vu[TN][4], dot = 0.0f;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const float in = 16 * j < cols ? 1.0f : 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float h, hz, hu;
                    act_grad<ACT>(z[i][j][e],
                                  PANELS > 1 ? z[i][j + TN * (PANELS - 1)][e] : 0.0f, h,
                                  hz, hu);
                    const float qq = q[j][e] * in;
                    dot = fmaf(qq, h, dot);
                    vh[j][e] = w * h;
                    vz[j][e] = w * qq * hz;
                    if (PANELS > 1) vu[j][e] = w * qq * hu;
                }
            }
            dot += __shfl_xor(dot, 16, 64);
            dot += __shfl_xor(dot, 32, 64);
            if (lane < 16 && l16 < rows)
                p.dw_part[(size_t)row * p.dw_tiles + c0 / (TN * 16)] = dot;
            const size_t at = (size_t)(t.row0 + m0) * F + c0;
            store_rows<TN>(scr, vh, (bf16 *)p.h + at, F, rows, cols, lane);
            store_rows<TN>(scr, vz, (bf16 *)p.dz + at, F, rows, cols, lane);
            if (PANELS > 1) store_rows<TN>(scr, vu, (bf16 *)p.du + at, F, rows, cols, lane);
            // one row block at a time: the accumulators are read as they are
            // used, not all at once
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// Tiles of one matrix's gradient go in strips of 8 row tiles, so that the 32
// consecutive tiles of an XCD's round are 8 x 4 and read 12 operand panels.
template <int RB, int TN, int WM, int WN>
__global__ __launch_bounds__(256, 1) void ffn_weight_grad(FfnGradParams p) {
    typedef mt::Product<RB, TN, WM, WN, 1, true, true, true, false> P;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE];
    const int G = p.E + p.n_shared, d = p.d, F = p.d_ff;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int mats = p.act == ACT_SWIGLU ? 3 : 2;
    const int t_up = (F + P::BM - 1) / P::BM * ((d + P::BN - 1) / P::BN);
    const int t_down = (d + P::BM - 1) / P::BM * ((F + P::BN - 1) / P::BN);
    const int per_group = t_down + (mats - 1) * t_up;
    const long long total = (long long)G * per_group;
    for (int r = 0;; ++r) {
        const long long L = (long long)r * gridDim.x + tile_of(0);
        if (L >= total) break;
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63;
        const int g = (int)(L / per_group);
        int local = (int)(L - (long long)g * per_group);
        // dW1, dW3 (F x d), then dW2 (d x F)
        int which = 0;
        if (local >= t_up * (mats - 1)) {
            which = 1;
            local -= t_up * (mats - 1);
        } else if (local >= t_up) {
            which = 2;
            local -= t_up;
        }
        const int M = which == 1 ? d : F, N = which == 1 ? F : d;
        const int mtiles = (M + P::BM - 1) / P::BM, ntiles = (N + P::BN - 1) / P::BN;
        const int strip = local / (8 * ntiles), in = local - strip * 8 * ntiles;
        const int sm = min(8, mtiles - strip * 8);
        const int m0 = (strip * 8 + in % sm) * P::BM, n0 = in / sm * P::BN;
        const size_t mat = (size_t)F * d;
        bf16 *out = which == 0 ? of_group<bf16>(p.g_w1, p.g_ws1, g, p.E, mat)
                    : which == 1 ? of_group<bf16>(p.g_w2, p.g_ws2, g, p.E, mat)
                                 : of_group<bf16>(p.g_w3, p.g_ws3, g, p.E, mat);
        if (!out) continue;
        int start, rows;
        group_rows(p, g, start, rows);
        start = __builtin_amdgcn_readfirstlane(start);
        rows = __builtin_amdgcn_readfirstlane(rows);
        const bf16 *A = (const bf16 *)(which == 0 ? p.dz : which == 1 ? p.dys : p.du);
        const bf16 *B = (const bf16 *)(which == 1 ? p.h : p.xs);
        const mt::Operand a = {(const char *)(A + (size_t)start * M + m0), nullptr,
                               (size_t)M * 2, min(P::BM, M - m0), rows};
        const mt::Operand b = {(const char *)(B + (size_t)start * N + n0), nullptr,
                               (size_t)N * 2, min(P::BN, N - n0), rows};
        floatx4 acc[RB][TN];
        mt::clear(acc);
        // whole pairs of stages: rows past the group's end are zeros
        P::run(acc, a, b, slot0, slot1, (rows + 2 * mt::SK - 1) / (2 * mt::SK) * 2,
               wave, lane);
        __builtin_amdgcn_s_waitcnt(0);
        __builtin_amdgcn_s_barrier();
        const int c0 = n0 + wn * TN * 16;
        char *scr = (char *)slot0 + wave * (TN * 512);
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int mi = m0 + (wm * RB + i) * 16;
            if (mi >= M || c0 >= N) continue;
            float v[TN][4];
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j][e] = acc[i][j][e];
            store_rows<TN>(scr, v, out + (size_t)mi * N + c0, N, 16, N - c0, lane);
        }
        // run() of the next tile waits for every wave before it loads
    }
}

int cus() {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        n < 8)
        return 256;
    return n / 8 * 8;
}

int grid_for(long long tiles) {
    const int n = cus();
    const long long g = (tiles + 7) / 8 * 8;
    return (int)(g < n ? (g < 8 ? 8 : g) : n);
}

template <int RB, int TN, int WM, int WN, int ACT>
void act_as(const FfnGradParams &p, hipStream_t s) {
    const int grid = grid_for(ffn_row_tiles(p, RB * 16 * WM) *
                              ((p.d_ff + TN * 16 * WN - 1) / (TN * 16 * WN)));
    if (p.d / mt::SK & 1)
        hipLaunchKernelGGL((ffn_act_grad<RB, TN, WM, WN, ACT, true>), dim3(grid), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((ffn_act_grad<RB, TN, WM, WN, ACT, false>), dim3(grid), dim3(256), 0, s, p);
}

template <int RB, int TN, int WM, int WN, bool Q>
void rows_as(const FfnGradParams &p, hipStream_t s) {
    const int N = Q ? p.d_ff : p.d, bn = TN * 16 * WN;
    const int grid = grid_for(ffn_row_tiles(p, RB * 16 * WM) * ((N + bn - 1) / bn));
    if ((Q ? p.d : p.d_ff) / mt::SK & 1)
        hipLaunchKernelGGL((ffn_rows_by_weights<RB, TN, WM, WN, Q, true>), dim3(grid), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((ffn_rows_by_weights<RB, TN, WM, WN, Q, false>), dim3(grid), dim3(256), 0, s, p);
}

}  // namespace

// Columns of a wave's tile: 64 gated, 128 else.
int mfma_dw_tiles(int d_ff, int act) {
    return act == ACT_SWIGLU ? d_ff / 64 : (d_ff + 127) / 128;
}

hipError_t launch_act_grad_mfma(const FfnGradParams &p, hipStream_t s) {
    rows_as<8, 8, 2, 2, true>(p, s);
    if (p.act == ACT_GELU) act_as<8, 8, 2, 2, ACT_GELU>(p, s);
    else if (p.act == ACT_SILU) act_as<8, 8, 2, 2, ACT_SILU>(p, s);
    else act_as<8, 4, 2, 2, ACT_SWIGLU>(p, s);
    return hipGetLastError();
}

hipError_t launch_row_grad_mfma(const FfnGradParams &p, hipStream_t s) {
    rows_as<8, 8, 2, 2, false>(p, s);
    return hipGetLastError();
}

hipError_t launch_weight_grad_mfma(const FfnGradParams &p, hipStream_t s) {
    const long long up = (long long)((p.d_ff + 255) / 256) * ((p.d + 255) / 256);
    const int grid = grid_for(up * (p.E + p.n_shared) * (p.act == ACT_SWIGLU ? 3 : 2));
    hipLaunchKernelGGL((ffn_weight_grad<8, 8, 2, 2>), dim3(grid), dim3(256), 0, s, p);
    return hipGetLastError();
}
