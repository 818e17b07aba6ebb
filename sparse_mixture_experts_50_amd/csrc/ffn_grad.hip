// Gradient of the grouped expert FFNs.  With z = W1 x + b1 (u = W3 x + b3
// for SwiGLU), h = act(z) (times u), a row of routing weight r and output
// gradient dy, the expert's output W2 h + b2 entering y as r (W2 h + b2):
//   q  = W2^T dy                      (before the routing weight)
//   dr = <q, h> + <dy, b2>
//   dz = r q * dh/dz,  du = r q * dh/du
//   dx = W1^T dz + W3^T du
//   dW1 = dz x^T, dW3 = du x^T, dW2 = dy (r h)^T, db1 = dz, db3 = du,
//   db2 = r dy, summed over the group's rows.
// ("AI-Research-SKILLs MoE training guide", sec. 6.1 and "The expert group
// activated per token", sec. 3.1 give the FFN; this is its derivative.)
//
// The row weight multiplies h and q rather than dy, so the dispatched dy
// rows stay exactly the caller's values, and dr needs no expert outputs:
// the backward reads nothing of the forward but the routing.  z and u are
// computed again from x (2 or 4 d d_ff operations a row) instead of being
// kept by the forward (4 or 8 bytes a value, written and read).
#include "ffn_grad.h"
#include "simt.h"

namespace {

// h, dh/dz and dh/du at z, u, with the accurate library functions.
template <int ACT>
__device__ __forceinline__ void act_grad(float z, float u, float &h, float &hz,
                                         float &hu) {
    if (ACT == ACT_GELU) {
        // z Phi(z), Phi + z phi
        const float cdf = 0.5f * erfcf(z * -0.70710678f);
        h = z * cdf;
        hz = fmaf(z * 0.39894228f, expf(-0.5f * z * z), cdf);
        hu = 0.0f;
    } else {
        const float sg = 1.0f / (1.0f + expf(-z));
        const float a = z * sg;
        const float da = fmaf(a, 1.0f - sg, sg);
        if (ACT == ACT_SILU) {
            h = a;
            hz = da;
            hu = 0.0f;
        } else {
            h = a * u;
            hz = da * u;
            hu = a;
        }
    }
}

// Row tiles: 64 rows of one group by 64 columns.
struct RowTile {
    int g, row0, nrows, n_tile;
};
__device__ __forceinline__ bool row_tile(const TileTable &tt, int G, int L,
                                         RowTile &r) {
    if (L >= tt.base[G]) return false;
    r.g = find_group(tt, G, L);
    const int local = L - tt.base[r.g], mt = tt.mt[r.g];
    r.n_tile = local / mt;
    const int m = local - r.n_tile * mt;
    r.row0 = tt.start[r.g] + m * simt::BM;
    r.nrows = min(simt::BM, tt.rows[r.g] - m * simt::BM);
    return true;
}

template <typename T, int ACT>
__global__ __launch_bounds__(256) void ffn_act_grad_simt(FfnGradParams p) {
    __shared__ simt::Stage st;
    __shared__ TileTable tt;
    const int G = p.E + p.n_shared, d = p.d, F = p.d_ff;
    build_tile_table(tt, p.offsets, p.E, p.n_shared, p.shared_base, p.T,
                     simt::BM, F / simt::BN);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    RowTile r;
    for (int L = blockIdx.x; row_tile(tt, G, L, r); L += gridDim.x) {
        const int n0 = r.n_tile * simt::BN;
        const T *x = (const T *)p.xs + (size_t)r.row0 * d;
        const T *dy = (const T *)p.dys + (size_t)r.row0 * d;
        const size_t mat = (size_t)F * d;
        const T *w1 = of_group<T>(p.w1, p.ws1, r.g, p.E, mat);
        const T *w2 = of_group<T>(p.w2, p.ws2, r.g, p.E, mat);
        float z[4][4], u[4][4], q[4][4];
        simt::clear(z);
        simt::clear(u);
        simt::clear(q);
        simt::product<true, true>(z, st, x, d, r.nrows, w1 + (size_t)n0 * d, d,
                                  simt::BN, d);
        if (ACT == ACT_SWIGLU) {
            const T *w3 = of_group<T>(p.w3, p.ws3, r.g, p.E, mat);
            simt::product<true, true>(u, st, x, d, r.nrows,
                                      w3 + (size_t)n0 * d, d, simt::BN, d);
        }
        simt::product<true, false>(q, st, dy, d, r.nrows, w2 + n0, F, d, d);
        const T *b1 = of_group<T>(p.b1, p.bs1, r.g, p.E, F);
        const T *b3 = of_group<T>(p.b3, p.bs3, r.g, p.E, F);
        const int c = n0 + tx * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = ty * 4 + i;
            const bool live = m < r.nrows;
            const int row = r.row0 + m;
            const float w = live ? p.row_w[row] : 0.0f;
            float vh[4], vz[4], vu[4], dot = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float h, hz, hu;
                const float zz = z[i][j] + (b1 ? simt::load1(b1 + c + j) : 0.0f);
                const float uu = u[i][j] + (b3 ? simt::load1(b3 + c + j) : 0.0f);
                act_grad<ACT>(zz, uu, h, hz, hu);
                dot = fmaf(q[i][j], h, dot);
                const float wq = w * q[i][j];
                vh[j] = w * h;
                vz[j] = wq * hz;
                vu[j] = wq * hu;
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) dot += __shfl_xor(dot, o, 64);
            if (!live) continue;
            const size_t at = (size_t)row * F + c;
            simt::store4((T *)p.h + at, vh);
            simt::store4((T *)p.dz + at, vz);
            if (ACT == ACT_SWIGLU) simt::store4((T *)p.du + at, vu);
            if (tx == 0) p.dw_part[(size_t)row * p.dw_tiles + r.n_tile] = dot;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void ffn_row_grad_simt(FfnGradParams p) {
    __shared__ simt::Stage st;
    __shared__ TileTable tt;
    const int G = p.E + p.n_shared, d = p.d, F = p.d_ff;
    build_tile_table(tt, p.offsets, p.E, p.n_shared, p.shared_base, p.T,
                     simt::BM, d / simt::BN);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    RowTile r;
    for (int L = blockIdx.x; row_tile(tt, G, L, r); L += gridDim.x) {
        const int n0 = r.n_tile * simt::BN;
        const size_t mat = (size_t)F * d, at = (size_t)r.row0 * F;
        float acc[4][4];
        simt::clear(acc);
        simt::product<true, false>(
            acc, st, (const T *)p.dz + at, F, r.nrows,
            of_group<T>(p.w1, p.ws1, r.g, p.E, mat) + n0, d, F, F);
        if (p.act == ACT_SWIGLU)
            simt::product<true, false>(
                acc, st, (const T *)p.du + at, F, r.nrows,
                of_group<T>(p.w3, p.ws3, r.g, p.E, mat) + n0, d, F, F);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = ty * 4 + i;
            if (m < r.nrows)
                simt::store4(p.dxs + (size_t)(r.row0 + m) * d + n0 + tx * 4, acc[i]);
        }
    }
}

// dW[m][n] = sum over the group's rows s of L[s][m] R[s][n]; blockIdx.z:
// dW1 (dz, x), dW2 (dy, r h), dW3 (du, x).  A group without rows gets
// zeros.
template <typename T>
__global__ __launch_bounds__(256) void ffn_weight_grad_simt(FfnGradParams p) {
    __shared__ simt::Stage st;
    const int g = blockIdx.y, which = blockIdx.z, d = p.d, F = p.d_ff;
    const int M = which == 1 ? d : F, N = which == 1 ? F : d;
    const size_t mat = (size_t)F * d;
    T *out = which == 0 ? of_group<T>(p.g_w1, p.g_ws1, g, p.E, mat)
             : which == 1 ? of_group<T>(p.g_w2, p.g_ws2, g, p.E, mat)
                          : of_group<T>(p.g_w3, p.g_ws3, g, p.E, mat);
    if (!out) return;
    const int m0 = blockIdx.x / (N / simt::BN) * simt::BM;
    const int n0 = blockIdx.x % (N / simt::BN) * simt::BN;
    int start, rows;
    group_rows(p, g, start, rows);
    const T *L = (const T *)(which == 0 ? p.dz : which == 1 ? p.dys : p.du);
    const T *R = (const T *)(which == 1 ? p.h : p.xs);
    float acc[4][4];
    simt::clear(acc);
    simt::product<false, false>(acc, st, L + (size_t)start * M + m0, M, rows,
                                R + (size_t)start * N + n0, N, rows, rows);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        simt::store4(out + (size_t)(m0 + ty * 4 + i) * N + n0 + tx * 4, acc[i]);
}

// Column sums over a group's rows; blockIdx.z: db1 (dz), db2 (r dy), db3
// (du).  64 columns per block, 16 row lanes added in order.
template <typename T>
__global__ __launch_bounds__(1024) void ffn_bias_grad(FfnGradParams p) {
    __shared__ float part[16][64];
    const int g = blockIdx.y, which = blockIdx.z;
    const int n = which == 1 ? p.d : p.d_ff;
    const int lane = threadIdx.x & 63, rl = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    T *out = which == 0 ? of_group<T>(p.g_b1, p.g_bs1, g, p.E, n)
             : which == 1 ? of_group<T>(p.g_b2, p.g_bs2, g, p.E, n)
                          : of_group<T>(p.g_b3, p.g_bs3, g, p.E, n);
    if (!out || blockIdx.x * 64 >= n) return;
    int start, rows;
    group_rows(p, g, start, rows);
    const T *src = (const T *)(which == 0 ? p.dz : which == 1 ? p.dys : p.du) +
                   (size_t)start * n + c;
    float sum = 0.0f;
#pragma unroll 4
    for (int s = rl; s < rows; s += 16) {
        const float v = simt::load1(src + (size_t)s * n);
        sum = which == 1 ? fmaf(p.row_w[start + s], v, sum) : sum + v;
    }
    part[rl][lane] = sum;
    __syncthreads();
    if (rl) return;
    for (int i = 1; i < 16; ++i) sum += part[i][lane];
    if (sizeof(T) == 2)
        ((uint16_t *)out)[c] = (uint16_t)f32_to_bf16_bits(sum);
    else
        ((float *)out)[c] = sum;
}

// <dy, b2> of every row, into the last column of dw_part.
template <typename T>
__global__ __launch_bounds__(256) void ffn_bias_dot(FfnGradParams p) {
    __shared__ TileTable tt;
    const int G = p.E + p.n_shared;
    build_tile_table(tt, p.offsets, p.E, p.n_shared, p.shared_base, p.T, 4, 1);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int L = blockIdx.x; L < tt.base[G]; L += gridDim.x) {
        const int g = find_group(tt, G, L);
        const int r = (L - tt.base[g]) * 4 + wave;
        if (r >= tt.rows[g]) continue;
        const int row = tt.start[g] + r;
        const T *b2 = of_group<T>(p.b2, p.bs2, g, p.E, p.d);
        float dot = 0.0f;
        if (b2)
            for (int c = lane; c < p.d; c += 64)
                dot = fmaf(simt::load1((const T *)p.dys + (size_t)row * p.d + c),
                           simt::load1(b2 + c), dot);
        dot = wave_sum(dot);
        if (lane == 0) p.dw_part[(size_t)row * p.dw_tiles + p.dw_tiles - 1] = dot;
    }
}

int row_tiles(const FfnGradParams &p, int bm, int ncols) {
    const long long n = ffn_row_tiles(p, bm) * ncols;
    return (int)(n < 65536 ? n : 65536);
}

template <typename T>
void act_grad_simt(const FfnGradParams &p, hipStream_t s) {
    const dim3 grid(row_tiles(p, simt::BM, p.d_ff / simt::BN)), block(256);
    if (p.act == ACT_GELU)
        hipLaunchKernelGGL((ffn_act_grad_simt<T, ACT_GELU>), grid, block, 0, s, p);
    else if (p.act == ACT_SILU)
        hipLaunchKernelGGL((ffn_act_grad_simt<T, ACT_SILU>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((ffn_act_grad_simt<T, ACT_SWIGLU>), grid, block, 0, s, p);
}

}  // namespace

int ffn_grad_dw_tiles(int dtype, int d_ff, int act) {
    return dtype == 1 ? mfma_dw_tiles(d_ff, act) : d_ff / simt::BN;
}

hipError_t launch_ffn_act_grad(const FfnGradParams &p, int dtype,
                               hipStream_t s) {
    if (p.b2 || p.bs2) {
        const dim3 grid(row_tiles(p, 4, 1));
        if (dtype == 1)
            hipLaunchKernelGGL((ffn_bias_dot<uint16_t>), grid, dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL((ffn_bias_dot<float>), grid, dim3(256), 0, s, p);
    }
    if (dtype == 1) return launch_act_grad_mfma(p, s);
    act_grad_simt<float>(p, s);
    return hipGetLastError();
}

hipError_t launch_ffn_row_grad(const FfnGradParams &p, int dtype,
                               hipStream_t s) {
    if (dtype == 1) return launch_row_grad_mfma(p, s);
    const dim3 grid(row_tiles(p, simt::BM, p.d / simt::BN));
    hipLaunchKernelGGL((ffn_row_grad_simt<float>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_ffn_weight_grad(const FfnGradParams &p, int dtype,
                                  hipStream_t s) {
    if (dtype == 1) return launch_weight_grad_mfma(p, s);
    const dim3 grid(p.d / simt::BM * (p.d_ff / simt::BN), p.E + p.n_shared,
                    p.act == ACT_SWIGLU ? 3 : 2);
    hipLaunchKernelGGL((ffn_weight_grad_simt<float>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_ffn_bias_grad(const FfnGradParams &p, int dtype,
                                hipStream_t s) {
    const int widest = p.d > p.d_ff ? p.d : p.d_ff;
    const dim3 grid(widest / 64, p.E + p.n_shared, p.act == ACT_SWIGLU ? 3 : 2);
    if (dtype == 1)
        hipLaunchKernelGGL((ffn_bias_grad<uint16_t>), grid, dim3(1024), 0, s, p);
    else
        hipLaunchKernelGGL((ffn_bias_grad<float>), grid, dim3(1024), 0, s, p);
    return hipGetLastError();
}
