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
//
// Here: the f32 layer's products, the bias gradients and the padding of the
// bf16 layer's groups.  f32, 4000 tokens, 4 experts of 1024 x 1024, top-2:
// 1.1 ms for the whole gradient, 76 TFLOP/s of fp32 MFMAs; the smallest layer
// (256 tokens, 8 experts of 64 x 256) is bound by the latency of its 12
// launches, 2 to 14 us each, one after the other (what depends on what is six
// or seven deep).
#include "ffn_grad.h"
#include "f32_tile.h"

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

// Block (g, c): the padding rows of group g, a c-th of their columns.  Every
// block adds up the group sizes before its own by itself.
constexpr int PAD_PARTS = 8;
__global__ __launch_bounds__(256) void pad_groups(PadParams p, int elem_bytes) {
    __shared__ int part[4];
    const int g = blockIdx.x, tid = threadIdx.x;
    constexpr int M = MOE_GRAD_ROWS - 1;
    int start = 0, rows = p.T;
    if (g < p.E) {
        // padded sizes of the groups, the sum up to this lane's in `incl`
        const int n = tid < p.E ? p.offsets[tid + 1] - p.offsets[tid] : 0;
        int incl = (n + M) & ~M;
        const int own = incl;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(incl, o, 64);
            if ((tid & 63) >= o) incl += v;
        }
        if ((tid & 63) == 63) part[tid >> 6] = incl;
        __syncthreads();
        for (int w = 0; w < (tid >> 6); ++w) incl += part[w];
        const int first = p.n_shared ? (p.T + M) & ~M : 0;
        if (g == 0 && blockIdx.y == 0 && tid < p.E) {
            p.pad[tid] = first + incl - own;
            if (tid == p.E - 1) p.pad[p.E] = first + incl;
        }
        __shared__ int mine[2];
        if (tid == g) {
            mine[0] = first + incl - own;
            mine[1] = n;
        }
        __syncthreads();
        start = mine[0];
        rows = mine[1];
    }
    const int n = ((rows + M) & ~M) - rows;
    if (n == 0) return;
    const size_t row_bytes = (size_t)p.d * elem_bytes;
    const size_t bytes = n * row_bytes, at = (size_t)(start + rows) * row_bytes;
    const u32x4 zero = {0, 0, 0, 0};
    for (size_t b = ((size_t)blockIdx.y * 256 + tid) * 16; b < bytes; b += PAD_PARTS * 256 * 16) {
        *(u32x4 *)((char *)p.xs + at + b) = zero;
        *(u32x4 *)((char *)p.dys + at + b) = zero;
    }
    if (blockIdx.y == 0 && tid < n) p.row_w[start + rows + tid] = 0.0f;
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
    r.row0 = tt.start[r.g] + m * f32t::BM;
    r.nrows = min(f32t::BM, tt.rows[r.g] - m * f32t::BM);
    return true;
}

template <int ACT>
__global__ __launch_bounds__(256) void ffn_act_grad_f32(FfnGradParams p) {
    __shared__ f32t::Stage st;
    __shared__ TileTable tt;
    const int G = p.E + p.n_shared, d = p.d, F = p.d_ff;
    build_tile_table(tt, p.offsets, p.E, p.n_shared, 0, p.T,
                     f32t::BM, F / f32t::BN);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    RowTile r;
    for (int L = blockIdx.x; row_tile(tt, G, L, r); L += gridDim.x) {
        const int n0 = r.n_tile * f32t::BN;
        const float *x = (const float *)p.xs + (size_t)r.row0 * d;
        const float *dy = (const float *)p.dys + (size_t)r.row0 * d;
        const size_t mat = (size_t)F * d;
        const float *w1 = of_group<float>(p.w1, p.ws1, r.g, p.E, mat);
        const float *w2 = of_group<float>(p.w2, p.ws2, r.g, p.E, mat);
        f32t::Acc z, u, q;
        f32t::clear(z);
        f32t::clear(u);
        f32t::clear(q);
        f32t::product<true, true>(z, st, x, d, r.nrows, w1 + (size_t)n0 * d, d,
                                  f32t::BN, d);
        if (ACT == ACT_SWIGLU) {
            const float *w3 = of_group<float>(p.w3, p.ws3, r.g, p.E, mat);
            f32t::product<true, true>(u, st, x, d, r.nrows, w3 + (size_t)n0 * d, d,
                                      f32t::BN, d);
        }
        f32t::product<true, false>(q, st, dy, d, r.nrows, w2 + n0, F, d, d);
        const float *b1 = of_group<float>(p.b1, p.bs1, r.g, p.E, F);
        const float *b3 = of_group<float>(p.b3, p.bs3, r.g, p.E, F);
        const int c0 = n0 + (wave & 1) * 32;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = (wave >> 1) * 32 + 16 * i + (lane & 15);
            const bool live = m < r.nrows;
            const int row = r.row0 + m;
            const float w = live ? p.row_w[row] : 0.0f;
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = c0 + 16 * j + 4 * (lane >> 4);
                floatx4 vh, vz, vu;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float h, hz, hu;
                    act_grad<ACT>(z[i][j][e] + (b1 ? b1[c + e] : 0.0f),
                                  u[i][j][e] + (b3 ? b3[c + e] : 0.0f), h, hz, hu);
                    dot = fmaf(q[i][j][e], h, dot);
                    const float wq = w * q[i][j][e];
                    vh[e] = w * h;
                    vz[e] = wq * hz;
                    vu[e] = wq * hu;
                }
                if (!live) continue;
                const size_t at = (size_t)row * F + c;
                *(floatx4 *)((float *)p.h + at) = vh;
                *(floatx4 *)((float *)p.dz + at) = vz;
                if (ACT == ACT_SWIGLU) *(floatx4 *)((float *)p.du + at) = vu;
            }
            dot += __shfl_xor(dot, 16, 64);
            dot += __shfl_xor(dot, 32, 64);
            if (live && lane < 16) p.dw_part[(size_t)row * p.dw_tiles + c0 / 32] = dot;
        }
    }
}

__global__ __launch_bounds__(256) void ffn_row_grad_f32(FfnGradParams p) {
    __shared__ f32t::Stage st;
    __shared__ TileTable tt;
    const int G = p.E + p.n_shared, d = p.d, F = p.d_ff;
    build_tile_table(tt, p.offsets, p.E, p.n_shared, 0, p.T,
                     f32t::BM, d / f32t::BN);
    RowTile r;
    for (int L = blockIdx.x; row_tile(tt, G, L, r); L += gridDim.x) {
        const int n0 = r.n_tile * f32t::BN;
        const size_t mat = (size_t)F * d, at = (size_t)r.row0 * F;
        f32t::Acc acc;
        f32t::clear(acc);
        f32t::product<true, false>(acc, st, (const float *)p.dz + at, F, r.nrows,
                                   of_group<float>(p.w1, p.ws1, r.g, p.E, mat) + n0, d,
                                   F, F);
        if (p.act == ACT_SWIGLU)
            f32t::product<true, false>(acc, st, (const float *)p.du + at, F, r.nrows,
                                       of_group<float>(p.w3, p.ws3, r.g, p.E, mat) + n0,
                                       d, F, F);
        f32t::each(acc, [&](int m, int c, floatx4 v) {
            if (m < r.nrows) *(floatx4 *)(p.dxs + (size_t)(r.row0 + m) * d + n0 + c) = v;
        });
    }
}

// dW[m][n] = sum over the group's rows s of L[s][m] R[s][n]; blockIdx.z:
// dW1 (dz, x), dW2 (dy, r h), dW3 (du, x).  A group without rows gets
// zeros.
__global__ __launch_bounds__(256) void ffn_weight_grad_f32(FfnGradParams p) {
    __shared__ f32t::Stage st;
    const int g = blockIdx.y, which = blockIdx.z, d = p.d, F = p.d_ff;
    const int M = which == 1 ? d : F, N = which == 1 ? F : d;
    const size_t mat = (size_t)F * d;
    float *out = which == 0 ? of_group<float>(p.g_w1, p.g_ws1, g, p.E, mat)
                 : which == 1 ? of_group<float>(p.g_w2, p.g_ws2, g, p.E, mat)
                              : of_group<float>(p.g_w3, p.g_ws3, g, p.E, mat);
    if (!out) return;
    const int m0 = blockIdx.x / (N / f32t::BN) * f32t::BM;
    const int n0 = blockIdx.x % (N / f32t::BN) * f32t::BN;
    int start, rows;
    group_rows(p, g, start, rows);
    const float *L = (const float *)(which == 0 ? p.dz : which == 1 ? p.dys : p.du);
    const float *R = (const float *)(which == 1 ? p.h : p.xs);
    f32t::Acc acc;
    f32t::clear(acc);
    f32t::product<false, false>(acc, st, L + (size_t)start * M + m0, M, rows,
                                R + (size_t)start * N + n0, N, rows, rows);
    f32t::each(acc, [&](int m, int c, floatx4 v) {
        *(floatx4 *)(out + (size_t)(m0 + m) * N + n0 + c) = v;
    });
}

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_to_f32(*p); }

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
        const float v = load1(src + (size_t)s * n);
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
    build_tile_table(tt, p.offsets, p.E, p.n_shared, 0, p.T, 4, 1);
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
                dot = fmaf(load1((const T *)p.dys + (size_t)row * p.d + c),
                           load1(b2 + c), dot);
        dot = wave_sum(dot);
        if (lane == 0) p.dw_part[(size_t)row * p.dw_tiles + p.dw_tiles - 1] = dot;
    }
}

int row_tiles(const FfnGradParams &p, int bm, int ncols) {
    const long long n = ffn_row_tiles(p, bm) * ncols;
    return (int)(n < 65536 ? n : 65536);
}

void act_grad_f32(const FfnGradParams &p, hipStream_t s) {
    const dim3 grid(row_tiles(p, f32t::BM, p.d_ff / f32t::BN)), block(256);
    if (p.act == ACT_GELU)
        hipLaunchKernelGGL((ffn_act_grad_f32<ACT_GELU>), grid, block, 0, s, p);
    else if (p.act == ACT_SILU)
        hipLaunchKernelGGL((ffn_act_grad_f32<ACT_SILU>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((ffn_act_grad_f32<ACT_SWIGLU>), grid, block, 0, s, p);
}

}  // namespace

size_t padded_rows(long long T, int n_shared, long long R, int E) {
    const long long m = MOE_GRAD_ROWS;
    const long long shared = n_shared ? (T + m - 1) / m * m : 0;
    return (size_t)(shared + R + (m - 1) * (R < E ? R : E));
}

hipError_t launch_pad_groups(const PadParams &p, int dtype, hipStream_t s) {
    hipLaunchKernelGGL(pad_groups, dim3(p.E + p.n_shared, PAD_PARTS), dim3(256), 0, s, p,
                       dtype == 1 ? 2 : 4);
    return hipGetLastError();
}

int ffn_grad_q_splits(int dtype, long long routed, int E, int shared_rows, int d, int d_ff) {
    return dtype == 1 ? mfma_splits(routed, E, shared_rows, d_ff, d) : 1;
}
int ffn_grad_dx_splits(int dtype, long long routed, int E, int shared_rows, int d, int d_ff,
                       int act) {
    return dtype == 1 ? mfma_splits(routed, E, shared_rows, d,
                                    act == ACT_SWIGLU ? 2 * d_ff : d_ff)
                      : 1;
}

int ffn_grad_dw_tiles(int dtype, int d, int d_ff, int act, long long routed, int E) {
    return dtype == 1 ? mfma_dw_tiles(d_ff, act, mfma_few_rows(routed, E, d, d_ff)) : d_ff / 32;
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
    act_grad_f32(p, s);
    return hipGetLastError();
}

hipError_t launch_ffn_row_grad(const FfnGradParams &p, int dtype,
                               hipStream_t s) {
    if (dtype == 1) return launch_row_grad_mfma(p, s);
    const dim3 grid(row_tiles(p, f32t::BM, p.d / f32t::BN));
    hipLaunchKernelGGL(ffn_row_grad_f32, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_ffn_weight_grad(const FfnGradParams &p, int dtype,
                                  hipStream_t s) {
    if (dtype == 1) return launch_weight_grad_mfma(p, s);
    const dim3 grid(p.d / f32t::BM * (p.d_ff / f32t::BN), p.E + p.n_shared,
                    p.act == ACT_SWIGLU ? 3 : 2);
    hipLaunchKernelGGL(ffn_weight_grad_f32, grid, dim3(256), 0, s, p);
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
