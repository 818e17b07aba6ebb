// Small kernels around the dense layer's products: bias gradients (and in the
// same launch the last rows copied beside zeros), and the epilogue of products whose sums lie in
// planes.  All bound by memory.
#include "act.h"
#include "dense.h"

namespace {

// Rows copied, and rows zeroed after them, by all blocks of a plane of the grid.
__device__ void copy_tail(const DenseTails::Item &t) {
    const size_t bytes = (size_t)t.row_bytes * t.rows, copied = (size_t)t.row_bytes * t.copied;
    const size_t first = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
    for (size_t b = (first * 256 + threadIdx.x) * 16; b < bytes;
         b += (size_t)gridDim.x * gridDim.y * 256 * 16)
        *(u32x4 *)((char *)t.dst + b) =
            b < copied ? *(const u32x4 *)((const char *)t.src + b) : u32x4{0, 0, 0, 0};
}

// Eight (fp32: four) columns of a row as fp32.
template <typename T> struct Vec {
    static constexpr int N = sizeof(T) == 2 ? 8 : 4;
    float v[N];
    __device__ __forceinline__ void load(const T *p) {
        const u32x4 q = *(const u32x4 *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (N == 8) {
                v[2 * i] = bf16_lo(q[i]);
                v[2 * i + 1] = bf16_hi(q[i]);
            } else {
                v[i] = __uint_as_float(q[i]);
            }
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = N == 8 ? pack_bf16x2(v[(2 * i) % N], v[(2 * i + 1) % N])
                          : __float_as_uint(v[i]);
        *(u32x4 *)p = q;
    }
    // += N fp32 values
    __device__ __forceinline__ void add(const float *p) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const floatx4 q = *(const floatx4 *)(p + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i + e] += q[e];
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
    }
};

// Block (c, r, k): columns [256 c, 256 c + 256) (fp32: 128) of range r of
// item k, eight rows side by side; one range: the result itself.  Items after
// the sums' are tails.
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t *p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }

template <typename T>
__global__ __launch_bounds__(256) void dense_sums(DenseSums p, DenseTails tails) {
    if ((int)blockIdx.z >= p.count) {
        copy_tail(tails.t[blockIdx.z - p.count]);
        return;
    }
    constexpr int N = Vec<T>::N;
    __shared__ float red[8][32 * N];
    const DenseSums::Item &t = p.t[blockIdx.z];
    const int col = threadIdx.x & 31, lane = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + col) * N;
    if (blockIdx.x * 32 * N >= t.C) return;
    const int m0 = blockIdx.y * MOE_DENSE_SUM_ROWS, m1 = min(p.M, m0 + MOE_DENSE_SUM_ROWS);
    Vec<T> sum, x;
    sum.clear();
    if (c < t.C)
#pragma unroll 4
        for (int m = m0 + lane; m < m1; m += 8) {
            x.load((const T *)t.src + (size_t)m * t.C + c);
#pragma unroll
            for (int i = 0; i < N; ++i) sum.v[i] += x.v[i];
        }
#pragma unroll
    for (int i = 0; i < N; ++i) red[lane][col * N + i] = sum.v[i];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * N; i += 256) {
        float s = 0.0f;
#pragma unroll
        for (int l = 0; l < 8; ++l) s += red[l][i];
        const int at = blockIdx.x * 32 * N + i;
        if (at >= t.C) continue;
        if (gridDim.y == 1) put((T *)t.out + at, s);
        else t.part[(size_t)blockIdx.y * t.C + at] = s;
    }
}
// 64 columns by four ranges at a time.
template <typename T> __global__ __launch_bounds__(256) void dense_sums_join(DenseSums p) {
    __shared__ float red[4][64];
    const DenseSums::Item &t = p.t[blockIdx.y];
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), lane = threadIdx.x >> 6;
    const int ranges = dense_sum_ranges(p.M);
    if (blockIdx.x * 64 >= t.C) return;
    float s = 0.0f;
    for (int r = lane; r < ranges; r += 4) s += t.part[(size_t)r * t.C + c];
    red[lane][threadIdx.x & 63] = s;
    __syncthreads();
    if (lane) return;
    s = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
    put((T *)t.out + c, s);
}

// y = res + act(sums + bias), or h, dz, du: one vector of a row a thread.
template <typename T, int EPI, int ACT>
__global__ __launch_bounds__(256) void dense_finish(DenseRows p) {
    constexpr int N = Vec<T>::N, PANELS = act_gated(ACT) ? 2 : 1;
    constexpr bool FAST = sizeof(T) == 2;
    const size_t plane = (size_t)p.M * p.N;
    const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * N;
    if (at >= plane) return;
    const int c = (int)(at % p.N);
    Vec<T> z, u, a, o;
    z.clear();
    u.clear();
#pragma unroll 4
    for (int s = 0; s < p.plan.splits; ++s) {
        const float *q = p.plane + (size_t)s * PANELS * plane + at;
        z.add(q);
        if (PANELS > 1) u.add(q + plane);
    }
    if (p.bias) {
        a.load((const T *)p.bias + c);
#pragma unroll
        for (int i = 0; i < N; ++i) z.v[i] += a.v[i];
    }
    if (PANELS > 1 && p.bias2) {
        a.load((const T *)p.bias2 + c);
#pragma unroll
        for (int i = 0; i < N; ++i) u.v[i] += a.v[i];
    }
    if (EPI == DENSE_FORWARD) {
        a.clear();
        if (p.res) a.load((const T *)p.res + at);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            o.v[i] = act_value<ACT, FAST>(z.v[i], u.v[i]);
            if (p.res) o.v[i] += a.v[i];
        }
        o.store((T *)p.y + at);
        return;
    }
    if (p.dy) {
        a.load((const T *)p.dy + at);
    } else {
        a.clear();
        for (int s = 0; s < p.q_planes; ++s) a.add(p.q + (size_t)s * plane + at);
    }
    Vec<T> h, du;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float hz, hu;
        act_grad<ACT, FAST>(z.v[i], u.v[i], h.v[i], hz, hu);
        o.v[i] = a.v[i] * hz;
        du.v[i] = a.v[i] * hu;
    }
    o.store((T *)p.dz + at);
    if (PANELS > 1) du.store((T *)p.du + at);
    if (p.h) h.store((T *)p.h + at);
}

// The planes of weight gradients, added up: block row k is matrix k.
template <typename T> __global__ __launch_bounds__(256) void dense_weight_finish(DenseWeights p) {
    constexpr int N = Vec<T>::N;
    const DenseMat &m = p.m[blockIdx.y];
    const size_t size = (size_t)m.R * m.C;
    const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * N;
    if (at >= size) return;
    Vec<T> s;
    s.clear();
#pragma unroll 4
    for (int i = 0; i < p.splits; ++i) s.add(p.plane + p.offset[blockIdx.y] + i * size + at);
    s.store((T *)m.out + at);
}

template <typename T, int EPI> void finish_as(const DenseRows &p, hipStream_t s) {
    const long long vectors = (long long)p.M * p.N / Vec<T>::N;
    const dim3 grid((unsigned)((vectors + 255) / 256)), block(256);
    switch (p.act) {
    case ACT_GELU: hipLaunchKernelGGL((dense_finish<T, EPI, ACT_GELU>), grid, block, 0, s, p); break;
    case ACT_SILU: hipLaunchKernelGGL((dense_finish<T, EPI, ACT_SILU>), grid, block, 0, s, p); break;
    case ACT_SWIGLU:
        hipLaunchKernelGGL((dense_finish<T, EPI, ACT_SWIGLU>), grid, block, 0, s, p);
        break;
    case ACT_GEGLU: hipLaunchKernelGGL((dense_finish<T, EPI, ACT_GEGLU>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((dense_finish<T, EPI, ACT_NONE>), grid, block, 0, s, p);
    }
}

}  // namespace

hipError_t launch_dense_sums(const DenseSums &p, const DenseTails &t, int dtype, hipStream_t s) {
    if (p.count + t.count == 0) return hipSuccess;
    int widest = 0;
    for (int i = 0; i < p.count; ++i) widest = p.t[i].C > widest ? p.t[i].C : widest;
    const int per = dtype == 1 ? 256 : 128;
    const dim3 grid(p.count ? (widest + per - 1) / per : 32, p.count ? dense_sum_ranges(p.M) : 1,
                    p.count + t.count);
    if (dtype == 1) hipLaunchKernelGGL((dense_sums<uint16_t>), grid, dim3(256), 0, s, p, t);
    else hipLaunchKernelGGL((dense_sums<float>), grid, dim3(256), 0, s, p, t);
    return hipGetLastError();
}

hipError_t launch_dense_sums_join(const DenseSums &p, int dtype, hipStream_t s) {
    if (p.count == 0 || dense_sum_ranges(p.M) == 1) return hipSuccess;
    int widest = 0;
    for (int i = 0; i < p.count; ++i) widest = p.t[i].C > widest ? p.t[i].C : widest;
    const dim3 join(widest / 64, p.count);
    if (dtype == 1) hipLaunchKernelGGL((dense_sums_join<uint16_t>), join, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((dense_sums_join<float>), join, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_dense_finish(const DenseRows &p, int dtype, hipStream_t s) {
    if (dtype == 1) {
        if (p.epilogue == DENSE_FORWARD) finish_as<uint16_t, DENSE_FORWARD>(p, s);
        else finish_as<uint16_t, DENSE_GRAD>(p, s);
    } else {
        if (p.epilogue == DENSE_FORWARD) finish_as<float, DENSE_FORWARD>(p, s);
        else finish_as<float, DENSE_GRAD>(p, s);
    }
    return hipGetLastError();
}

// A split product leaves its planes, and the epilogue is a kernel of its own.
hipError_t launch_dense_rows(const DenseRows &p, int dtype, hipStream_t s) {
    if (p.plan.stream) return launch_dense_stream(p, dtype, s);
    DenseRows q = p;
    if (p.plan.splits > 1) q.epilogue = DENSE_PLANE;
    hipError_t e;
    if (dtype != 1) e = launch_dense_rows_f32(q, s);
    else if (q.epilogue == DENSE_PLANE) e = launch_dense_plane_mfma(q, s);
    else if (q.epilogue == DENSE_FORWARD) e = launch_dense_forward_mfma(q, s);
    else e = launch_dense_grad_mfma(q, s);
    if (e != hipSuccess || q.epilogue == p.epilogue) return e;
    return launch_dense_finish(p, dtype, s);
}

hipError_t launch_dense_weights(const DenseWeights &p, int dtype, hipStream_t s) {
    if (p.count == 0) return hipSuccess;
    const hipError_t e =
        dtype == 1 ? launch_dense_weights_mfma(p, s) : launch_dense_weights_f32(p, s);
    if (e != hipSuccess || p.splits == 1) return e;
    size_t most = 0;
    for (int k = 0; k < p.count; ++k) {
        const size_t n = (size_t)p.m[k].R * p.m[k].C;
        if (n > most) most = n;
    }
    const int per = 256 * (dtype == 1 ? 8 : 4);
    const dim3 grid((unsigned)((most + per - 1) / per), p.count);
    if (dtype == 1) hipLaunchKernelGGL((dense_weight_finish<uint16_t>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((dense_weight_finish<float>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}
