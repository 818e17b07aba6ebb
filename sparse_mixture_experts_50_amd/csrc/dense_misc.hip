// Small kernels around the dense layer's products, and what is launched of
// them: bias gradients (and in the same launch the last rows copied beside
// zeros), the epilogue of products whose sums lie in planes, planes and ranges
// joined.  All bound by memory.
#include "dense_parts.h"

namespace {

using namespace dense_parts;

__global__ __launch_bounds__(256) void dense_sums(DenseSums p, DenseTails tails) {
    __shared__ float lds[SUMS_LDS / 4];
    sums_and_tails<uint16_t>(p, tails, blockIdx.x, lds);
}

template <typename T>
__global__ __launch_bounds__(256) void dense_joins(DenseRows p, DenseWeights w, DenseSums b,
                                                   int rows, int weights) {
    __shared__ float lds[256];
    join<T>(p, w, b, blockIdx.x, rows, weights, lds);
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

template <typename T, int EPI> void finish_as(const DenseRows &p, hipStream_t s) {
    const long long vectors = (long long)p.M * p.N / Vec<T>::N;
    const dim3 grid((unsigned)((vectors + 255) / 256)), block(256);
    switch (p.act) {
    case ACT_GELU:
        hipLaunchKernelGGL((dense_finish<T, EPI, ACT_GELU>), grid, block, 0, s, p);
        break;
    case ACT_SILU:
        hipLaunchKernelGGL((dense_finish<T, EPI, ACT_SILU>), grid, block, 0, s, p);
        break;
    case ACT_SWIGLU:
        hipLaunchKernelGGL((dense_finish<T, EPI, ACT_SWIGLU>), grid, block, 0, s, p);
        break;
    case ACT_GEGLU:
        hipLaunchKernelGGL((dense_finish<T, EPI, ACT_GEGLU>), grid, block, 0, s, p);
        break;
    default:
        // (a layer without an activation has no pre-activation's gradient)
        if constexpr (EPI == DENSE_FORWARD)
            hipLaunchKernelGGL((dense_finish<T, EPI, ACT_NONE>), grid, block, 0, s, p);
    }
}

}  // namespace

hipError_t launch_dense_sums(const DenseSums &p, const DenseTails &t, hipStream_t s) {
    const int blocks = sums_blocks(p, t, 256);
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(dense_sums, dim3(blocks), dim3(256), 0, s, p, t);
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
hipError_t launch_dense_product(const DenseRows &p, int dtype, hipStream_t s) {
    if (p.plan.stream) return launch_dense_stream(p, dtype, s);
    DenseRows q = p;
    if (p.plan.splits > 1) q.epilogue = DENSE_PLANE;
    if (dtype != 1) return launch_dense_rows_f32(q, s);
    if (q.epilogue == DENSE_PLANE) return launch_dense_plane_mfma(q, s);
    return q.epilogue == DENSE_FORWARD ? launch_dense_forward_mfma(q, s)
                                       : launch_dense_grad_mfma(q, s);
}

hipError_t launch_dense_rows(const DenseRows &p, int dtype, hipStream_t s) {
    const hipError_t e = launch_dense_product(p, dtype, s);
    if (e != hipSuccess || p.plan.stream || p.plan.splits == 1 || p.epilogue == DENSE_PLANE)
        return e;
    return launch_dense_finish(p, dtype, s);
}

// A launch that waits for another costs 4 to 6 us, so small parts that do not
// depend on each other share one: the sums and the last rows with the rows'
// gradient, what that leaves to join with the weights', in fp32 both products
// (fp32, 256 tokens, 64 x 256, all gradients 36 us apart, 26 so; bf16, 33 rows,
// 1024 to 2816: 27 and 20; 1030 tokens, 1024 x 704: 54 and 46).
hipError_t launch_dense_back(const DenseBack &p, int dtype, hipStream_t s) {
    // what is left to join
    const int per = 256 * (dtype == 1 ? 8 : 4);
    int rows = 0, weights = 0, sums = 0;
    if (p.rows && p.dx.plan.splits > 1)
        rows = (int)(((size_t)p.dx.M * p.dx.N + per - 1) / per);
    if (p.w.count && p.w.splits > 1) {
        size_t most = 0;
        for (int k = 0; k < p.w.count; ++k) {
            const size_t n = (size_t)p.w.m[k].R * p.w.m[k].C;
            if (n > most) most = n;
        }
        weights = (int)((most + per - 1) / per) * p.w.count;
    }
    if (dense_sum_ranges(p.b.M) > 1)
        for (int k = 0; k < p.b.count; ++k) sums += p.b.t[k].C / 64;
    hipError_t e;
    if (dtype != 1) {
        e = launch_dense_back_f32(p, s);
    } else {
        if (p.rows && p.dx.plan.small) {
            e = launch_dense_dx_sums(p.dx, p.b, p.t, s);
        } else {
            e = launch_dense_sums(p.b, p.t, s);
            if (e == hipSuccess && p.rows) e = launch_dense_product(p.dx, dtype, s);
        }
        if (e == hipSuccess && p.w.count && p.w.small) {
            e = launch_dense_weights_joins(p.w, p.dx, p.b, rows, sums, s);
            rows = sums = 0;
        } else if (e == hipSuccess && p.w.count) {
            e = launch_dense_weights_mfma(p.w, s);
        }
    }
    if (e != hipSuccess || rows + weights + sums == 0) return e;
    const dim3 grid(rows + weights + sums);
    if (dtype == 1)
        hipLaunchKernelGGL((dense_joins<uint16_t>), grid, dim3(256), 0, s, p.dx, p.w, p.b, rows,
                           weights);
    else
        hipLaunchKernelGGL((dense_joins<float>), grid, dim3(256), 0, s, p.dx, p.w, p.b, rows,
                           weights);
    return hipGetLastError();
}
