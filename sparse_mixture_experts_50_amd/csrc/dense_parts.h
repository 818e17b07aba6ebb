// Column sums and the joining of planes: the parts of the dense layer's small
// kernels that share a launch with others.
#pragma once

#include "act.h"
#include "dense.h"

namespace dense_parts {

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

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t *p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }

// Bytes of LDS of sum_columns().
constexpr int SUMS_LDS = 8 * 32 * 8 * 4;

// Columns [256 c, 256 c + 256) (fp32: 128) of range r of an item, eight rows
// side by side; one range: the result itself.
template <typename T>
__device__ __forceinline__ void sum_columns(const DenseSums::Item &t, int M, int c, int r,
                                            float *lds) {
    constexpr int N = Vec<T>::N;
    const int col = threadIdx.x & 31, lane = threadIdx.x >> 5;
    const int c0 = c * 32 * N, at = c0 + col * N;
    if (c0 >= t.C) return;
    const int m0 = r * MOE_DENSE_SUM_ROWS, m1 = min(M, m0 + MOE_DENSE_SUM_ROWS);
    Vec<T> sum, x;
    sum.clear();
    if (at < t.C)
#pragma unroll 4
        for (int m = m0 + lane; m < m1; m += 8) {
            x.load((const T *)t.src + (size_t)m * t.C + at);
#pragma unroll
            for (int i = 0; i < N; ++i) sum.v[i] += x.v[i];
        }
#pragma unroll
    for (int i = 0; i < N; ++i) lds[lane * 32 * N + col * N + i] = sum.v[i];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * N; i += 256) {
        float s = 0.0f;
#pragma unroll
        for (int l = 0; l < 8; ++l) s += lds[l * 32 * N + i];
        if (c0 + i >= t.C) continue;
        if (M <= MOE_DENSE_SUM_ROWS) put((T *)t.out + c0 + i, s);
        else t.part[(size_t)r * t.C + c0 + i] = s;
    }
}

}  // namespace dense_parts
