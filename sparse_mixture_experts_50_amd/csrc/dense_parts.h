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

// What products and sums of ranges left behind, added up: the rows' gradient
// (blocks up to `rows`), the weights' (up to `weights` more, as many for each
// matrix), the column sums (64 columns by four ranges at a time; 256 floats of
// LDS).
template <typename T>
__device__ __forceinline__ void join(const DenseRows &p, const DenseWeights &w,
                                     const DenseSums &b, int block, int rows, int weights,
                                     float *lds) {
    constexpr int N = Vec<T>::N;
    if (block < rows) {
        const size_t plane = (size_t)p.M * p.N, at = ((size_t)block * 256 + threadIdx.x) * N;
        if (at >= plane) return;
        Vec<T> s, a;
        s.clear();
#pragma unroll 4
        for (int i = 0; i < p.plan.splits; ++i) s.add(p.plane + i * plane + at);
        if (p.res) {
            a.load((const T *)p.res + at);
#pragma unroll
            for (int i = 0; i < N; ++i) s.v[i] += a.v[i];
        }
        s.store((T *)p.y + at);
        return;
    }
    block -= rows;
    if (block < weights) {
        const int each = weights / w.count, k = block / each;
        const DenseMat &m = w.m[k];
        const size_t size = (size_t)m.R * m.C;
        const size_t at = ((size_t)(block - k * each) * 256 + threadIdx.x) * N;
        if (at >= size) return;
        Vec<T> s;
        s.clear();
#pragma unroll 4
        for (int i = 0; i < w.splits; ++i) s.add(w.plane + w.offset[k] + i * size + at);
        s.store((T *)m.out + at);
        return;
    }
    block -= weights;
    int k = 0;
    for (; k + 1 < b.count && block >= b.t[k].C / 64; ++k) block -= b.t[k].C / 64;
    const DenseSums::Item &t = b.t[k];
    const int in = threadIdx.x & 63, c = block * 64 + in, lane = threadIdx.x >> 6;
    float s = 0.0f;
    for (int r = lane; r < dense_sum_ranges(b.M); r += 4) s += t.part[(size_t)r * t.C + c];
    lds[threadIdx.x] = s;
    __syncthreads();
    if (lane) return;
    put((T *)t.out + c, (lds[in] + lds[64 + in]) + (lds[128 + in] + lds[192 + in]));
}

// Rows copied, and rows zeroed after them, by block `block` of TAIL_BLOCKS.
constexpr int TAIL_BLOCKS = 8;
__device__ __forceinline__ void copy_tail(const DenseTails::Item &t, int block) {
    const size_t bytes = (size_t)t.row_bytes * t.rows, copied = (size_t)t.row_bytes * t.copied;
    for (size_t b = ((size_t)block * 256 + threadIdx.x) * 16; b < bytes;
         b += TAIL_BLOCKS * 256 * 16)
        *(u32x4 *)((char *)t.dst + b) =
            b < copied ? *(const u32x4 *)((const char *)t.src + b) : u32x4{0, 0, 0, 0};
}

// Blocks of all items' sums, and of the tails.  per: columns of a block.
inline int sums_blocks(const DenseSums &p, const DenseTails &t, int per) {
    int n = t.count * TAIL_BLOCKS;
    for (int k = 0; k < p.count; ++k) n += (p.t[k].C + per - 1) / per * dense_sum_ranges(p.M);
    return n;
}
// Block `block` of them: the tails come first.
template <typename T>
__device__ __forceinline__ void sums_and_tails(const DenseSums &p, const DenseTails &t, int block,
                                               float *lds) {
    if (block < t.count * TAIL_BLOCKS) {
        copy_tail(t.t[block / TAIL_BLOCKS], block % TAIL_BLOCKS);
        return;
    }
    block -= t.count * TAIL_BLOCKS;
    constexpr int per = 32 * Vec<T>::N;
    const int ranges = dense_sum_ranges(p.M);
    int k = 0;
    for (; k + 1 < p.count; ++k) {
        const int n = (p.t[k].C + per - 1) / per * ranges;
        if (block < n) break;
        block -= n;
    }
    const int columns = (p.t[k].C + per - 1) / per;
    sum_columns<T>(p.t[k], p.M, block % columns, block / columns, lds);
}

}  // namespace dense_parts
