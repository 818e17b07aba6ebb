// A 64 x 64 tile product on the vector units with fp32 accumulation, for
// either order of each operand: the f32 layer's gradient GEMMs and the
// router's small ones.
#pragma once

#include "common.h"

namespace simt {

constexpr int BM = 64, BN = 64, BK = 16;
struct Stage {
    float a[BK][BM + 4];
    float b[BK][BN + 4];
};

__device__ __forceinline__ float4 load4(const float *p) {
    return *(const float4 *)p;
}
__device__ __forceinline__ float4 load4(const uint16_t *p) {
    const u32x2 q = *(const u32x2 *)p;
    return make_float4(bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y));
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
    *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4]) {
    u32x2 q;
    q.x = pack_bf16x2(v[0], v[1]);
    q.y = pack_bf16x2(v[2], v[3]);
    *(u32x2 *)p = q;
}

// One operand's stage: 64 rows (or columns) by 16 k, four values a thread.
// KC: element (r, k) at p[r * ld + k], rows r >= valid read as 0;
// else at p[k * ld + r], k >= valid read as 0.  (Bounds of the other axis
// are the caller's: multiples of 64 and 16.)
template <bool KC, typename T>
__device__ __forceinline__ float4 fetch(const T *p, size_t ld, int k0,
                                        int valid) {
    const int tid = threadIdx.x;
    const int row = KC ? tid >> 2 : (tid & 15) * 4;
    const int k = k0 + (KC ? (tid & 3) * 4 : tid >> 4);
    if ((KC ? row : k) >= valid) return make_float4(0.f, 0.f, 0.f, 0.f);
    return load4(KC ? p + row * ld + k : p + k * ld + row);
}
template <bool KC>
__device__ __forceinline__ void put(float (*s)[BM + 4], float4 v) {
    const int tid = threadIdx.x;
    if (KC) {
        const int row = tid >> 2, k = (tid & 3) * 4;
        s[k + 0][row] = v.x;
        s[k + 1][row] = v.y;
        s[k + 2][row] = v.z;
        s[k + 3][row] = v.w;
    } else {
        *(float4 *)&s[tid >> 4][(tid & 15) * 4] = v;
    }
}

// acc[i][j] += sum over k < K of A(4 ty + i, k) B(4 tx + j, k), the block's
// 256 threads being 16 x 16.  a_valid / b_valid: see fetch.  Begins and
// ends with the stage free.
template <bool AK, bool BKC, typename TA, typename TB>
__device__ __forceinline__ void product(float (&acc)[4][4], Stage &st,
                                        const TA *A, size_t lda, int a_valid,
                                        const TB *B, size_t ldb, int b_valid,
                                        int K) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    if (K <= 0) return;
    float4 av = fetch<AK>(A, lda, 0, a_valid);
    float4 bv = fetch<BKC>(B, ldb, 0, b_valid);
    for (int k0 = 0; k0 < K; k0 += BK) {
        put<AK>(st.a, av);
        put<BKC>(st.b, bv);
        __syncthreads();
        if (k0 + BK < K) {
            av = fetch<AK>(A, lda, k0 + BK, a_valid);
            bv = fetch<BKC>(B, ldb, k0 + BK, b_valid);
        }
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const float4 a4 = *(const float4 *)&st.a[k][ty * 4];
            const float4 b4 = *(const float4 *)&st.b[k][tx * 4];
            const float a[4] = {a4.x, a4.y, a4.z, a4.w};
            const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
}

__device__ __forceinline__ void clear(float (&acc)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
}

}  // namespace simt
