// The f32 layer's tile product: acc += A B with fp32 MFMAs (16x16x4, fp32
// operands and accumulation) on a 64 x 64 tile of four waves, 32 x 32 each,
// for either order of each operand.
#pragma once

#include "common.h"

namespace f32t {

constexpr int BM = 64, BN = 64, BK = 16;
struct Stage {
    float a[BK][BM + 4];
    float b[BK][BN + 4];
};
// Wave w: rows 32 (w / 2), columns 32 (w % 2); block (i, j) of 16 x 16; the
// lane's element e: row l % 16, column 4 (l / 16) + e.
typedef floatx4 Acc[2][2];

__device__ __forceinline__ floatx4 load4(const float *p) { return *(const floatx4 *)p; }

// One operand's stage: 64 rows (or columns) by 16 k, four values a thread.
// KC: element (r, k) at p[r * ld + k], rows r >= valid read as 0;
// else at p[k * ld + r], k >= valid read as 0.  (Bounds of the other axis
// are the caller's: multiples of 64 and 16.)
template <bool KC>
__device__ __forceinline__ floatx4 fetch(const float *p, size_t ld, int k0, int valid) {
    const int tid = threadIdx.x;
    const int row = KC ? tid >> 2 : (tid & 15) * 4;
    const int k = k0 + (KC ? (tid & 3) * 4 : tid >> 4);
    if ((KC ? row : k) >= valid) return floatx4{0.f, 0.f, 0.f, 0.f};
    return load4(KC ? p + row * ld + k : p + k * ld + row);
}
template <bool KC>
__device__ __forceinline__ void put(float (*s)[BM + 4], floatx4 v) {
    const int tid = threadIdx.x;
    if (KC) {
        const int row = tid >> 2, k = (tid & 3) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[k + i][row] = v[i];
    } else {
        *(floatx4 *)&s[tid >> 4][(tid & 15) * 4] = v;
    }
}

// acc += sum over k < K; a_valid / b_valid: see fetch.  Begins and ends with
// the stage free.
template <bool AK, bool BKC>
__device__ __forceinline__ void product(Acc &acc, Stage &st, const float *A, size_t lda,
                                        int a_valid, const float *B, size_t ldb,
                                        int b_valid, int K) {
    if (K <= 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = (wave >> 1) * 32 + (lane & 15), c = (wave & 1) * 32 + (lane & 15);
    const int kq = lane >> 4;
    floatx4 av = fetch<AK>(A, lda, 0, a_valid);
    floatx4 bv = fetch<BKC>(B, ldb, 0, b_valid);
    for (int k0 = 0; k0 < K; k0 += BK) {
        put<AK>(st.a, av);
        put<BKC>(st.b, bv);
        __syncthreads();
        if (k0 + BK < K) {
            av = fetch<AK>(A, lda, k0 + BK, a_valid);
            bv = fetch<BKC>(B, ldb, k0 + BK, b_valid);
        }
#pragma unroll
        for (int k = 0; k < BK; k += 4) {
            float a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = st.a[k + kq][r + 16 * i];
                b[i] = st.b[k + kq][c + 16 * i];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[j], a[i], acc[i][j],
                                                                     0, 0, 0);
        }
        __syncthreads();
    }
}

// Calls f(row, column, values) for each of the lane's four runs of 4
// consecutive columns.
template <typename F> __device__ __forceinline__ void each(const Acc &acc, F f) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            f((wave >> 1) * 32 + 16 * i + (lane & 15),
              (wave & 1) * 32 + 16 * j + 4 * (lane >> 4), acc[i][j]);
}

__device__ __forceinline__ void clear(Acc &acc) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
}

}  // namespace f32t
