// The f32 layer's tile product: acc += A B with fp32 MFMAs (16x16x4, fp32
// operands and accumulation) on a 64 x 64 tile of four waves, 32 x 32 each,
// for either order of each operand.  Two stages of 32 k, one barrier each.
// Sums run over 64 k at a time and are then added to the total: one chain of
// fp32 additions over 4000 tokens errs by 1e-6 of a weight gradient, these by
// 3e-7.
#pragma once

#include "common.h"

namespace f32t {

constexpr int BM = 64, BN = 64, BK = 32;
constexpr int CHAIN = 64;                // k added up before joining the total
struct Stage {
    float a[2][BK][BM + 4];
    float b[2][BK][BN + 4];
};
// Wave w: rows 32 (w / 2), columns 32 (w % 2); block (i, j) of 16 x 16; the
// lane's element e: row l % 16, column 4 (l / 16) + e.
typedef floatx4 Acc[2][2];

__device__ __forceinline__ floatx4 load4(const float *p) { return *(const floatx4 *)p; }

// One operand's stage: 64 rows (or columns) by 32 k, eight values a thread.
// KC: element (r, k) at p[r * ld + k], rows r >= valid read as 0;
// else at p[k * ld + r], k >= valid read as 0.  (Bounds of the other axis
// are the caller's: multiples of 64 and 32.)
template <bool KC> struct Part {
    floatx4 v[2];
    __device__ __forceinline__ void fetch(const float *p, size_t ld, int k0, int valid) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = KC ? tid >> 2 : (tid & 15) * 4;
            const int k = k0 + 16 * h + (KC ? (tid & 3) * 4 : tid >> 4);
            v[h] = (KC ? row : k) < valid ? load4(KC ? p + row * ld + k : p + k * ld + row)
                                          : floatx4{0.f, 0.f, 0.f, 0.f};
        }
    }
    __device__ __forceinline__ void put(float (*s)[BM + 4]) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (KC) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[16 * h + (tid & 3) * 4 + i][tid >> 2] = v[h][i];
            } else {
                *(floatx4 *)&s[16 * h + (tid >> 4)][(tid & 15) * 4] = v[h];
            }
        }
    }
};

__device__ __forceinline__ void clear(Acc &acc) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
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
    Part<AK> pa;
    Part<BKC> pb;
    pa.fetch(A, lda, 0, a_valid);
    pb.fetch(B, ldb, 0, b_valid);
    pa.put(st.a[0]);
    pb.put(st.b[0]);
    Acc part;
    clear(part);
    int cur = 0;
    for (int k0 = 0; k0 < K; k0 += BK) {
        const bool more = k0 + BK < K;
        if (more) {
            pa.fetch(A, lda, k0 + BK, a_valid);
            pb.fetch(B, ldb, k0 + BK, b_valid);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < BK; k += 4) {
            float a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = st.a[cur][k + kq][r + 16 * i];
                b[i] = st.b[cur][k + kq][c + 16 * i];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    part[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[j], a[i], part[i][j],
                                                                      0, 0, 0);
        }
        if (more) {
            // (last read before the barrier above)
            pa.put(st.a[cur ^ 1]);
            pb.put(st.b[cur ^ 1]);
            cur ^= 1;
        }
        if (!more || (k0 + BK) % CHAIN == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] += part[i][j];
            clear(part);
        }
    }
    __syncthreads();
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

}  // namespace f32t
