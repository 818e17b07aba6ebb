// Global norm of many gradient tensors and their clipping:
//   norm = sqrt(sum of squares over every element of every tensor)
//   dst = src * min(1, max_norm / (norm + 1e-6))
//
// Bound by HBM: one read for the norm, one read and one write for the
// clipping.  Both passes walk 32 KB chunks of all tensors, dealt round-robin
// to the blocks, so tensors of any mix of sizes keep every CU busy; the
// second pass walks them (and the tables of 96 tensors, one a launch)
// backwards and finds the first pass's last 256 MB in the last-level cache.
// Squares are summed in double: HBM leaves the double rate idle, large values
// cannot overflow and the sum of 1e9 squares keeps its digits.  Every block of
// the second pass adds the partial sums by itself instead of waiting for a
// launch that does only that: at most 2048 of them up to 32 tables (16 KB out
// of L2), 64 for each table of a longer list.  The order of every sum is
// fixed.
//
// Measured: 24 tensors of both types, 8.5 GB read and written, 2.35 ms, 5.4
// TB/s of the 12.7 GB that two passes move; 40 tensors of 0.7 MB together 45
// us, most of it the host's work on the list.
#include "grad.h"

namespace {

constexpr int THREADS = 256;
constexpr int CHUNK = 32768;          // bytes of source

struct Chunk {
    const char *src;                  // first element of the tensor
    char *dst;
    long long n;                      // elements of the tensor
    long long v0, v1;                 // 16-byte vectors of this chunk
    long long nv;                     // vectors of the tensor
    int head;                         // elements before the first vector
    bool first, last, f32;
};

__device__ __forceinline__ int chunk_vectors() { return CHUNK / 16; }

__device__ __forceinline__ Chunk chunk_of(const ClipTable &tab, int c) {
    int lo = 0, hi = tab.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.first[mid] <= c) lo = mid; else hi = mid;
    }
    Chunk k;
    const ClipTensor &t = tab.t[lo];
    k.src = (const char *)t.src;
    k.dst = (char *)t.dst;
    k.n = t.n;
    k.f32 = (tab.f32[lo >> 5] >> (lo & 31)) & 1;
    const int es = k.f32 ? 4 : 2;
    const int off = (int)((uintptr_t)k.src & 15);
    long long head = off ? (16 - off) / es : 0;
    if (head > k.n) head = k.n;
    k.head = (int)head;
    k.nv = (k.n - head) / (16 / es);
    const int i = c - tab.first[lo];
    k.first = i == 0;
    k.last = c + 1 == tab.first[lo + 1];
    k.v0 = (long long)i * chunk_vectors();
    k.v1 = k.last ? k.nv : k.v0 + chunk_vectors();
    if (k.v1 > k.nv) k.v1 = k.nv;
    return k;
}

__device__ __forceinline__ float elem(const char *p, long long i, bool f32) {
    return f32 ? ((const float *)p)[i] : bf16_to_f32(((const uint16_t *)p)[i]);
}
__device__ __forceinline__ void set_elem(char *p, long long i, bool f32, float v) {
    if (f32) ((float *)p)[i] = v;
    else ((uint16_t *)p)[i] = (uint16_t)f32_to_bf16_bits(v);
}

// Sum of v over the block, the same in every thread.
__device__ double block_sum(double v, double *lds) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < THREADS / 64; ++i) v += lds[i];
    return v;
}

__device__ __forceinline__ double sq(float v) { return (double)v * (double)v; }

__global__ __launch_bounds__(THREADS) void clip_norm(ClipTable tab,
                                                     double *part) {
    __shared__ double lds[THREADS / 64];
    double sum = 0.0;
    for (int c = blockIdx.x; c < tab.first[tab.count]; c += gridDim.x) {
        const Chunk k = chunk_of(tab, c);
        const u32x4 *v = (const u32x4 *)(k.src + (size_t)k.head * (k.f32 ? 4 : 2));
        double s0 = 0.0, s1 = 0.0;
#pragma unroll 4
        for (long long i = k.v0 + threadIdx.x; i < k.v1; i += THREADS) {
            const u32x4 q = v[i];
            if (k.f32) {
                s0 += sq(__uint_as_float(q[0])) + sq(__uint_as_float(q[1]));
                s1 += sq(__uint_as_float(q[2])) + sq(__uint_as_float(q[3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s0 += sq(bf16_lo(q[e]));
                    s1 += sq(bf16_hi(q[e]));
                }
            }
        }
        sum += s0 + s1;
        // elements before the first and after the last vector (< 8 each)
        if (k.first && threadIdx.x < k.head) sum += sq(elem(k.src, threadIdx.x, k.f32));
        if (k.last) {
            const long long i = k.head + k.nv * (k.f32 ? 4 : 8) + threadIdx.x;
            if (i < k.n) sum += sq(elem(k.src, i, k.f32));
        }
    }
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// parts: partial sums of every table; norm: written by block 0 if not null.
__global__ __launch_bounds__(THREADS) void clip_scale(ClipTable tab,
                                                      const double *part,
                                                      int parts, float max_norm,
                                                      float *norm) {
    __shared__ double lds[THREADS / 64];
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += THREADS) sum += part[i];
    const double len = sqrt(block_sum(sum, lds));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)len;
    // not fmin: a norm that is not a number has to reach the gradients
    const double c = (double)max_norm / (len + 1e-6);
    const float f = c >= 1.0 ? 1.0f : (float)c;
    const int chunks = tab.first[tab.count];
    for (int b = blockIdx.x; b < chunks; b += gridDim.x) {
        const Chunk k = chunk_of(tab, chunks - 1 - b);
        if (!k.dst) continue;
        const int es = k.f32 ? 4 : 2;
        const size_t h = (size_t)k.head * es;
        const u32x4 *v = (const u32x4 *)(k.src + h);
        if ((((uintptr_t)k.dst ^ (uintptr_t)k.src) & 15) == 0) {
            u32x4 *o = (u32x4 *)(k.dst + h);
#pragma unroll 4
            for (long long i = k.v0 + threadIdx.x; i < k.v1; i += THREADS) {
                u32x4 q = v[i];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    q[e] = k.f32 ? __float_as_uint(__uint_as_float(q[e]) * f)
                                 : pack_bf16x2(bf16_lo(q[e]) * f, bf16_hi(q[e]) * f);
                o[i] = q;
            }
        } else {
            // source and destination lie differently to 16 bytes
            const int vn = 16 / es;
            const long long e1 = k.head + k.v1 * vn;
            for (long long i = k.head + k.v0 * vn + threadIdx.x; i < e1; i += THREADS)
                set_elem(k.dst, i, k.f32, elem(k.src, i, k.f32) * f);
        }
        if (k.first && threadIdx.x < k.head)
            set_elem(k.dst, threadIdx.x, k.f32, elem(k.src, threadIdx.x, k.f32) * f);
        if (k.last) {
            const long long i = k.head + k.nv * (16 / es) + threadIdx.x;
            if (i < k.n) set_elem(k.dst, i, k.f32, elem(k.src, i, k.f32) * f);
        }
    }
}

}  // namespace

// Chunks of a tensor of n elements (the caller fills ClipTable::first): by
// bytes, and a part of a vector more at either end.
long long clip_chunks(long long n, int f32) {
    return (n * (f32 ? 4 : 2) + CHUNK - 1) / CHUNK;
}

hipError_t launch_clip_norm(const ClipTable &tab, double *part, int grid,
                            hipStream_t s) {
    hipLaunchKernelGGL(clip_norm, dim3(grid), dim3(THREADS), 0, s, tab, part);
    return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipTable &tab, const double *part,
                             int parts, float max_norm, float *norm, int grid,
                             hipStream_t s) {
    hipLaunchKernelGGL(clip_scale, dim3(grid), dim3(THREADS), 0, s, tab, part,
                       parts, max_norm, norm);
    return hipGetLastError();
}
