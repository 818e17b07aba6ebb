// Linear layers of few rows (M <= 64) and enough columns to give most CUs a
// block, both types: the weights are streamed once from memory.
//
// A block takes 16 columns (of each panel) at a time and all rows; its four
// waves split K.  Both operands pass through LDS: a stage is 16 rows by 1 KB
// of each, fetched in whole runs of 1 KB into a ring of four slots (three
// stages, 48 KB a block, in flight) that runs on across units; x's rows come
// first in each range of K and stay in registers while the weights' follow.
// The waves' sums are added in order before the epilogue.  (fp32: the four k
// of a lane go to four MFMAs; which k an MFMA adds up does not matter as long
// as both operands agree.)  Rows past M re-read the last.  A wave's quarter of
// K is one chain of fp32 sums: f32, 4096 deep, off by 5.7e-7 of the norm, 16384
// deep by 1.1e-6, where tiles that join a total every 64 terms are off by 1.7e-7
// and 1.8e-7.
//
// Bound by HBM, from 32 rows on by what x adds to the loads (MB stages for
// every P of weights, from L2).  Fragments straight from memory, 16 rows by 64
// bytes an instruction, end at 12 bytes a clock and CU, however many are in
// flight: 32 rows, 4096 to 14336 features, gated (235 MB of weights) 78 us,
// through the ring 43 (5.5 TB/s; the median of 40 calls 45); 14336 to 4096
// (117 MB) 46 and 32; one row, 41 and 25.  Two or four groups of 16 columns a
// unit: 46 and 42 us of the first, 39 and 52 of the second; six to nine slots,
// one block a CU: 46 to 48, and 32 to 34.
#include <type_traits>
#include <utility>

#include "act.h"
#include "dense.h"

namespace {

template <typename T>
__device__ __forceinline__ void mac(floatx4 &acc, u32x4 w, u32x4 x) {
    if constexpr (sizeof(T) == 2) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), as_bf16x8(x), acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[e]),
                                                       __uint_as_float(x[e]), acc, 0, 0, 0);
    }
}

__device__ __forceinline__ floatx4 load4(const float *p) { return *(const floatx4 *)p; }
__device__ __forceinline__ floatx4 load4(const uint16_t *p) {
    const u32x2 v = *(const u32x2 *)p;
    return floatx4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}
__device__ __forceinline__ void store4(float *p, floatx4 v) { *(floatx4 *)p = v; }
__device__ __forceinline__ void store4(uint16_t *p, floatx4 v) {
    *(u32x2 *)p = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// The epilogue of 4 columns of a row, at element `at`.
template <typename T, int EPI, int ACT>
__device__ __forceinline__ void finish(const DenseRows &p, floatx4 z, floatx4 u, size_t at) {
    constexpr bool FAST = sizeof(T) == 2;
    if (EPI == DENSE_FORWARD) {
        floatx4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = act_value<ACT, FAST>(z[e], u[e]);
        if (p.res) y += load4((const T *)p.res + at);
        store4((T *)p.y + at, y);
        return;
    }
    floatx4 q;
    if (p.dy) {
        q = load4((const T *)p.dy + at);
    } else {
        q = load4(p.q + at);
        for (int s = 1; s < p.q_planes; ++s) q += load4(p.q + (size_t)s * p.M * p.N + at);
    }
    floatx4 h, dz, du;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float v, hz, hu;
        act_grad<ACT, FAST>(z[e], u[e], v, hz, hu);
        h[e] = v;
        dz[e] = q[e] * hz;
        du[e] = q[e] * hu;
    }
    store4((T *)p.dz + at, dz);
    if (act_gated(ACT)) store4((T *)p.du + at, du);
    if (p.h) store4((T *)p.h + at, h);
}

constexpr int CB = 1024;          // bytes of a row in a stage
constexpr int SLOTS = 4;          // of 16 rows each

// Slot I of a ring, 16 rows: an array of its own each, so that the compiler
// sees that the loads into one and the reads of another do not alias.
template <int I> __device__ __forceinline__ u32x4 *ring_slot() {
    __shared__ u32x4 slot[CB];
    return slot;
}

// 64 lanes' 16 bytes to LDS; weights are read once (non-temporal).
template <bool ONCE> __device__ __forceinline__ void dma16(const char *src, u32x4 *lds) {
    __builtin_amdgcn_global_load_lds((const void *)src,
                                     (__attribute__((address_space(3))) void *)lds, 16, 0,
                                     ONCE ? 2 : 0);
}

// The block's waves meet, their LDS operations done (and loads in flight left
// alone, which __syncthreads() waits for).
__device__ __forceinline__ void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// f(integral_constant<int, I>) for each I.
template <int... I, typename F>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f) {
    (f(std::integral_constant<int, I>{}), ...);
}

// k ranges that are whole rounds of the slots
constexpr int ring_ranges(int stages) {
    int r = 1;
    while (stages * r % SLOTS) ++r;
    return r;
}

template <typename T, int EPI, int P, int MB>
__global__ __launch_bounds__(256, 2) void dense_stream(DenseRows p) {
    constexpr int STAGES = MB + P;              // of a k range: x, then weights
    constexpr int R = ring_ranges(STAGES);      // ranges of a trip
    __shared__ floatx4 red[4][P][64];
    const int M = p.M, N = p.N, K = p.K;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, hq = lane >> 4;
    const uint32_t row_bytes = (uint32_t)K * sizeof(T);
    const int ranges = (int)((row_bytes + CB - 1) / CB);
    const int trips = (ranges + R - 1) / R;
    const int units = N / 16;
    // The next stage to load: of k range lr of unit lu.  Every wave loads
    // rows wave, wave + 4, ... of it, a run of CB bytes each, whose 16-byte
    // chunks are XOR-swizzled by the row within 128 bytes.  (Past the end of
    // a row, its first chunk; past the last unit, that one again.)
    int lu = blockIdx.x, lr = 0;
    auto load = [&](auto at) __attribute__((always_inline)) {
        constexpr int J = decltype(at)::value % STAGES;
        u32x4 *to = ring_slot<decltype(at)::value % SLOTS>() + wave * (CB / 16);
        const char *base;
        if constexpr (J < MB)
            base = (const char *)p.a;
        else
            base = (const char *)(J > MB ? p.b2 : p.b) + (size_t)(lu * 16) * row_bytes;
        const uint32_t from = (uint32_t)lr * CB;
        const uint32_t left = row_bytes > from ? row_bytes - from : 0;
        base += left ? from : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = wave + 4 * i;
            uint32_t c = (uint32_t)(lane ^ (row & 7)) * 16;
            c *= c < left;
            const int m = J < MB ? min(J * 16 + row, M - 1) : row;
            dma16<(J >= MB)>(base + (size_t)m * row_bytes + c, to + 4 * i * (CB / 16));
        }
        if constexpr (J == STAGES - 1) {
            if (++lr == trips * R) {
                lr = 0;
                lu = min(lu + (int)gridDim.x, units - 1);
            }
        }
    };
    auto fragment = [&](const u32x4 *from, int s) __attribute__((always_inline)) {
        return from[l16 * (CB / 16) + ((4 * s + hq) ^ (l16 & 7))];
    };
    each_of(std::make_integer_sequence<int, SLOTS - 1>{}, load);
    floatx4 acc[MB][P];
    u32x4 x[MB][4];
    int steps = 0;
    // Stage `at` of a trip: landed in every wave (younger ones of four loads
    // each may be in flight), the slot of the one before is free.
    auto stage = [&](auto at) __attribute__((always_inline)) {
        constexpr int J = decltype(at)::value % STAGES;
        constexpr int AHEAD = 4 * (SLOTS - 2);
        __builtin_amdgcn_s_waitcnt((AHEAD & 0xF) | ((AHEAD >> 4) << 14) | (0x7 << 4));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        load(std::integral_constant<int, decltype(at)::value + SLOTS - 1>{});
        __builtin_amdgcn_sched_barrier(0);
        const u32x4 *from = ring_slot<decltype(at)::value % SLOTS>();
        if constexpr (J < MB) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[J][i] = fragment(from, wave + 4 * i);
        } else {
            u32x4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = fragment(from, wave + 4 * i);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (wave + 4 * i < steps) {
#pragma unroll
                    for (int m = 0; m < MB; ++m) mac<T>(acc[m][J - MB], w[i], x[m][i]);
                }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int g = 0; g < P; ++g) acc[m][g] = floatx4{0.f, 0.f, 0.f, 0.f};
        for (int t = 0; t < trips; ++t) {
            auto next = [&](auto at) __attribute__((always_inline)) {
                if constexpr (decltype(at)::value % STAGES == 0) {
                    // the waves share the range's steps of 64 bytes
                    const int left = (int)row_bytes - (t * R + decltype(at)::value / STAGES) * CB;
                    steps = max(min(left, CB), 0) / 64;
                }
                stage(at);
            };
            each_of(std::make_integer_sequence<int, R * STAGES>{}, next);
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            meet();
#pragma unroll
            for (int g = 0; g < P; ++g) red[wave][g][lane] = acc[m][g];
            meet();
            if (wave != (m & 3)) continue;
            floatx4 z = red[0][0][lane], v = red[0][P - 1][lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) {
                z += red[w][0][lane];
                if (P > 1) v += red[w][P - 1][lane];
            }
            const int row = 16 * m + l16, col = u * 16 + 4 * hq;
            if (row >= M) continue;
            if (p.bias) z += load4((const T *)p.bias + col);
            if (P > 1 && p.bias2) v += load4((const T *)p.bias2 + col);
            const size_t at = (size_t)row * N + col;
            if (P > 1) {
                if (p.act == ACT_SWIGLU) finish<T, EPI, ACT_SWIGLU>(p, z, v, at);
                else finish<T, EPI, ACT_GEGLU>(p, z, v, at);
            } else {
                if (p.act == ACT_GELU) finish<T, EPI, ACT_GELU>(p, z, v, at);
                else if (EPI == DENSE_GRAD || p.act == ACT_SILU)
                    finish<T, EPI, ACT_SILU>(p, z, v, at);
                else finish<T, DENSE_FORWARD, ACT_NONE>(p, z, v, at);
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(0);
}

template <typename T, int EPI, int P, int MB> void launch(const DenseRows &p, hipStream_t s) {
    // as few blocks as give each the same number of units
    const int units = p.N / 16, most = 512;
    const int per = (units + most - 1) / most, grid = (units + per - 1) / per;
    hipLaunchKernelGGL((dense_stream<T, EPI, P, MB>), dim3(grid), dim3(256), 0, s, p);
}
template <typename T, int EPI, int P> void by_rows(const DenseRows &p, hipStream_t s) {
    if (p.M <= 16) launch<T, EPI, P, 1>(p, s);
    else if (p.M <= 32) launch<T, EPI, P, 2>(p, s);
    else if (p.M <= 48) launch<T, EPI, P, 3>(p, s);
    else launch<T, EPI, P, 4>(p, s);
}
template <typename T> void by_form(const DenseRows &p, hipStream_t s) {
    if (p.epilogue == DENSE_FORWARD) {
        if (p.panels() == 2) by_rows<T, DENSE_FORWARD, 2>(p, s);
        else by_rows<T, DENSE_FORWARD, 1>(p, s);
    } else {
        if (p.panels() == 2) by_rows<T, DENSE_GRAD, 2>(p, s);
        else by_rows<T, DENSE_GRAD, 1>(p, s);
    }
}

}  // namespace

hipError_t launch_dense_stream(const DenseRows &p, int dtype, hipStream_t s) {
    if (dtype == 1) by_form<uint16_t>(p, s);
    else by_form<float>(p, s);
    return hipGetLastError();
}
