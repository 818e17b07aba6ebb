// One AdamW step over many tensors.  With g the gradient (times the clipping
// factor min(1, max_norm / (norm + 1e-6)) where a norm is given) and t the
// number of the step:
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   x = x - (lr decay x + lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps))
// The clipping factor enters here instead of in a pass of its own over the
// gradients, and is not rounded to their type.
//
// 8-bit states.  Blocks of 32 elements share a power of two, the least one
// under which the block's largest magnitude is at most 448, and hold e4m3
// codes: a power of two costs no rounding of its own.  v is held as its root,
// which has m's range: v itself would need twice the exponents.  Codes are
// rounded at random, with probabilities that make the mean of m and of the
// root right in each step: a step of e4m3 is 2^-3 of the value, and rounding
// to nearest would throw away every change of less than half of it, as (1 - b2)
// g^2 nearly always is.  A root that is not 0 never becomes 0 (m / eps would be
// what follows).  v, the root's square, gains the rounding's variance: of a
// root u that comes from a code c, with steps of s <= u / 8, at most |u - c| s
// <= (1 - b2) |g^2 - c^2| / 8, and half of that where u is near c.  So a long
// run ends with E c^2 - E g^2 <= (E g^2 + E c^2) / 8, or 2/7 over the 32-bit v
// at most; with normal gradients it is 2 % (b2 = 0.95) to 5 % (0.999), and
// updates are 1 to 2.5 % smaller.  (Codes under 2^-6, of roots under 2^-14 of
// their block's largest, have longer steps.)  The update
// itself uses m and v before they are rounded.  The random bits are a hash of
// seed, step, tensor and element, so the same call gives the same bits: its
// mixing steps are published ones of low bias (C. Wellons, "Prospecting for
// Hash Functions", 2018), the multipliers that make its key are primes of Y.
// Collet's published xxHash specification.
// bf16 parameters without a master copy can be rounded in the same way: lr
// is far below 2^-9 of a parameter, and nearest rounding keeps small updates
// out.
//
// m and v are computed without contraction, in the order written above, and
// the root is correctly rounded: the codes are then a function of the inputs
// that plain elementary operations reproduce bit for bit.
//
// Bound by HBM: every operand is read and written once, none comes back soon
// enough for a cache (non-temporal), and eight waves a SIMD hide what stands
// between a load and its store.  0.18 G bf16 elements with master copies (28
// bytes each) 0.99 ms, 5.1 TB/s; 0.58 G with 8-bit states (10.1 bytes) 1.25 ms,
// 4.7 TB/s (by the card 1.24 to 1.30), with four waves 1.47, by way of the caches 1.32, with the codes'
// rounding by integer steps instead of the conversion's 0.04 more.  Chunks of
// 16384 elements of all tensors (fewer where that leaves blocks without work)
// are dealt round-robin to the blocks, as the clipping's are.
#include "adamw.h"

namespace {

constexpr int THREADS = 256;

__device__ __forceinline__ uint32_t hash32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7FEB352Du;
    x ^= x >> 15;
    x *= 0x846CA68Bu;
    return x ^ (x >> 16);
}

// V elements from e0 on, as fp32 (zero from n on).  whole: all of them, at an
// address of a vector's alignment.
template <int V>
__device__ __forceinline__ void load(float (&x)[V], const void *p, bool f32, long long e0,
                                     long long n, bool whole) {
    if (whole) {
        if (f32) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const floatx4 q =
                    __builtin_nontemporal_load((const floatx4 *)((const float *)p + e0 + i));
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i + e] = q[e];
            }
        } else {
            const uint16_t *h = (const uint16_t *)p + e0;
            uint32_t w[V / 2];
            if (V == 8) *(u32x4 *)w = __builtin_nontemporal_load((const u32x4 *)h);
            else *(u32x2 *)w = __builtin_nontemporal_load((const u32x2 *)h);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                x[2 * i] = bf16_lo(w[i]);
                x[2 * i + 1] = bf16_hi(w[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = 0.0f;
            if (e0 + i < n)
                x[i] = f32 ? ((const float *)p)[e0 + i]
                           : bf16_to_f32(((const uint16_t *)p)[e0 + i]);
        }
    }
}

template <int V>
__device__ __forceinline__ void store(const float (&x)[V], void *p, bool f32, long long e0,
                                      long long n, bool whole) {
    if (whole) {
        if (f32) {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                __builtin_nontemporal_store(floatx4{x[i], x[i + 1], x[i + 2], x[i + 3]},
                                            (floatx4 *)((float *)p + e0 + i));
        } else {
            uint16_t *h = (uint16_t *)p + e0;
            uint32_t w[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            if (V == 8) __builtin_nontemporal_store(*(u32x4 *)w, (u32x4 *)h);
            else __builtin_nontemporal_store(*(u32x2 *)w, (u32x2 *)h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e0 + i < n) {
                if (f32) ((float *)p)[e0 + i] = x[i];
                else ((uint16_t *)p)[e0 + i] = (uint16_t)f32_to_bf16_bits(x[i]);
            }
    }
}

// The largest of 4 neighbouring lanes' values, in each of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
}

// Correctly rounded root of v >= 2^-96: the hardware's, off by one place at
// most, moved to a neighbour where the residual says so.  0, infinity and NaN
// fail both comparisons.  (Below, the residual loses bits, and the hardware
// takes a denormal for 0.)
__device__ __forceinline__ float root_of(float v) {
    const float s = __builtin_amdgcn_sqrtf(v);
    const float under = __uint_as_float(__float_as_uint(s) - 1);
    const float over = __uint_as_float(__float_as_uint(s) + 1);
    float r = fmaf(-under, s, v) <= 0.0f ? under : s;
    return fmaf(-over, s, v) > 0.0f ? over : r;
}

// The lane's 8 codes times s as fp32.
__device__ __forceinline__ void decode(float (&x)[8], u32x2 code, float s) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(code[w], false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(code[w], true);
        x[4 * w] = a[0] * s;
        x[4 * w + 1] = a[1] * s;
        x[4 * w + 2] = b[0] * s;
        x[4 * w + 3] = b[1] * s;
    }
}

// The 8 codes of a lane's values, in a block of 4 lanes; scale: exponent + 127
// of the block's power of two.  16 bits of rnd make the rounding (ROOT: the
// upper ones), as the top ones of the 20 that the conversion adds to the bits
// it drops (checked against that definition over values and bits).  A block
// with a value that is not finite is not-a-number throughout.
template <bool ROOT>
__device__ __forceinline__ u32x2 encode(const float (&x)[8], const uint32_t (&rnd)[8],
                                        uint32_t &scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = quad_max(top);
    // one more where the mantissa is over 1.75: 448 = 1.75 * 2^8
    int e = (int)((top + 0x1FFFFFu) >> 23) - 8;
    e = top == 0 ? 127 : max(e, 1);
    const bool finite = top < 0x7F800000u;
    if (!finite) e = 127;
    scale = (uint32_t)e;
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
    auto value = [&](int i) __attribute__((always_inline)) {
        const float y = x[i] * inv;
        // 2^-9: the least code that is not 0
        return ROOT ? fmaxf(y, x[i] > 0.0f ? 0.001953125f : 0.0f) : y;
    };
    auto seed = [&](int i) __attribute__((always_inline)) {
        return ROOT ? rnd[i] & 0xFFFF0000u : rnd[i] << 16;
    };
    u32x2 out;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int i = 4 * w;
        int word = 0;
        word = __builtin_amdgcn_cvt_sr_fp8_f32(value(i), seed(i), word, 0);
        word = __builtin_amdgcn_cvt_sr_fp8_f32(value(i + 1), seed(i + 1), word, 1);
        word = __builtin_amdgcn_cvt_sr_fp8_f32(value(i + 2), seed(i + 2), word, 2);
        word = __builtin_amdgcn_cvt_sr_fp8_f32(value(i + 3), seed(i + 3), word, 3);
        out[w] = finite ? (uint32_t)word : 0x7F7F7F7Fu;
    }
    return out;
}

template <bool Q8>
__global__ __launch_bounds__(THREADS, 8) void adamw(AdamwTable tab, AdamwParams p) {
#pragma clang fp contract(off)
    constexpr int V = Q8 ? 8 : 4;
    double lr = p.lr, bias1 = p.bias1, bias2 = p.bias2;
    uint32_t step = (uint32_t)p.step;
    if (p.steps) {
        const int64_t t = *p.steps + 1;
        step = (uint32_t)t;
        bias1 = -expm1((double)t * p.log_b1);
        bias2 = -expm1((double)t * p.log_b2);
    }
    if (p.lr_scale) lr *= (double)*p.lr_scale;
    const float size = (float)(lr / bias1), unbias = (float)(1.0 / sqrt(bias2));
    float f = 1.0f;
    if (p.norm) {
        // not fmin: a norm that is not a number has to reach the parameters
        const double c = p.max_norm / ((double)*p.norm + 1e-6);
        f = c >= 1.0 ? 1.0f : (float)c;
    }
    const int chunk = p.chunk;
    for (int c = blockIdx.x; c < tab.first[tab.count]; c += gridDim.x) {
        int lo = 0, hi = tab.count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tab.first[mid] <= c) lo = mid; else hi = mid;
        }
        const AdamwTensor &t = tab.t[lo];
        const bool pf32 = t.flags & ADAMW_PARAM_F32, gf32 = t.flags & ADAMW_GRAD_F32;
        const bool aligned = t.flags & ADAMW_ALIGNED;
        const long long n = t.n;
        const float decay = (float)(lr * t.decay);
        const uint32_t key = p.seed * 0x9E3779B1u + step * 0x85EBCA77u +
                             (uint32_t)(p.index0 + lo) * 0xC2B2AE3Du;
        const bool any = p.stochastic && !pf32 && !t.master;
        const long long start = (long long)(c - tab.first[lo]) * chunk;
        const long long end = min(start + chunk, n);
        // (whole blocks of 4 lanes go round together)
        for (long long b0 = start; b0 < end; b0 += THREADS * V) {
            const long long e0 = b0 + (long long)threadIdx.x * V;
            const bool live = e0 < n;
            const bool whole = e0 + V <= n, vec = whole && aligned;
            float x[V], g[V], m[V], v[V];
            u32x2 mc = {0, 0}, vc = {0, 0};
            uint32_t ms = 127, vs = 127;
            load(g, t.grad, gf32, e0, n, vec);
            if (t.master) load(x, t.master, true, e0, n, whole);
            else load(x, t.param, pf32, e0, n, vec);
            if constexpr (Q8) {
                if (whole) {
                    mc = __builtin_nontemporal_load((const u32x2 *)((const uint8_t *)t.m + e0));
                    vc = __builtin_nontemporal_load((const u32x2 *)((const uint8_t *)t.v + e0));
                } else if (live) {
                    for (int i = 0; i < n - e0; ++i) {
                        mc[i >> 2] |= (uint32_t)((const uint8_t *)t.m)[e0 + i] << (8 * (i & 3));
                        vc[i >> 2] |= (uint32_t)((const uint8_t *)t.v)[e0 + i] << (8 * (i & 3));
                    }
                }
                if (live) {
                    ms = t.m_scale[e0 / MOE_ADAMW_BLOCK];
                    vs = t.v_scale[e0 / MOE_ADAMW_BLOCK];
                }
                // (a power of two: the products with b1 are rounded alike)
                decode(m, mc, __uint_as_float(ms << 23) * p.b1);
                decode(v, vc, __uint_as_float(vs << 23));
            } else {
                load(m, t.m, true, e0, n, whole);
                load(v, t.v, true, e0, n, whole);
            }
            float root[V];
            uint32_t least = 0xFFFFFFFFu;            // (0 counts as the most)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float gi = g[i] * f;
                if (Q8) v[i] = v[i] * v[i];
                m[i] = (Q8 ? m[i] : m[i] * p.b1) + gi * p.c1;
                v[i] = v[i] * p.b2 + gi * gi * p.c2;
                root[i] = root_of(v[i]);
                least = min(least, __float_as_uint(v[i]) - 1);
            }
            if (least < 0x0F800000u - 1) {           // 2^-96
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (v[i] < 0x1p-96f) root[i] = root_of(v[i] * 0x1p64f) * 0x1p-32f;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float upd = size * m[i] * __builtin_amdgcn_rcpf(root[i] * unbias + p.eps);
                x[i] = x[i] - (x[i] * decay + upd);
            }
            uint32_t rnd[V];
            if (Q8 || any) {
                const uint32_t base = (uint32_t)e0 ^ key;       // (e0 % V == 0)
#pragma unroll
                for (int i = 0; i < V; ++i) rnd[i] = hash32(base ^ (uint32_t)i);
            }
            if (any) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    // (bits apart from the states'; a NaN stays one)
                    const uint32_t u = __float_as_uint(x[i]);
                    const uint32_t up = u + (hash32(rnd[i] ^ 0x5BD1E995u) >> 16);
                    x[i] = __uint_as_float((x[i] == x[i] ? up : u) & 0xFFFF0000u);
                }
            }
            if (t.master) store(x, t.master, true, e0, n, whole);
            store(x, t.param, pf32, e0, n, vec);
            if constexpr (Q8) {
                mc = encode<false>(m, rnd, ms);
                vc = encode<true>(root, rnd, vs);
                if (whole) {
                    __builtin_nontemporal_store(mc, (u32x2 *)((uint8_t *)t.m + e0));
                    __builtin_nontemporal_store(vc, (u32x2 *)((uint8_t *)t.v + e0));
                } else if (live) {
                    for (int i = 0; i < n - e0; ++i) {
                        ((uint8_t *)t.m)[e0 + i] = (uint8_t)(mc[i >> 2] >> (8 * (i & 3)));
                        ((uint8_t *)t.v)[e0 + i] = (uint8_t)(vc[i >> 2] >> (8 * (i & 3)));
                    }
                }
                if (live && (e0 & (MOE_ADAMW_BLOCK - 1)) == 0) {
                    t.m_scale[e0 / MOE_ADAMW_BLOCK] = (uint8_t)ms;
                    t.v_scale[e0 / MOE_ADAMW_BLOCK] = (uint8_t)vs;
                }
            } else {
                store(m, t.m, true, e0, n, whole);
                store(v, t.v, true, e0, n, whole);
            }
        }
    }
}

__global__ void adamw_tick(int64_t *steps) { *steps += 1; }

}  // namespace

hipError_t launch_adamw(const AdamwTable &tab, const AdamwParams &p, int bits,
                        int grid, hipStream_t s) {
    if (bits == 8)
        hipLaunchKernelGGL(adamw<true>, dim3(grid), dim3(THREADS), 0, s, tab, p);
    else
        hipLaunchKernelGGL(adamw<false>, dim3(grid), dim3(THREADS), 0, s, tab, p);
    return hipGetLastError();
}

hipError_t launch_adamw_tick(int64_t *steps, hipStream_t s) {
    hipLaunchKernelGGL(adamw_tick, dim3(1), dim3(1), 0, s, steps);
    return hipGetLastError();
}
