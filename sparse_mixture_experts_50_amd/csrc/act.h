// Activations of a pre-activation z (gated: times u) and their derivatives.
#pragma once

#include "common.h"

constexpr bool act_gated(int act) { return act == ACT_SWIGLU || act == ACT_GEGLU; }

// h, dh/dz and dh/du.  FAST: with the forms of common.h, gelu_erf's erfc and
// silu_f's exponential (relative errors of a few 1e-7); else the accurate
// library functions.
template <int ACT, bool FAST>
__device__ __forceinline__ void act_grad(float z, float u, float &h, float &hz,
                                         float &hu) {
    float a, da;
    if (ACT == ACT_NONE) {
        a = z;
        da = 1.0f;
    } else if (ACT == ACT_GELU || ACT == ACT_GEGLU) {
        // z Phi(z), Phi + z phi
        if (FAST) {
            a = gelu_erf(z);
            // Phi = a / z loses nothing but its value at 0
            const float pdf = 0.39894228f * __builtin_amdgcn_exp2f(z * z * -0.72134752f);
            const float az = fabsf(z);
            const float cdf = az > 1e-3f ? a * __builtin_amdgcn_rcpf(z)
                                         : fmaf(0.39894228f, z, 0.5f);
            da = fmaf(z, pdf, cdf);
        } else {
            const float cdf = 0.5f * erfcf(z * -0.70710678f);
            a = z * cdf;
            da = fmaf(z * 0.39894228f, expf(-0.5f * z * z), cdf);
        }
    } else {
        const float sg = FAST ? __builtin_amdgcn_rcpf(1.0f + __expf(-z))
                              : 1.0f / (1.0f + expf(-z));
        a = z * sg;
        da = fmaf(a, 1.0f - sg, sg);
    }
    if (act_gated(ACT)) {
        h = a * u;
        hz = da * u;
        hu = a;
    } else {
        h = a;
        hz = da;
        hu = 0.0f;
    }
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_value(float z, float u) {
    float a = z;
    if (ACT == ACT_GELU || ACT == ACT_GEGLU)
        a = FAST ? gelu_erf(z) : z * (0.5f * erfcf(z * -0.70710678f));
    else if (ACT != ACT_NONE)
        a = FAST ? silu_f(z) : z / (1.0f + expf(-z));
    return act_gated(ACT) ? a * u : a;
}
