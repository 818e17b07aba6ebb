// Host helpers shared by the C ABI's translation units: descriptor checks
// and the queries that every entry point makes before its first HIP call.
#pragma once

#include <math.h>

#include <atomic>

#include "../../include/moe.h"
#include "kernels.h"

namespace moe_host {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline int elem_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

inline bool expert_choice(const moe_desc *d) {
    return d->routing == MOE_ROUTE_EXPERT_CHOICE;
}

// Routed expert rows: T*k assignments, or E*C picks for expert choice.
inline long long routed_rows(const moe_desc *d) {
    return expert_choice(d) ? (long long)d->E * d->capacity
                            : (long long)d->T * d->k;
}

inline int check_desc(const moe_desc *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->T < 0 || d->E < 1 || d->k < 1 || d->k > d->E || d->d < 1 ||
        d->d_ff < 1 || d->capacity < -1 ||
        (d->n_shared != 0 && d->n_shared != 1) ||
        (d->routing != MOE_ROUTE_TOPK && !expert_choice(d)))
        return MOE_ERR_INVALID_ARG;
    if (expert_choice(d) &&
        (d->k != d->E || d->capacity < 0 || d->capacity > d->T))
        return MOE_ERR_INVALID_ARG;
    if (d->expert_fp8 != 0 && d->expert_fp8 != 1) return MOE_ERR_INVALID_ARG;
    if (d->activation < MOE_ACT_GELU || d->activation > MOE_ACT_SWIGLU)
        return MOE_ERR_INVALID_ARG;
    // the gated bf16 up GEMM runs on tiles whose waves cover whole 64-column
    // chunks of the 2*d_ff virtual panel (256-column tiles, 64-column
    // streaming units)
    if (d->activation == MOE_ACT_SWIGLU && d->dtype == MOE_BF16 &&
        d->d_ff % 128 != 0)
        return MOE_ERR_UNSUPPORTED;
    if (d->dtype != MOE_F32 && d->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    // FP8 weights run on the weight-streaming kernel: its four K quarters
    // hold whole 256-deep load batches
    if (d->expert_fp8 && (d->dtype != MOE_BF16 || d->d % 1024 != 0 ||
                          d->d_ff % 1024 != 0))
        return MOE_ERR_UNSUPPORTED;
    if (d->E > MOE_MAX_E || (!expert_choice(d) && d->k > 64))
        return MOE_ERR_UNSUPPORTED;
    if (d->d % 64 != 0 || d->d_ff % 64 != 0) return MOE_ERR_UNSUPPORTED;
    // 32-bit element offsets inside the kernels
    if ((double)d->T * d->k >= 2147483647.0) return MOE_ERR_UNSUPPORTED;
    const double rows = (double)routed_rows(d) + (double)d->n_shared * d->T;
    if (rows * d->d_ff >= 2147483647.0 || rows * d->d >= 2147483647.0 ||
        2.0 * d->d * d->d_ff >= 2147483647.0)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

inline char *at(void *ws, size_t off) { return (char *)ws + off; }

inline int to_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Compute units of the current device (host query, cached per device).
// The cache is the library's one piece of state kept between calls: a
// per-device constant, written with relaxed atomics, so concurrent first
// calls at worst both query the device and store the same value.
inline int device_cus() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount,
                                  dev) != hipSuccess || n <= 0)
            n = 256;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace moe_host
