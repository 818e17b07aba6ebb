// Host side of moe_adamw_step: argument checks and the launches' tables.
#include "../../include/moe.h"
#include "adamw.h"
#include "host.h"

using namespace moe_host;

namespace {

int check_tensor(const moe_adamw *h, const moe_adamw_tensor &t) {
    if (t.numel < 0 || !(t.weight_decay >= 0.0) || t.weight_decay > 1e30)
        return MOE_ERR_INVALID_ARG;
    if ((t.param_dtype != MOE_F32 && t.param_dtype != MOE_BF16) ||
        (t.grad_dtype != MOE_F32 && t.grad_dtype != MOE_BF16))
        return MOE_ERR_UNSUPPORTED;
    if (t.numel == 0) return MOE_OK;
    // chunk numbers are 32-bit within a launch
    if (t.numel > (1ll << 40)) return MOE_ERR_UNSUPPORTED;
    const bool q8 = h->state_bits == 8;
    if (!t.param || !t.grad || !t.m || !t.v || (q8 && (!t.m_scale || !t.v_scale)) ||
        (t.master && t.param_dtype != MOE_BF16))
        return MOE_ERR_INVALID_ARG;
    if ((uintptr_t)t.param % elem_bytes(t.param_dtype) ||
        (uintptr_t)t.grad % elem_bytes(t.grad_dtype) || !aligned(t.master) ||
        !aligned(t.m) || !aligned(t.v))
        return MOE_ERR_INVALID_ARG;
    const void *own[] = {t.param, t.grad, t.m, t.v, t.master,
                         q8 ? t.m_scale : nullptr, q8 ? t.v_scale : nullptr,
                         h->steps, h->lr_scale, h->norm};
    constexpr int count = sizeof(own) / sizeof(own[0]);
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < i; ++j)
            // (two of the call's inputs may be one; a tensor's are its own)
            if (own[i] && own[i] == own[j] && j < 7) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace

extern "C" int moe_adamw_step(const moe_adamw *h, int32_t n,
                              const moe_adamw_tensor *tensors, void *stream) {
    if (!h || n < 0 || (n > 0 && !tensors)) return MOE_ERR_INVALID_ARG;
    // (negated, so that what is not a number fails; 1 / eps has to be finite)
    if (!(h->lr >= 0.0 && h->lr < 1e30) || !(h->beta1 >= 0.0 && h->beta1 < 1.0) ||
        !(h->beta2 >= 0.0 && h->beta2 < 1.0) || !(h->eps >= 0x1p-126 && h->eps < 1e30) ||
        (!h->steps && h->step < 1) ||
        (h->norm && !(h->max_norm >= 0.0 && h->max_norm <= 1.7e308)) ||
        (h->stochastic != 0 && h->stochastic != 1) ||
        ((uintptr_t)h->steps & 7) || ((uintptr_t)h->lr_scale & 3) ||
        ((uintptr_t)h->norm & 3) ||
        (h->steps && ((const void *)h->steps == h->lr_scale ||
                      (const void *)h->steps == h->norm)))
        return MOE_ERR_INVALID_ARG;
    if (h->state_bits != 8 && h->state_bits != 32) return MOE_ERR_UNSUPPORTED;
    for (int i = 0; i < n; ++i) {
        const int st = check_tensor(h, tensors[i]);
        if (st != MOE_OK) return st;
    }
    hipStream_t s = (hipStream_t)stream;
    AdamwParams p = {};
    p.lr = h->lr;
    p.log_b1 = log(h->beta1);
    p.log_b2 = log(h->beta2);
    p.steps = h->steps;
    p.step = h->step;
    if (!h->steps) {
        p.bias1 = -expm1((double)h->step * p.log_b1);
        p.bias2 = -expm1((double)h->step * p.log_b2);
    }
    p.lr_scale = h->lr_scale;
    p.norm = h->norm;
    p.max_norm = h->max_norm;
    p.b1 = (float)h->beta1;
    p.c1 = (float)(1.0 - h->beta1);
    p.b2 = (float)h->beta2;
    p.c2 = (float)(1.0 - h->beta2);
    p.eps = (float)h->eps;
    p.seed = h->seed;
    p.stochastic = h->stochastic;
    const int most = 8 * device_cus();
    double total = 0;
    for (int i = 0; i < n; ++i) total += (double)tensors[i].numel;
    p.chunk = MOE_ADAMW_CHUNK;
    while (p.chunk > MOE_ADAMW_LEAST && total < (double)p.chunk * most) p.chunk /= 2;
    // the tensors from i on that one launch takes
    auto fill = [&](int &i, AdamwTable &tab) {
        tab = AdamwTable{};
        long long chunks = 0;
        for (; i < n && tab.count < MOE_ADAMW_TENSORS; ++i) {
            const moe_adamw_tensor &t = tensors[i];
            const long long own = (t.numel + p.chunk - 1) / p.chunk;
            if (chunks + own > 0x7fffffffll - most) break;
            const bool ok = aligned(t.param) && aligned(t.grad);
            const int flags = (t.param_dtype == MOE_F32 ? ADAMW_PARAM_F32 : 0) |
                              (t.grad_dtype == MOE_F32 ? ADAMW_GRAD_F32 : 0) |
                              (ok ? ADAMW_ALIGNED : 0);
            tab.t[tab.count] = {t.param, t.grad, t.master, t.m, t.v, t.m_scale,
                                t.v_scale, (long long)t.numel, t.weight_decay, flags, 0};
            tab.first[tab.count++] = (int32_t)chunks;
            chunks += own;
        }
        tab.first[tab.count] = (int32_t)chunks;
        return chunks;
    };
    AdamwTable tab;
    for (int i = 0; i < n;) {
        p.index0 = i;
        const long long chunks = fill(i, tab);
        if (chunks == 0) continue;
        const int grid = (int)(chunks < most ? chunks : most);
        if (launch_adamw(tab, p, h->state_bits, grid, s) != hipSuccess)
            return MOE_ERR_HIP;
    }
    if (h->steps && launch_adamw_tick(h->steps, s) != hipSuccess) return MOE_ERR_HIP;
    return MOE_OK;
}
