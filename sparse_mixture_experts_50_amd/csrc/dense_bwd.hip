// Products of rows by weights whose pre-activations are computed again for
// the gradient.
#include "dense_tile.h"

hipError_t launch_dense_grad_mfma(const DenseRows &p, hipStream_t s) {
    using namespace dn;
    switch (p.act) {
    case ACT_GELU: return launch_by_plan<1, false, false, DENSE_GRAD, ACT_GELU, false>(p, s);
    case ACT_SILU: return launch_by_plan<1, false, false, DENSE_GRAD, ACT_SILU, false>(p, s);
    case ACT_SWIGLU: return launch_by_plan<2, false, false, DENSE_GRAD, ACT_SWIGLU, false>(p, s);
    default: return launch_by_plan<2, false, false, DENSE_GRAD, ACT_GEGLU, false>(p, s);
    }
}
