// Gated linear layers: two products of rows by weights on one output tile,
// the activation of one times the other.
#include "dense_tile.h"

hipError_t launch_dense_gated_mfma(const DenseRows &p, hipStream_t s) {
    using namespace dn;
    return p.act == ACT_SWIGLU ? launch_forward<2, ACT_SWIGLU>(p, s)
                               : launch_forward<2, ACT_GEGLU>(p, s);
}
