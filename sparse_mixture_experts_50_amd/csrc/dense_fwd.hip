// Linear layers: products of rows by weights with the forward's epilogue.
#include "dense_tile.h"

hipError_t launch_dense_forward_mfma(const DenseRows &p, hipStream_t s) {
    using namespace dn;
    if (p.bk) return launch_dense_dx_mfma(p, s);
    if (p.panels() == 2) return launch_dense_gated_mfma(p, s);
    switch (p.act) {
    case ACT_GELU: return launch_forward<1, ACT_GELU>(p, s);
    case ACT_SILU: return launch_forward<1, ACT_SILU>(p, s);
    default: return launch_forward<1, ACT_NONE>(p, s);
    }
}
