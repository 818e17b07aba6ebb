// The rows' gradient: dz W (+ du W3), plus what comes in beside it.
#include "dense_tile.h"

hipError_t launch_dense_dx_mfma(const DenseRows &p, hipStream_t s) {
    using namespace dn;
    return p.two ? launch_forward<1, true, true, ACT_NONE>(p, s)
                 : launch_forward<1, true, false, ACT_NONE>(p, s);
}
