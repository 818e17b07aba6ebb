// Products of rows by weights that leave fp32 sums, over ranges of K.
#include "dense_tile.h"

hipError_t launch_dense_plane_mfma(const DenseRows &p, hipStream_t s) {
    using namespace dn;
    // (in small tiles, a sum of two is launched with the column sums)
    if (p.two) return launch_large<1, true, true, DENSE_PLANE, ACT_NONE, false>(p, s);
    if (p.bk) return launch_by_plan<1, true, false, DENSE_PLANE, ACT_NONE, false>(p, s);
    if (p.panels() == 2)
        return launch_by_plan<2, false, false, DENSE_PLANE, ACT_SWIGLU, false>(p, s);
    return launch_by_plan<1, false, false, DENSE_PLANE, ACT_NONE, false>(p, s);
}
