// The rows' gradient: dz W (+ du W3), plus what comes in beside it; in small
// tiles together with the column sums and the last rows, which nothing in this
// launch waits for.
#include "dense_parts.h"
#include "dense_tile.h"

namespace {

using namespace dn;

// The product by the first `rows` blocks, the others are sums_and_tails().
template <bool TWO, int EPI>
__global__ __launch_bounds__(256, 2) void dense_dx_sums(DenseRows p, DenseSums b, DenseTails t,
                                                        int rows) {
    typedef RowTiles<1, true, TWO, true> P;
    __shared__ u32x4 slot0[P::STAGE], slot1[P::STAGE], slot2[P::STAGE];
    static_assert(sizeof(slot0) >= dense_parts::SUMS_LDS, "sums in a slot");
    const int block = blockIdx.x;
    if (block >= rows)
        dense_parts::sums_and_tails<bf16>(b, t, block - rows, (float *)slot0);
    else if (EPI == DENSE_FORWARD && p.res)
        rows_work<1, true, TWO, EPI, ACT_NONE, true, mt::EVEN, true>(p, block, rows, slot0, slot1,
                                                                    slot2, nullptr);
    else
        rows_work<1, true, TWO, EPI, ACT_NONE, false, mt::EVEN, true>(p, block, rows, slot0, slot1,
                                                                     slot2, nullptr);
}

}  // namespace

hipError_t launch_dense_dx_mfma(const DenseRows &p, hipStream_t s) {
    // (of large tiles)
    if (p.res)
        return p.two ? launch_large<1, true, true, DENSE_FORWARD, ACT_NONE, true>(p, s)
                     : launch_large<1, true, false, DENSE_FORWARD, ACT_NONE, true>(p, s);
    return p.two ? launch_large<1, true, true, DENSE_FORWARD, ACT_NONE, false>(p, s)
                 : launch_large<1, true, false, DENSE_FORWARD, ACT_NONE, false>(p, s);
}

hipError_t launch_dense_dx_sums(const DenseRows &p, const DenseSums &b, const DenseTails &t,
                                hipStream_t s) {
    const int rows = mt::grid_for(p.plan.tiles(), 2);
    const dim3 grid(rows + dense_parts::sums_blocks(b, t, 256));
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, p, b, t, rows);
        return hipGetLastError();
    };
    if (p.plan.splits > 1)
        return p.two ? run(dense_dx_sums<true, DENSE_PLANE>)
                     : run(dense_dx_sums<false, DENSE_PLANE>);
    return p.two ? run(dense_dx_sums<true, DENSE_FORWARD>)
                 : run(dense_dx_sums<false, DENSE_FORWARD>);
}
