// The block-scaled 8-bit product (fp8_gemm.cuh): one SM or a pair per tile, D as
// the accumulator or its transpose.
#include "fp8_gemm.cuh"

namespace wstma {

namespace {

template <int CG, bool kTransposed>
const void *pick(bool long_sums)
{
    return long_sums ? reinterpret_cast<const void *>(&fp8_gemm_kernel<CG, kTransposed, true>)
                     : reinterpret_cast<const void *>(&fp8_gemm_kernel<CG, kTransposed, false>);
}

}  // namespace

const void *fp8_gemm_kernel_fn(int cta_group, bool transposed, bool long_sums)
{
    if (cta_group == 2)
        return transposed ? pick<2, true>(long_sums) : pick<2, false>(long_sums);
    return transposed ? pick<1, true>(long_sums) : pick<1, false>(long_sums);
}

}  // namespace wstma
