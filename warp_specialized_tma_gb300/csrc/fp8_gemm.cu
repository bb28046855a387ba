// The block-scaled 8-bit product (fp8_gemm.cuh): one SM or a pair per tile, D as
// the accumulator or its transpose.
#include "fp8_gemm.cuh"

namespace wstma {

const void *fp8_gemm_kernel_fn(int cta_group, bool transposed)
{
    if (cta_group == 2)
        return transposed ? reinterpret_cast<const void *>(&fp8_gemm_kernel<2, true>)
                          : reinterpret_cast<const void *>(&fp8_gemm_kernel<2, false>);
    return transposed ? reinterpret_cast<const void *>(&fp8_gemm_kernel<1, true>)
                      : reinterpret_cast<const void *>(&fp8_gemm_kernel<1, false>);
}

}  // namespace wstma
