// The feed-forward products' kernel (ffn_gemm.cuh) with the gated epilogue: one SM or a pair per
// tile, the result as the accumulator or its transpose.
#include "ffn_gemm.cuh"

namespace wstma {

const void *ffn_gated_fn(int cta_group, bool transposed)
{
    if (cta_group == 2)
        return transposed ? reinterpret_cast<const void *>(&ffn_gemm_kernel<2, true, kFfnGated>)
                          : reinterpret_cast<const void *>(&ffn_gemm_kernel<2, false, kFfnGated>);
    return transposed ? reinterpret_cast<const void *>(&ffn_gemm_kernel<1, true, kFfnGated>)
                      : reinterpret_cast<const void *>(&ffn_gemm_kernel<1, false, kFfnGated>);
}

}  // namespace wstma
