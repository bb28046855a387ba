// The feed-forward products' kernel (ffn_gemm.cuh) with the plain epilogue: one SM or a pair per
// tile, the result as the accumulator or its transpose.
#include "ffn_gemm.cuh"

namespace wstma {

const void *ffn_plain_fn(int cta_group, bool transposed)
{
    if (cta_group == 2)
        return transposed ? reinterpret_cast<const void *>(&ffn_gemm_kernel<2, true, kFfnPlain>)
                          : reinterpret_cast<const void *>(&ffn_gemm_kernel<2, false, kFfnPlain>);
    return transposed ? reinterpret_cast<const void *>(&ffn_gemm_kernel<1, true, kFfnPlain>)
                      : reinterpret_cast<const void *>(&ffn_gemm_kernel<1, false, kFfnPlain>);
}

const void *ffn_together_fn(int cta_group)
{
    return cta_group == 2 ? reinterpret_cast<const void *>(&ffn_gemm_kernel<2, false, kFfnPlain, kFfnMaxProducts>)
                          : reinterpret_cast<const void *>(&ffn_gemm_kernel<1, false, kFfnPlain, kFfnMaxProducts>);
}

}  // namespace wstma
