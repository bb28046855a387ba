// The feed-forward products' kernel (ffn_gemm.cuh) whose sums are added up in segments: plain products
// with an fp32 result, alone or several in a launch, and the gated pair to 8 bits.
#include "ffn_gemm.cuh"

namespace wstma {

const void *ffn_plain_segments_fn(int cta_group, bool transposed)
{
    if (cta_group == 2)
        return transposed ? reinterpret_cast<const void *>(&ffn_gemm_kernel<2, true, kFfnPlain, 1, true>)
                          : reinterpret_cast<const void *>(&ffn_gemm_kernel<2, false, kFfnPlain, 1, true>);
    return transposed ? reinterpret_cast<const void *>(&ffn_gemm_kernel<1, true, kFfnPlain, 1, true>)
                      : reinterpret_cast<const void *>(&ffn_gemm_kernel<1, false, kFfnPlain, 1, true>);
}

const void *ffn_together_segments_fn(int cta_group)
{
    return cta_group == 2
               ? reinterpret_cast<const void *>(&ffn_gemm_kernel<2, false, kFfnPlain, kFfnMaxProducts, true>)
               : reinterpret_cast<const void *>(&ffn_gemm_kernel<1, false, kFfnPlain, kFfnMaxProducts, true>);
}

const void *ffn_gated_codes_fn(int cta_group)
{
    return cta_group == 2 ? reinterpret_cast<const void *>(&ffn_gemm_kernel<2, false, kFfnGated, 1, true>)
                          : reinterpret_cast<const void *>(&ffn_gemm_kernel<1, false, kFfnGated, 1, true>);
}

}  // namespace wstma
