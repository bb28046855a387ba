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

// The flags of a split launch, ahead of it.  Not left at 0 by the launch before: one that
// gave up leaves some of them set, and the next would take old partials for its own.  Hidden
// behind the kernel before: 0.9 us of 114 for 6143 x 5999 x 4104, nothing of 8192^3.
__global__ void __launch_bounds__(256) fp8_clear_kernel(uint32_t *flags, int32_t n)
{
    // the product's start overlaps the kernel before this one, and its wait is for this one
    grid_launch_dependents();
    grid_dependency_wait();
    for (int32_t i = (int32_t)threadIdx.x; i < n; i += 256)
        flags[i] = 0u;
}

}  // namespace

int launch_fp8_clear(uint32_t *flags, int32_t n, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp8_clear_kernel, flags, n);
}

const void *fp8_gemm_kernel_fn(int cta_group, bool transposed, bool long_sums)
{
    if (cta_group == 2)
        return transposed ? pick<2, true>(long_sums) : pick<2, false>(long_sums);
    return transposed ? pick<1, true>(long_sums) : pick<1, false>(long_sums);
}

}  // namespace wstma
