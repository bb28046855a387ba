// Internal interface between the 8-bit operators' host library (fp8_api.cu)
// and their kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wstma {

// ----------------------------------------------------------------- quantiser
struct QuantizeParams {
    const void *x;
    int64_t ldx;
    int32_t R, C;
    int32_t x_fp32;
    int32_t tile;
    const float *row_factor;
    const void *column_factor;
    int32_t column_fp32;
    int32_t x_vec;       // rows of x are 16-byte aligned
    int32_t column_vec;  // column_factor is
    uint8_t *codes;
    int64_t ldq;
    uint8_t *scales;
    uint8_t *codes_t;
    int64_t ldqt;
    uint8_t *scales_t;
};

int launch_quantize(const QuantizeParams &p, cudaStream_t stream);  // a cudaError_t value

// ----------------------------------------------------------------- norm
struct NormParams {
    const uint16_t *x;
    int64_t ldx;
    const uint16_t *residual;
    int64_t ldr;
    const void *weight;
    int32_t w_fp32;
    int32_t R, C;
    float inv_c;  // 1 / C
    float eps;
    int32_t vec;    // every row is 16-byte aligned
    int32_t w_vec;  // the weight is
    uint16_t *h;
    int64_t ldh;
    uint8_t *codes;
    int64_t ldq;
    uint8_t *scales;
    float *rstd;
};

int launch_rmsnorm(const NormParams &p, int num_sms, cudaStream_t stream);

struct NormBackwardParams {
    const uint16_t *dy;
    int64_t lddy;
    const uint16_t *h;
    int64_t ldh;
    const void *weight;
    int32_t w_fp32;
    const float *rstd;
    const uint16_t *dres;
    int64_t lddr;
    uint16_t *dx;
    int64_t lddx;
    float *dw;
    int32_t R, C;
    int32_t vec;    // as in NormParams
    int32_t w_vec;
    float *partials;  // rmsnorm_backward_ctas() rows of C floats
};

int rmsnorm_backward_ctas(int64_t R, int64_t C, int num_sms);
int launch_rmsnorm_backward(const NormBackwardParams &p, int num_sms, cudaStream_t stream);

// ----------------------------------------------------------------- product
constexpr int kFp8RowsPerCta = 128;   // rows of the MMA's row side per CTA
constexpr int kFp8BlockK = 128;       // k per ring stage: 128 e4m3, one 128-byte swizzle row
constexpr int kFp8MaxWidth = 224;     // column side of a tile: two accumulators and the scales fit tensor memory
constexpr int kFp8Threads = 384;      // warps 0-3: producer, MMA, tensor memory, scales; 4-11: epilogue
constexpr int kFp8EpiWarps = 8;
constexpr int kFp8ScaleBytes = 512 + 1024;  // a stage's scales: 128 words of the row side, 256 of the column side
constexpr int kFp8StagingBytes = 4096;      // per epilogue warp: two buffers of 32 rows of 64 bytes
constexpr int kFp8MaxStages = 12;
constexpr int kFp8MaxLongWidth = 192;  // the same where an fp32 D's sums are held in registers (three chunks a warp)
constexpr int kFp8Segment = 32;             // k-blocks an accumulator takes before its sums are moved on (fp32 D)
constexpr int kFp8SpreadFrom = 5;            // CTAs of a cluster from which each of them adds up a part of their tile
constexpr int kFp8PartialFloats = kFp8RowsPerCta * 256;  // one CTA's fp32 partial of a split tile

struct Fp8GemmParams {
    int32_t rows;           // of the operand on the MMA's row side
    int32_t cols;           // rows of the operand on its column side
    int32_t num_k_blocks;
    int32_t num_row_tiles, num_col_tiles, num_tiles;
    int32_t raster_group;   // tiles are walked in bands of this many row tiles
    int32_t width;          // of a tile on the column side
    int32_t stages;
    int32_t sk_tiles;       // tiles [0, sk_tiles) are split along k among all clusters
    int64_t sk_units;       // sk_tiles * num_k_blocks
    int32_t cluster;        // > 1 (one SM per tile only): each tile is split among the CTAs of a cluster
    int32_t D_rows, D_cols;
    int32_t out_fp32;
    int32_t d_tma;          // D's layout allows TMA stores
    int64_t ldd;
    void *D;
    const uint32_t *s_rows; // scale words [ceil(K/512)][rows]
    const uint32_t *s_cols;
    float *partials;        // per CTA: kFp8PartialFloats
    uint32_t *flags;        // per CTA and epilogue warp: 1 once its partial can be read, 0 before the launch
    uint32_t *err;
    uint64_t watchdog_ns;
    int32_t fault_skip_it;
};

// Height in row tiles of the bands that tiles are walked in: 8 unless asked for, and never more
// than there are, so that a band's tiles can be counted in 32 bits.
inline int32_t fp8_raster_group(int64_t asked, int64_t row_tiles)
{
    const int64_t group = asked ? asked : 8;
    return (int32_t)(group < row_tiles ? group : row_tiles);
}

inline size_t fp8_stage_bytes(int cta_group, int width)
{
    return (size_t)kFp8RowsPerCta * kFp8BlockK + (size_t)(width / cta_group) * kFp8BlockK;
}

inline size_t fp8_smem_bytes(int cta_group, int width, int stages)
{
    return 1024 /* alignment slack */ + (size_t)stages * (fp8_stage_bytes(cta_group, width) + kFp8ScaleBytes) +
           (size_t)kFp8EpiWarps * kFp8StagingBytes + 512 /* barriers */;
}

// (CUtensorMap rows, CUtensorMap cols, CUtensorMap D, Fp8GemmParams)
// `long_sums`: fp32 D, accumulated in segments of kFp8Segment k-blocks.
const void *fp8_gemm_kernel_fn(int cta_group, bool transposed, bool long_sums);

// Sets the n flags of the split launch that follows on the stream to 0 (a cudaError_t value).
int launch_fp8_clear(uint32_t *flags, int32_t n, cudaStream_t stream);

}  // namespace wstma
