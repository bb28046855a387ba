// Internal interface between the feed-forward operators' host library (ffn_api.cu)
// and their kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wstma {

// ----------------------------------------------------------------- product
constexpr int kFfnRowsPerCta = 128;  // rows of the MMA's row side per CTA
constexpr int kFfnBlockK = 64;       // k per ring stage: 64 bf16, one 128-byte swizzle row
constexpr int kFfnMaxWidth = 256;    // column side of a tile: two accumulators fill tensor memory
constexpr int kFfnDualWidth = 128;   // the same where a tile has a gate's and an up projection's accumulators
constexpr int kFfnThreads = 384;     // warps 0-3: producer, MMA, tensor memory; 4-11: epilogue
constexpr int kFfnEpiWarps = 8;
constexpr int kFfnPieceBytes = 2048;     // 32 rows of 64 bytes
constexpr int kFfnStagingBytes = 2 * kFfnPieceBytes;  // per epilogue warp
constexpr int kFfnMaxStages = 12;
constexpr int kFfnPartialFloats = kFfnRowsPerCta * 256;  // one CTA's fp32 partial of a split tile
constexpr int kFfnMaxCluster = 8;
// k-blocks that an accumulator takes before its sums are moved on
constexpr int kFfnSegment = 8;        // of an fp32 result
constexpr int kFfnCodesSegment = 16;  // of 8-bit codes
// The widest tile whose sums are then held in registers: four chunks a warp for the large tiles of SM pairs, three
// elsewhere (with four 64 x 8192 x 8192 took 32.8 us, not 28.9, for what spills).
__host__ __device__ constexpr int ffn_long_width(int cta_group, bool transposed)
{
    return cta_group == 2 && !transposed ? 256 : 192;
}
constexpr int kFfnEarlyColumns = 64;  // of a transposed tile, whose residual is loaded ahead: each half's first chunk
constexpr int kFfnBarrierBytes = 512;
constexpr int kFfnBlockBytes = 1024;  // where the warps of the gated form to 8 bits exchange scales

enum FfnEpilogue : int32_t {
    kFfnPlain = 0,   // D0 = act(S + bias) + residual, D1 = S + bias
    kFfnGated = 1,   // S = gate, S2 = up: D0 = act(S) S2, D1 = S, D2 = S2
    kFfnGrad = 2     // S = dh, with g and u: D0 = dh u act'(g), D1 = dh act(g), D2 = act(g) u
};

enum FfnAct : int32_t { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// One result: rows x cols of the product (never its transpose).
struct FfnOut {
    void *p = nullptr;
    int64_t ld = 0;
    int32_t tma = 0;  // its layout allows TMA stores
};

// One bf16 matrix that an epilogue reads, of the results' size; or 8-bit codes with scales.  Rows
// are 16-byte aligned where a thread reads a row (the result is not transposed).
struct FfnAux {
    const void *p = nullptr;
    int64_t ld = 0;
    const uint8_t *scales = nullptr;  // not null: codes
    int32_t sectors = 0;  // rows start at multiples of 32 bytes
};

struct FfnParams {
    int32_t rows, cols;        // of the accumulator: the operands' row side and column side
    int32_t D_rows, D_cols;    // of the results
    int32_t num_k_blocks;      // of all products that are added up
    int32_t k_split;           // k-blocks of the first of them; the second's operands are maps 1
    int32_t num_row_tiles, num_col_tiles, num_tiles;
    int32_t row_split;         // row tiles of the first of two row operands, whose results are D0 and D1
    int32_t r_mn, c_mn;        // operand's rows are contiguous (an operand is contiguous along k otherwise)
    int32_t width;             // of a tile on the column side, per accumulator
    int32_t c_rows;            // rows of the column operand that a CTA loads per stage
    int32_t r_rows;            // and of the row operand (of each, transposed gated): 128, or 64 where there are no more
    int32_t stage_bytes;       // of the ring, the same for all products of a launch
    int32_t stages;
    int32_t raster_group;
    uint32_t band_tiles;       // ffn_band_tiles()
    int32_t segment;           // kernels that add up segments: their k-blocks (a bf16 result's: all)
    int32_t sk_tiles;          // tiles [0, sk_tiles) are split along k among all clusters
    int64_t sk_units;          // sk_tiles * num_k_blocks
    int32_t cluster;           // > 1 (one SM per tile only): each tile is split among the CTAs of a cluster
    int32_t act;
    int32_t out_fp32;          // D0 (kFfnPlain)
    FfnOut D[3];
    FfnAux aux[2];             // kFfnPlain: residual; kFfnGrad: g, u
    const void *bias;
    int32_t bias_fp32;
    int32_t save;              // kFfnPlain: 1 = D1; kFfnGated: 1 = D1 and D2, 2 = codes, by a kernel of their own
    uint8_t *codes[2];         // kFfnGated, save == 2: of g and u
    uint8_t *scales[2];
    int64_t ldq[2];
    float *partials;
    uint32_t *flags;
    uint32_t *err;
    uint64_t watchdog_ns;
    int32_t fault_skip_it;
};

struct FfnMaps {
    CUtensorMap R[2], C[2], D[3];
};

// The products of one launch; more than one (of the plain epilogue, none split) one after the other,
// product i's tiles first[i] .. first[i + 1] - 1.
constexpr int kFfnMaxProducts = 3;
template <int kN>
struct FfnArgs {
    FfnMaps maps[kN];
    FfnParams p[kN];
    int32_t first[kN + 1];
};

// Tiles of a band of row tiles, as many as 32 bits hold: there are fewer in all.
inline uint32_t ffn_band_tiles(int64_t raster_group, int64_t col_tiles)
{
    const int64_t n = raster_group * col_tiles;
    return n < 0x7FFFFFFF ? (uint32_t)n : 0x7FFFFFFFu;
}

inline int ffn_chunk_rows(bool mn, int rows) { return mn ? (rows + 63) / 64 * 64 : rows; }

inline size_t ffn_smem_bytes(size_t stage_bytes, int stages)
{
    return 1024 /* alignment slack */ + (size_t)stages * stage_bytes + (size_t)kFfnEpiWarps * kFfnStagingBytes +
           kFfnBarrierBytes + kFfnBlockBytes;
}

// (FfnArgs<1>), the last (FfnArgs<kFfnMaxProducts>).  Sums that are not rounded to bf16 at once, but
// stay in fp32 or go to 8 bits, are added up in segments (`segments`, `codes`).
const void *ffn_plain_fn(int cta_group, bool transposed);
const void *ffn_plain_segments_fn(int cta_group, bool transposed);
const void *ffn_gated_fn(int cta_group, bool transposed);
const void *ffn_gated_codes_fn(int cta_group);
const void *ffn_grad_fn(int cta_group, bool transposed);
const void *ffn_together_fn(int cta_group);
const void *ffn_together_segments_fn(int cta_group);

uint32_t *ffn_status_word();  // of the current device, or null

// ----------------------------------------------------------------- few tokens
constexpr int kFfnStreamTokens = 32;  // at most

struct FfnStreamParams {
    const uint16_t *x;
    int64_t ldx;
    const uint16_t *w[2];  // the second null, or gated
    int64_t ldw[2];
    int32_t M, N, K;       // rows of x and w 16-byte aligned, K a multiple of 8
    int32_t groups;        // the launch's: of up to 16 rows that a CTA works on at once
    int32_t act;
    int32_t bias_fp32;
    const void *bias;
    const uint16_t *residual;
    int64_t ldr;
    FfnOut D[3];           // as in FfnParams
    int32_t out_fp32;
    int32_t save;
};

int64_t ffn_stream_rows(int num_sms);  // N at most
int launch_ffn_stream(FfnStreamParams &p, int num_sms, cudaStream_t stream);  // a cudaError_t value

constexpr int kFfnStreamBackTokens = 16;  // at most

// D0 = d[0] w[0] (+ d[1] w[1]); with aux, the gated gradient's results (kFfnGrad) of that sum.
struct FfnStreamBackParams {
    const uint16_t *d[2];  // M x N, rows 8-byte aligned
    int64_t ldd[2];
    const uint16_t *w[2];  // N x C, rows 16-byte aligned
    int64_t ldw[2];
    int32_t products;
    int32_t M, N, C;
    int32_t ranks, share, groups;  // the launch's: CTAs of a cluster, eights of columns of one, their groups
    int32_t act;
    FfnAux aux[2];         // g and u
    FfnOut D[3];
};

int64_t ffn_stream_back_columns(int num_sms);  // C at most
int launch_ffn_stream_back(FfnStreamBackParams &p, int device, int num_sms, cudaStream_t stream);

// ----------------------------------------------------------------- rows
// Copies of R rows of C bf16 to rows that are 16-byte aligned (ldd a multiple of 8), a cudaError_t value.
struct FfnPackJob {
    const uint16_t *src;
    int64_t lds;
    uint16_t *dst;
    int64_t ldd;
    int64_t R;
    int32_t C;
    int32_t blocks;  // the launch's: units of a row, and in all; whether rows are 16-byte aligned
    int64_t units;
    int32_t vec;
};
struct FfnPackJobs {
    FfnPackJob job[7];  // gated_backward reads seven matrices that may be copied
    int n;
    int64_t units;
    uint32_t *flags;  // set to 0 on the way
    int32_t num_flags;
};
int launch_ffn_pack(FfnPackJobs &jobs, int num_sms, cudaStream_t stream);

struct FfnSlopeParams {
    const uint16_t *dy;
    int64_t lddy;
    const uint16_t *z;  // null: no activation
    int64_t ldz;
    uint16_t *dz;       // null without an activation
    int64_t lddz;       // a multiple of 8, dz 16-byte aligned
    float *dbias;       // or null
    float *partials;    // ffn_slope_slices() rows of N floats, where dbias is not null
    int32_t R, C;
    int32_t vec;        // rows of dy and z are 16-byte aligned
    int32_t act;
};
int ffn_slope_slices(int64_t R, int64_t C, int num_sms);
int launch_ffn_slope(const FfnSlopeParams &p, int num_sms, cudaStream_t stream);

}  // namespace wstma
