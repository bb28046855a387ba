// The block-scaled 8-bit product: D = A * B^T of two quantised matrices.
//
//   D[m][n] = sum over blocks b of 128: 2^(ea[m][b]) 2^(eb[n][b]) sum_{k in b} a[m][k] b[n][k]
//
// tcgen05.mma's block-scaled kind multiplies each product of 32 elements of k by
// the two rows' e8m0 scales before adding it to the fp32 accumulator; four such
// MMAs make a block of 128, with the same scales.  So the scales cost no pass over
// the accumulator: they are copied to tensor memory once per four blocks (one
// 32-bit word per row) and picked by a byte index in the instruction descriptor.
//
// One of A and B is on the MMA's row side (128 rows to a CTA, 256 to an SM pair),
// the other on its column side (`width` <= 224 columns to a tile).  For a few
// tokens the weights take the row side, and the accumulator holds D transposed.
//
// Roles (384 threads, one CTA per SM):
//   warp 0           TMA producer: per (item, k-block) wait "empty", load both tiles
//   warp 1           MMA issuer (leader CTA only in pairs), one elected lane
//   warps 2, 3       scales: 4 k-blocks' words per row from global to shared memory,
//                    with the ring stage of the first of them; warp 2 also allocates
//                    and frees tensor memory
//   warps 4..11      epilogue: tensor memory -> registers -> D
//
// Work: tiles [0, sk_tiles) are split along k, their (tile, k-block) units cut
// into one contiguous range per cluster; the other tiles are walked whole.  The
// pieces of a split tile meet through global memory as fp32, added in range
// order by the piece that holds k-block 0, so the result is the same every time.
// A flag per CTA and epilogue warp says that its partial is there; a kernel of one
// CTA ahead of each such launch sets them to 0 (fp8_clear_kernel).
// Where the tiles times 2..8 nearly fill the GPU, the CTAs of a thread-block
// cluster share a tile instead (the same ranges, every C-th of which starts at a
// tile's start), and the pieces meet through distributed shared memory: the
// exchange through global memory takes 4 us at the end of a 17 us call.
// Every wait is bounded by the watchdog (WaitCtl in ptx.cuh).
//
// What bounds it, and what it measured.  Many tokens: the tensor pipe.  An SM pair's
// 256 x 224 tile keeps both accumulators in tensor memory beside the scales and asks
// L2 for the fewest bytes a product (17 TB/s all the same); 8192^3 takes 305 us in a
// burst, 3.6 PFLOP/s, with the pipe 89 % active, and 360 us under the power cap.  On the
// GPU alone (replayed from a graph) and, in brackets, as a call on changing inputs: 6143 x
// 5999 x 4104 99 us, 3.1 PFLOP/s (114); an fp32 D 2048 x 2048 x 32768 95 us, 2.9 PFLOP/s
// (105).  Few tokens: the weights' stream, 67 MB in 16.9 us (4.0 TB/s) for 1 x 8192 x 8192
// (17.4), of which about 5 us are the launch, the first loads and the pieces' meeting.
#pragma once

#include <stdint.h>

#include "fp8_kernels.h"
#include "fp8_ptx.cuh"
#include "gemm_common.cuh"

namespace wstma {

// Copies and MMAs in flight are waited for at a CTA's end however short the watchdog's
// limit is: they land in a few microseconds, and must not outlive it.
constexpr uint64_t kFp8DrainNs = 20000000;

struct Fp8Item {
    int32_t tile, kb0, kb1;
};

__host__ __device__ __forceinline__ int64_t fp8_range_begin(int64_t units, int32_t clusters, int32_t c)
{
    return (int64_t)c * units / clusters;
}

__host__ __device__ __forceinline__ bool fp8_range_holds(int64_t units, int32_t clusters, int32_t c)
{
    return fp8_range_begin(units, clusters, c) < fp8_range_begin(units, clusters, c + 1);
}

// The range that holds unit u.
__host__ __device__ __forceinline__ int32_t fp8_range_of(int64_t units, int32_t clusters, int64_t u)
{
    return (int32_t)(((u + 1) * clusters + units - 1) / units) - 1;
}

// End of the accumulation that k-block kb belongs to (kLong): a multiple of 4, so
// that a group of scales never spans two.
__device__ __forceinline__ int32_t fp8_segment_end(int32_t kb) { return kb / kFp8Segment * kFp8Segment + kFp8Segment; }
static_assert(kFp8Segment % 4 == 0, "scales come in groups of 4 k-blocks");

// A cluster's items in order: its range of the split tiles' units (a range is no
// longer than a tile, since sk_tiles < clusters, so it touches at most two
// tiles), then every clusters-th whole tile.  A range's first piece may start
// inside a tile (it then leaves a partial); a piece that starts at k-block 0 and
// does not reach the tile's end is the last of its range.  So no cluster waits
// for a partial before it has left its own.
struct Fp8Work {
    int64_t u, u_end;
    int32_t dp, C, T, KB;

    __host__ __device__ __forceinline__ void init(const Fp8GemmParams &p, int32_t cluster, int32_t clusters)
    {
        KB = p.num_k_blocks;
        C = clusters;
        T = p.num_tiles;
        dp = p.sk_tiles + cluster;
        u = fp8_range_begin(p.sk_units, clusters, cluster);
        u_end = fp8_range_begin(p.sk_units, clusters, cluster + 1);
    }

    __host__ __device__ __forceinline__ bool next(Fp8Item &w)
    {
        if (u < u_end) {
            const int64_t t = u / KB;
            const int64_t k0 = u - t * KB;
            const int64_t k1 = k0 + (u_end - u) < KB ? k0 + (u_end - u) : KB;
            w.tile = (int32_t)t;
            w.kb0 = (int32_t)k0;
            w.kb1 = (int32_t)k1;
            u += k1 - k0;
            return true;
        }
        if (dp < T) {
            w.tile = dp;
            w.kb0 = 0;
            w.kb1 = KB;
            dp += C;
            return true;
        }
        return false;
    }
};

// Tile -> (row tile, column tile): bands of raster_group row tiles, walked column
// by column, odd bands right to left, so that tiles running at the same time
// share operands in L2.
__host__ __device__ __forceinline__ TileCoord fp8_tile_coord(int32_t t, const Fp8GemmParams &p)
{
    const int32_t span = p.raster_group * p.num_col_tiles;
    const int32_t band = t / span;
    const int32_t first = band * p.raster_group;
    const int32_t rows = p.num_row_tiles - first < p.raster_group ? p.num_row_tiles - first : p.raster_group;
    const int32_t r = t - band * span;
    const int32_t col = r / rows;
    return {first + r % rows, (band & 1) ? p.num_col_tiles - 1 - col : col};
}

constexpr uint32_t kFp8ScaleCol = 2u * kFp8MaxWidth;  // tensor-memory columns of the scales: two buffers of 32
constexpr uint32_t kFp8ScaleColB = 16u;               // inside a buffer: row side at 0..3, column side at 16..23

constexpr uint32_t kFp8PieceBytes = 2048;  // a warp stages two

// A piece of D, staged in shared memory as 32 rows of 64 bytes (32 columns of bf16,
// 16 of fp32) in the TMA swizzle of that row size: byte offset of element (r, c).
__device__ __forceinline__ uint32_t fp8_piece_offset(uint32_t r, uint32_t c, bool fp32)
{
    const uint32_t byte = fp32 ? c * 4u : c * 2u;
    return r * 64u + (((byte >> 4) ^ ((r >> 1) & 3u)) << 4) + (byte & 15u);
}

// Stores 32 x 32 staged elements (a piece of bf16, or two of fp32 side by side) by the
// warp, a row at a time, an element a lane: whatever the row's alignment, its
// sectors then leave in one request (pairs of bf16 to a lane diverge by alignment
// and split the odd rows' sectors).  Eight rows' loads come before their stores.
__device__ __forceinline__ void fp8_store_masked(uint32_t from, int lane, int32_t x, int32_t y, bool fp32,
                                                 const Fp8GemmParams &p)
{
    const int32_t rows = p.D_rows - y < 32 ? p.D_rows - y : 32;
    if (x + lane >= p.D_cols)
        return;
    const int64_t at = (int64_t)y * p.ldd + x + lane;
    if (fp32) {
        float *dst = static_cast<float *>(p.D) + at;
        from += lane >= 16 ? kFp8PieceBytes : 0u;
        for (int32_t r = 0; r < rows; r += 8) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[k] = ld_shared_u32(from + fp8_piece_offset((uint32_t)(r + k), (uint32_t)lane & 15u, true));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (r + k < rows)
                    *dst = __uint_as_float(w[k]);
                dst += p.ldd;
            }
        }
        return;
    }
    uint16_t *dst = static_cast<uint16_t *>(p.D) + at;
    for (int32_t r = 0; r < rows; r += 8) {
        uint16_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            asm volatile("ld.shared.u16 %0, [%1];"
                         : "=h"(w[k])
                         : "r"(from + fp8_piece_offset((uint32_t)(r + k), (uint32_t)lane, false))
                         : "memory");
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (r + k < rows)
                *dst = w[k];
            dst += p.ldd;
        }
    }
}

// Stores one or two staged pieces, at D[y0..y0+31][x0..] and D[y1..][x1..], by TMA
// stores, or, where D's layout or its last columns do not allow one (a TMA store
// writes whole 16-byte groups), by the warp's masked stores.  Pieces outside D are
// dropped.  One proxy fence serves both pieces: it takes 300 clocks.
__device__ __forceinline__ void fp8_store_pieces(uint32_t staging, int lane, const CUtensorMap *tmD, int pieces,
                                                 int32_t x0, int32_t y0, int32_t x1, int32_t y1, bool fp32,
                                                 const Fp8GemmParams &p)
{
    const int32_t wide = fp32 ? 16 : 32;
    const int32_t far = pieces == 2 && x1 > x0 ? x1 : x0;
    if (p.d_tma && (far + wide <= p.D_cols || p.D_cols % (fp32 ? 4 : 8) == 0)) {
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (x0 < p.D_cols && y0 < p.D_rows)
                tma_store_2d(tmD, staging, x0, y0);
            if (pieces == 2 && x1 < p.D_cols && y1 < p.D_rows)
                tma_store_2d(tmD, staging + kFp8PieceBytes, x1, y1);
            bulk_commit_group();
        }
        return;
    }
    __syncwarp();
    fp8_store_masked(staging, lane, x0, y0, fp32, p);
    if (!fp32 && pieces == 2)
        fp8_store_masked(staging + kFp8PieceBytes, lane, x1, y1, false, p);
}

// The staging buffers are free once their last stores have read them (or every
// lane has finished the masked path's loads).
__device__ __forceinline__ void fp8_staging_free(int lane)
{
    if (lane == 0)
        bulk_wait_read_all();
    __syncwarp();
}

// Stages 32 accumulator rows x 32 columns (thread = row) of bf16 as one piece.
__device__ __forceinline__ void fp8_stage_bf16(const uint32_t (&v)[32], uint32_t at, int lane)
{
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u)
        st_shared_v4(at + fp8_piece_offset((uint32_t)lane, 8 * u, false), pack_bf16x2(v[8 * u], v[8 * u + 1]),
                     pack_bf16x2(v[8 * u + 2], v[8 * u + 3]), pack_bf16x2(v[8 * u + 4], v[8 * u + 5]),
                     pack_bf16x2(v[8 * u + 6], v[8 * u + 7]));
}

// Stores the warp's 32 accumulator rows x 32 columns (thread = row): accumulator
// row `row`, column `col` onward.  D is the accumulator or (kTransposed) its transpose.
template <bool kTransposed>
__device__ __forceinline__ void fp8_store_chunk(const uint32_t (&v)[32], uint32_t staging, int lane, bool fp32,
                                                const CUtensorMap *tmD, int32_t row, int32_t col, const Fp8GemmParams &p)
{
    fp8_staging_free(lane);
    if constexpr (kTransposed) {
        // columns of the accumulator are rows of D: `live` of them exist.  An fp32
        // piece is half as wide: lanes 0-15 fill one, 16-31 the other.
        const int32_t live = p.cols - col;
        const uint32_t mine = staging + (fp32 && lane >= 16 ? kFp8PieceBytes : 0u);
        const uint32_t at_lane = fp32 ? (uint32_t)lane & 15u : (uint32_t)lane;
#pragma unroll
        for (uint32_t i = 0; i < 32; ++i) {
            if ((int32_t)i >= live)
                break;
            const uint32_t at = mine + fp8_piece_offset(i, at_lane, fp32);
            if (fp32)
                st_shared_u32(at, v[i]);
            else
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)pack_bf16x2(v[i], 0u)) : "memory");
        }
        fp8_store_pieces(staging, lane, tmD, fp32 ? 2 : 1, row, col, row + 16, col, fp32, p);
    } else if (fp32) {
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u)
            st_shared_v4(staging + (u >= 4 ? kFp8PieceBytes : 0u) + fp8_piece_offset((uint32_t)lane, 4 * (u & 3), true),
                         v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
        fp8_store_pieces(staging, lane, tmD, 2, col, row, col + 16, row, true, p);
    } else {
        fp8_stage_bf16(v, staging, lane);
        fp8_store_pieces(staging, lane, tmD, 1, col, row, col, row, false, p);
    }
}

// Stores accumulator row `row`, columns col .. col+3, to D or (kTransposed) its transpose.
template <bool kTransposed>
__device__ __forceinline__ void fp8_store_four(const uint32_t (&v)[4], int32_t row, int32_t col, bool fp32,
                                               const Fp8GemmParams &p)
{
    if (row >= p.rows)
        return;
    const int64_t at = kTransposed ? (int64_t)col * p.ldd + row : (int64_t)row * p.ldd + col;
    const int64_t step = kTransposed ? p.ldd : 1;
    if (fp32) {
        float *const d = static_cast<float *>(p.D) + at;
        if (!kTransposed && col + 4 <= p.cols && (reinterpret_cast<uintptr_t>(d) & 15u) == 0) {
            *reinterpret_cast<uint4 *>(d) = make_uint4(v[0], v[1], v[2], v[3]);
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < p.cols)
                d[e * step] = __uint_as_float(v[e]);
        return;
    }
    uint16_t *const d = static_cast<uint16_t *>(p.D) + at;
    const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (!kTransposed && col + 4 <= p.cols && (reinterpret_cast<uintptr_t>(d) & 7u) == 0) {
        *reinterpret_cast<uint2 *>(d) = make_uint2(lo, hi);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < p.cols)
            d[e * step] = (uint16_t)((e < 2 ? lo : hi) >> (16 * (e & 1)));
}

// This rank's share of the float4s of its cluster's tile, each summed over the
// ranks' shared memories in their order and stored.
template <bool kTransposed>
__device__ __forceinline__ void fp8_add_spread(const Fp8GemmParams &p, uint32_t sums, int32_t row0, int32_t col0,
                                            int nchunks, int ew, int lane)
{
    const bool fp32 = p.out_fp32 != 0;
    const int live = kTransposed && nchunks == 1 ? min(8, (p.cols - col0 + 3) >> 2) : 8;  // float4s of a chunk's row
    const int units = nchunks * 4 * live;
    for (int u = (int)cluster_ctarank() + p.cluster * ew; u < units; u += p.cluster * kFp8EpiWarps) {
        const int j = u % live, c = (u / live) >> 2, quad = (u / live) & 3;
        const uint32_t from = sums + (uint32_t)((((((c & 1) * 4 + quad) * 4 + (c >> 1)) * 8 + j) * 32 + lane) * 16);
        uint32_t x[8][4];
#pragma unroll
        for (int rk = 0; rk < 8; ++rk)
            if (rk < p.cluster)
                ld_shared_cluster_v4(mapa_shared(from, (uint32_t)rk), x[rk][0], x[rk][1], x[rk][2], x[rk][3]);
#pragma unroll
        for (int rk = 1; rk < 8; ++rk)
            if (rk < p.cluster) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[0][e] = __float_as_uint(__uint_as_float(x[0][e]) + __uint_as_float(x[rk][e]));
            }
        fp8_store_four<kTransposed>(x[0], row0 + quad * 32 + lane, col0 + c * 32 + 4 * j, fp32, p);
    }
}

// This thread's 32 values of chunk number `ci` of its warp in a CTA's partial:
// float4 groups, each 512 contiguous bytes over the warp.
__device__ __forceinline__ float4 *fp8_partial(float *partials, int32_t cta, int ew, int ci, int lane)
{
    return reinterpret_cast<float4 *>(partials + (size_t)cta * kFp8PartialFloats) + ((ew * 4 + ci) * 8) * 32 + lane;
}

__device__ __forceinline__ void fp8_store_partial(const uint32_t (&v)[32], float4 *part)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        __stcg(part + j * 32, make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                          __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])));
}

template <int kBatch>
__device__ __forceinline__ void fp8_add_partial(uint32_t (&v)[32], const float4 *part)
{
#pragma unroll
    for (int j0 = 0; j0 < 8; j0 += kBatch) {
        float4 f[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            f[j] = __ldcg(part + (j0 + j) * 32);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            uint32_t *const x = &v[4 * (j0 + j)];
            x[0] = __float_as_uint(__uint_as_float(x[0]) + f[j].x);
            x[1] = __float_as_uint(__uint_as_float(x[1]) + f[j].y);
            x[2] = __float_as_uint(__uint_as_float(x[2]) + f[j].z);
            x[3] = __float_as_uint(__uint_as_float(x[3]) + f[j].w);
        }
    }
}

template <int CG, bool kTransposed, bool kLong>
__global__ void __launch_bounds__(kFp8Threads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmR, const __grid_constant__ CUtensorMap tmC,
                    const __grid_constant__ CUtensorMap tmD, const Fp8GemmParams p)
{
    constexpr bool kCluster = CG == 2;
    constexpr uint32_t kRBytes = (uint32_t)kFp8RowsPerCta * kFp8BlockK;
    const int32_t width = p.width;
    const uint32_t stage_bytes = kRBytes + (uint32_t)(width / CG) * kFp8BlockK;  // a multiple of 1024

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int S = p.stages;  // even: stages are released in pairs
    const uint32_t stage0 = base;
    const uint32_t staging0 = base + (uint32_t)S * stage_bytes;
    const uint32_t scales0 = staging0 + kFp8EpiWarps * kFp8StagingBytes;
    const uint32_t full_bar = scales0 + (uint32_t)S * kFp8ScaleBytes;
    const uint32_t empty_bar = full_bar + 8u * S;
    const uint32_t accf_bar = empty_bar + 8u * S;
    const uint32_t acce_bar = accf_bar + 16u;
    const uint32_t done_bar = acce_bar + 16u;
    const uint32_t tmem_slot = done_bar + 8u;
    const uint32_t abort_flag = tmem_slot + 4u;
    const uint32_t go_words = abort_flag + 4u;  // 2 words, alternating by item
    const uint32_t ready_bar = go_words + 8u;   // cluster form: one per epilogue warp of rank 0, or one per rank;
                                                // behind its eight, one that nothing waits for

    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);  // uniform, and known to be
    const int lane = threadIdx.x & 31;
    const uint32_t rank = kCluster ? cluster_ctarank() : 0u;  // in an SM pair
    // the cluster form: rank 0 adds up the pieces, or each rank a part of the tile (not
    // where the registers hold an fp32 D's sums already: they spill)
    const bool shared_tile = !kCluster && p.cluster > 1;
    const bool spread = !kCluster && !kLong && p.cluster >= kFp8SpreadFrom;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar + 8u * s, 1 + 2 * CG);  // the producer's expect_tx, each CTA's two scale warps
            mbar_init(empty_bar + 8u * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(accf_bar + 8u * a, 1);
            mbar_init(acce_bar + 8u * a, kFp8EpiWarps * CG);
        }
        mbar_init(done_bar, 1);
        mbar_init(ready_bar + 64u, 1);
        if (spread)
            mbar_init(ready_bar, (uint32_t)p.cluster * kFp8EpiWarps);  // every epilogue warp of every rank
        else if (shared_tile)
            for (int e = 0; e < kFp8EpiWarps; ++e)
                mbar_init(ready_bar + 8u * e, (uint32_t)p.cluster - 1u);  // that warp of every other rank
        st_shared_u32(abort_flag, 0u);
        fence_mbarrier_init();
    }
    if (threadIdx.x == 32) {
        prefetch_tensormap(&tmR);
        prefetch_tensormap(&tmC);
        if (p.d_tma)
            prefetch_tensormap(&tmD);
    }
    // all CTAs of a cluster have initialised their barriers before any cross-CTA
    // arrive, TMA completion or the paired allocation
    if (kCluster || shared_tile) {
        __syncwarp();
        cluster_arrive_wait();
    } else {
        __syncthreads();
    }
    if (warp == 2) {
        tmem_alloc<CG>(tmem_slot, 512);
        tmem_relinquish<CG>();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = ld_shared_u32(tmem_slot);
    // Up to here only shared and tensor memory was touched: it overlaps the
    // previous kernel on the stream.  Every role that reads or writes global
    // memory waits for that kernel first.

    WaitCtl ctl;
    ctl.abort_flag = abort_flag;
    ctl.peer_abort_flag = kCluster ? mapa_shared(abort_flag, rank ^ 1u) : 0u;
    ctl.err = p.err;
    ctl.set_limit(p.watchdog_ns);

    const int32_t cluster_id = (int32_t)blockIdx.x / CG;
    const int32_t num_clusters = (int32_t)gridDim.x / CG;
    const int32_t KB = p.num_k_blocks;
    Fp8Work wi;
    wi.init(p, cluster_id, num_clusters);
    Fp8Item w;

    if (warp < 4) {
        if (warp == 0) {
            // ---------------- TMA producer ----------------
            const uint32_t full_target = kCluster ? mapa_shared(full_bar, 0u) : full_bar;
            const uint32_t leader = elect_one();
            int s = 0;
            uint32_t ph = 0;
            int32_t it = 0;
            bool ok = true;
            grid_dependency_wait();
            while (ok && wi.next(w)) {
                const TileCoord tc = fp8_tile_coord(w.tile, p);
                const int32_t yr = (tc.mb * CG + (int32_t)rank) * kFp8RowsPerCta;
                const int32_t yc = tc.nb * width + (int32_t)rank * (width / CG);
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    if (ring_group_first(s, 1u)) {
                        const uint32_t bar = empty_bar + 8u * ring_group(s, 1u), parity = ring_empty_parity(ph);
                        if (!__all_sync(0xFFFFFFFFu, mbar_wait_tries(bar, parity, ctl.suspend_ns, 1u)) &&
                            !warp_wait<false>(ctl, bar, parity, kRoleProducer, (uint32_t)s, lane)) {
                            ok = false;
                            break;
                        }
                    }
                    if (it != p.fault_skip_it) {
                        if (rank == 0)
                            expect_tx_elected(full_bar + 8u * s, stage_bytes * CG, leader);
                        const uint32_t fb = full_target + 8u * s;
                        const uint32_t sa = stage0 + (uint32_t)s * stage_bytes;
                        tma_load_2d_elected<CG>(sa, &tmR, kb * kFp8BlockK, yr, fb, leader);
                        tma_load_2d_elected<CG>(sa + kRBytes, &tmC, kb * kFp8BlockK, yc, fb, leader);
                    }
                    ++it;
                    ring_advance(s, ph, S);
                }
            }
            grid_launch_dependents();
            // Teardown: the last S loads may still be in flight if a role gave up.
            if (lane == 0 && rank == 0) {
                ctl.limit_ns = max(ctl.limit_ns, kFp8DrainNs);
                const int32_t n = it < S ? it : S;
                for (int32_t d = 1; d <= n; ++d) {
                    const int32_t j = it - d;
                    if (j == p.fault_skip_it)
                        continue;
                    // one that runs out has outlasted the others' loads too
                    if (!ctl.wait_drain<kCluster>(full_bar + 8u * (uint32_t)ring_stage_of(j, S),
                                                    ring_parity_of(j, S), (uint32_t)ring_stage_of(j, S)))
                        break;
                }
            } else if (lane == 0 && ctl.aborted()) {
                // the peer's loads complete on the leader's barriers, which this CTA
                // cannot poll: a fixed grace period instead
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 50000ull) {
                }
            }
            __syncwarp();
        } else if (warp == 1 && rank == 0) {
            // ---------------- MMA issuer ----------------
            const uint64_t rdesc0 = smem_desc_sw128(stage0);
            const uint64_t cdesc0 = smem_desc_sw128(stage0 + kRBytes);
            const uint64_t sdesc0 = smem_desc_scales(scales0);
            const uint32_t idesc0 = idesc_mxf8(kFp8RowsPerCta * CG, 0) | ((uint32_t)(width >> 3) << 17);
            const uint32_t step = stage_bytes >> 4;
            const uint32_t leader = elect_one();
            // Waits here are loops inside one statement, and a wait that runs out does
            // not leave the k loop (a branch out of it takes 1 x 8192 x 8192 from 16.8 to 17.3
            // us; a leader that is not constant takes 8192^3 from 304 to 345): it records the
            // fact, and the rest of the item runs with short single probes and tells
            // nobody.  Above all it releases no stage: one filled again before its first
            // load has landed would count arrivals into a phase that has all of them,
            // which faults.
            const uint32_t nobody_bar = ready_bar + 64u;
            uint32_t probe_ns = ctl.suspend_ns;
            uint32_t tries = (uint32_t)(ctl.limit_ns / probe_ns) + 1u;
            uint32_t bad = 0u;
            auto wait = [&](uint32_t bar, uint32_t parity, uint32_t role, uint32_t where) {
                if (mbar_wait_tries(bar, parity, probe_ns, tries) == 0u) {
                    if (bad == 0u && leader)
                        ctl.fail(role, where);
                    bad = 1u;
                    tries = 1u;
                    probe_ns = 1u;
                }
            };
            int s = 0;
            uint32_t ph = 0;
            int acc = 0;
            uint32_t acc_ph = 0;
            uint32_t ready = 0u;  // the next stage was seen full
            uint32_t group = 0;  // groups of 4 k-blocks so far: their parity picks the scales' buffer
            while (wi.next(w)) {
                wait(acce_bar + 8u * acc, acc_ph ^ 1u, kRoleMmaAcc, (uint32_t)acc);
                tc_fence_after_sync();
                uint32_t d_tmem = tmem_base + (uint32_t)(acc * kFp8MaxWidth);
                uint32_t stm = 0;
                int32_t cut = kLong ? fp8_segment_end(w.kb0) : INT32_MAX;  // the accumulator's sums move on there
                uint32_t fresh = 1u;                      // the accumulator starts over
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    if (kLong && kb == cut) {
                        mma_commit_elected<CG>(bad ? nobody_bar : accf_bar + 8u * acc, leader);
                        acc ^= 1;
                        acc_ph ^= acc == 0 ? 1u : 0u;
                        wait(acce_bar + 8u * acc, acc_ph ^ 1u, kRoleMmaAcc, (uint32_t)acc);
                        tc_fence_after_sync();
                        d_tmem = tmem_base + (uint32_t)(acc * kFp8MaxWidth);
                        cut = fp8_segment_end(kb);
                        fresh = 1u;
                    }
                    if (!__all_sync(0xFFFFFFFFu, ready))
                        wait(full_bar + 8u * s, ring_full_parity(ph), kRoleMmaFull, (uint32_t)s);
                    tc_fence_after_sync();
                    if (kb == w.kb0 || (kb & 3) == 0) {
                        // copies and MMAs of one thread execute in order: the copy
                        // into a buffer follows the MMAs that last read it
                        stm = tmem_base + kFp8ScaleCol + 32u * (group & 1u);
                        ++group;
                        const uint64_t sd = sdesc0 + (uint64_t)((uint32_t)s * (kFp8ScaleBytes >> 4));
                        copy_scales<CG>(stm, sd, leader);
                        copy_scales<CG>(stm + kFp8ScaleColB, sd + (512u >> 4), leader);
                        if (width > 128)
                            copy_scales<CG>(stm + kFp8ScaleColB + 4u, sd + (1024u >> 4), leader);
                    }
                    const uint64_t off = (uint64_t)((uint32_t)s * step);
                    const uint32_t idesc = idesc0 | scale_id((uint32_t)kb & 3u);
                    int s1 = s;
                    uint32_t ph1 = ph;
                    ring_advance(s1, ph1, S);
                    ready = mma_mxf8_block<CG>(d_tmem, rdesc0 + off, cdesc0 + off, idesc, stm, stm + kFp8ScaleColB,
                                               fresh ^ 1u, leader, full_bar + 8u * s1, ring_full_parity(ph1));
                    fresh = 0u;
                    if (ring_group_last(s, 1u))
                        mma_commit_elected<CG>(bad ? nobody_bar : empty_bar + 8u * ring_group(s, 1u), leader);
                    ring_advance(s, ph, S);
                }
                mma_commit_elected<CG>(bad ? nobody_bar : accf_bar + 8u * acc, leader);
                acc ^= 1;
                if (acc == 0)
                    acc_ph ^= 1u;
                if (__any_sync(0xFFFFFFFFu, bad))
                    break;
            }
            // no MMA may still be writing tensor memory when it is freed
            mma_commit_elected<CG>(done_bar, leader);
            if (leader) {
                ctl.limit_ns = max(ctl.limit_ns, kFp8DrainNs);
                ctl.wait_drain<kCluster>(done_bar, 0u, 0xFFFu);
            }
            __syncwarp();
        } else if (warp == 2 || warp == 3) {
            // ---------------- scales ----------------
            // The stage of a group's first k-block carries the group's words: 32 rows of
            // four, the words of rows r, r + 32, r + 64 and r + 96 of the row side at
            // 16 r, those of the column side's rows behind them in two such blocks.
            // Rows past the end count as scale 1; they meet only zeros, in parts of the
            // tile that are not stored.  The two warps bring groups in turn (one alone
            // is busy 400 of the 450 clocks that a wide tile's k-block lasts), each with
            // its next group's words in flight while it hands over the last ones.  Both
            // wait for every release and arrive on every stage's full barrier: so the
            // MMA issuer waits for scales and operands at once, and neither warp can
            // run two phases of a barrier ahead or behind, which its parity would not
            // tell.
            const uint32_t full_target = kCluster ? mapa_shared(full_bar, 0u) : full_bar;
            const uint32_t which = (uint32_t)warp & 1u;
            Fp8Work wl = wi;  // the loads' place in the work
            Fp8Item il = {0, 0, 0};
            int32_t left = 0;       // groups of the loads' item still to come
            uint32_t gl = 0;        // groups the loads have passed
            uint32_t live = 0u;     // which of the twelve words exist
            const uint32_t *sr = nullptr, *sc = nullptr;
            uint32_t v[2][12];
            auto load = [&](uint32_t(&x)[12]) {
                for (;;) {
                    if (left == 0) {
                        if (!wl.next(il))
                            return;
                        const TileCoord tc = fp8_tile_coord(il.tile, p);
                        const int32_t yr = (tc.mb * CG + (int32_t)rank) * kFp8RowsPerCta + lane;
                        const int32_t yc = tc.nb * width + lane;
                        const int32_t kt = il.kb0 >> 2;
                        left = ((il.kb1 - 1) >> 2) + 1 - kt;
                        sr = p.s_rows + (int64_t)kt * p.rows + yr;
                        sc = p.s_cols + (int64_t)kt * p.cols + yc;
                        live = 0u;
#pragma unroll
                        for (int j = 0; j < 12; ++j)
                            if (j < 4 ? yr + 32 * j < p.rows : 32 * (j - 4) < width && yc + 32 * (j - 4) < p.cols)
                                live |= 1u << j;
                    }
                    const bool mine = (gl & 1u) == which;
                    if (mine) {
#pragma unroll
                        for (int j = 0; j < 12; ++j)
                            x[j] = live & (1u << j) ? (j < 4 ? sr[32 * j] : sc[32 * (j - 4)]) : 0x7F7F7F7Fu;
                    }
                    sr += p.rows;
                    sc += p.cols;
                    --left;
                    ++gl;
                    if (mine)
                        return;
                }
            };
            grid_dependency_wait();
            load(v[0]);
            load(v[1]);
            int s = 0;
            uint32_t ph = 0;
            uint32_t g = 0;
            bool ok = true;
            while (ok && wi.next(w)) {
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    if (ring_group_first(s, 1u)) {
                        const uint32_t bar = empty_bar + 8u * ring_group(s, 1u), parity = ring_empty_parity(ph);
                        if (!__all_sync(0xFFFFFFFFu, mbar_wait_tries(bar, parity, ctl.suspend_ns, 1u)) &&
                            !warp_wait<false>(ctl, bar, parity, kRoleScales, (uint32_t)s, lane)) {
                            ok = false;
                            break;
                        }
                    }
                    const bool first = kb == w.kb0 || (kb & 3) == 0;
                    const bool last = kb == w.kb1 - 1 || (kb & 3) == 3;
                    const bool mine = (g & 1u) == which;
                    if (mine && first) {
                        const uint32_t at = scales0 + (uint32_t)s * kFp8ScaleBytes + 16u * (uint32_t)lane;
                        st_shared_v4(at, v[0][0], v[0][1], v[0][2], v[0][3]);
                        st_shared_v4(at + 512u, v[0][4], v[0][5], v[0][6], v[0][7]);
                        if (width > 128)
                            st_shared_v4(at + 1024u, v[0][8], v[0][9], v[0][10], v[0][11]);
                        fence_proxy_async_shared();
                        __syncwarp();
                    }
                    // Each CTA's words stay in its own shared memory, where its own half
                    // of the paired copy reads them: the proxy fence has put them there
                    // before the arrive leaves.  So the arrive on the leader's barrier
                    // releases at CTA scope; at cluster scope it waits for all of this
                    // thread's memory traffic, loads too (measured 600 ns).
                    if (lane == 0) {
                        if constexpr (kCluster)
                            mbar_arrive_cluster_handoff(full_target + 8u * s);
                        else
                            mbar_arrive(full_target + 8u * s);
                    }
                    if (mine && last) {
#pragma unroll
                        for (int j = 0; j < 12; ++j)
                            v[0][j] = v[1][j];
                        load(v[1]);
                    }
                    g += last ? 1u : 0u;
                    ring_advance(s, ph, S);
                }
            }
        }
    } else {
        // ---------------- epilogue ----------------
        grid_dependency_wait();
        const int ew = warp - 4;
        const int q = warp & 3;         // tensor-memory lane quadrant
        const int half = ew >> 2;       // takes chunks half, half + 2, ... of 32 columns
        const int nchunks = (width + 31) / 32;
        const uint32_t staging = staging0 + (uint32_t)ew * kFp8StagingBytes;
        const uint32_t acce_target = kCluster ? mapa_shared(acce_bar, 0u) : acce_bar;
        const bool fp32 = kLong || p.out_fp32 != 0;
        const int32_t cta = cluster_id * CG + (int32_t)rank;
        int acc = 0;
        uint32_t acc_ph = 0;
        uint32_t item_parity = 0;
        bool ok = true;
        const bool dense = p.sk_units >= num_clusters;  // every range holds a unit
        // one thread waits for the accumulator and posts the outcome, so that all
        // warps take the same branch; the word alternates with the accumulations
        auto accumulated = [&]() {
            const uint32_t go = go_words + 4u * item_parity;
            item_parity ^= 1u;
            if (threadIdx.x == 128)
                st_volatile_shared_u32(
                    go, ctl.wait<kCluster>(accf_bar + 8u * acc, acc_ph, kRoleEpilogue, (uint32_t)acc) ? 1u : 0u);
            named_barrier_sync(1u, kFp8EpiWarps * 32u);
            return ld_volatile_shared_u32(go) != 0u;
        };
        // this warp has read its part of the accumulator: hand it back
        auto hand_back = [&]() {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kCluster)
                    mbar_arrive_cluster_handoff(acce_target + 8u * acc);
                else
                    mbar_arrive(acce_bar + 8u * acc);
            }
        };
        auto load_chunk = [&](int c, uint32_t(&v)[32]) {
            tmem_load_32x32(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kFp8MaxWidth + c * 32), v);
            tmem_load_wait();
            reg_fence(v);
        };
        while (wi.next(w)) {
            const TileCoord tc = fp8_tile_coord(w.tile, p);
            const int32_t yr = (tc.mb * CG + (int32_t)rank) * kFp8RowsPerCta + q * 32;
            const int32_t yc = tc.nb * width;
            const bool contributor = w.kb0 > 0;
            const bool owner = w.kb0 == 0 && w.kb1 < KB;
            // the clusters whose ranges start inside this tile, owner only; a range
            // may be empty (fewer units than clusters), and then leaves nothing
            int32_t last = cluster_id;
            bool parts = owner;
            auto collect = [&]() {
                if (owner && spread) {
                    parts = false;  // they meet below
                } else if (owner && shared_tile) {
                    uint32_t got = 1u;
                    if (lane == 0)
                        got = ctl.wait<true>(ready_bar + 8u * (uint32_t)ew, 0u, kRoleFixup, (uint32_t)ew) ? 1u : 0u;
                    __syncwarp();  // lane 0's acquire comes before the lanes' loads
                    parts = __shfl_sync(0xFFFFFFFFu, got, 0) != 0u;
                } else if (owner) {
                    last = fp8_range_of(p.sk_units, num_clusters, (int64_t)(w.tile + 1) * KB - 1);
                    for (int32_t j2 = cluster_id + 1; parts && j2 <= last; ++j2)
                        if (dense || fp8_range_holds(p.sk_units, num_clusters, j2))
                            // a give-up stores the tile unsummed, and the status says so
                            parts = warp_wait_flag(ctl, p.flags + (j2 * CG + (int32_t)rank) * kFp8EpiWarps + ew, 1u,
                                                   lane);
                    __syncwarp();  // lane 0's acquires come before the lanes' loads
                }
            };
            // one chunk's sums: left for the tile's owner, or completed and stored
            auto finish = [&](int c, uint32_t(&v)[32]) {
                // The cluster form keeps a partial in the CTA's own ring: a
                // contributor's only item has consumed all of its loads by now.
                const uint32_t local = stage0 + (uint32_t)(((ew * 4 + (c >> 1)) * 8) * 32 + lane) * 16u;
                // (of a transposed D, only its rows' columns, four at a time)
                const int live = kTransposed ? min(8, (p.cols - (yc + c * 32) + 3) >> 2) : 8;
                if (spread || (contributor && shared_tile)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < live)
                            st_shared_v4(local + 512u * j, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    return;
                }
                if (contributor) {
                    fp8_store_partial(v, fp8_partial(p.partials, cta, ew, c >> 1, lane));
                    return;
                }
                if (parts && shared_tile) {
                    // Several loads before their adds, so that the round trips
                    // overlap: of one piece after another, or, where few columns
                    // come from many pieces, of several at a time.
                    constexpr int kBatch = kLong ? 4 : 8;
                    if (!kLong && live <= 2) {
                        for (int32_t rk = 1; rk < p.cluster; rk += 4) {
                            uint32_t x[4][8];
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                const uint32_t remote = mapa_shared(local, (uint32_t)min(rk + b, p.cluster - 1));
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    ld_shared_cluster_v4(remote + 512u * j, x[b][4 * j], x[b][4 * j + 1],
                                                         x[b][4 * j + 2], x[b][4 * j + 3]);
                            }
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                if (rk + b < p.cluster) {
#pragma unroll
                                    for (int j = 0; j < 8; ++j)
                                        v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(x[b][j]));
                                }
                        }
                    } else {
                        for (int32_t rk = 1; rk < p.cluster; ++rk) {
                            const uint32_t remote = mapa_shared(local, (uint32_t)rk);
#pragma unroll
                            for (int j0 = 0; j0 < 8; j0 += kBatch) {
                                uint32_t x[4 * kBatch];
#pragma unroll
                                for (int j = 0; j < kBatch; ++j)
                                    ld_shared_cluster_v4(remote + 512u * (j0 + j), x[4 * j], x[4 * j + 1],
                                                         x[4 * j + 2], x[4 * j + 3]);
#pragma unroll
                                for (int j = 0; j < 4 * kBatch; ++j)
                                    v[4 * j0 + j] =
                                        __float_as_uint(__uint_as_float(v[4 * j0 + j]) + __uint_as_float(x[j]));
                            }
                        }
                    }
                } else if (parts) {
                    for (int32_t j2 = cluster_id + 1; j2 <= last; ++j2) {
                        if (!dense && !fp8_range_holds(p.sk_units, num_clusters, j2))
                            continue;
                        fp8_add_partial<kLong ? 4 : 8>(
                            v, fp8_partial(p.partials, j2 * CG + (int32_t)rank, ew, c >> 1, lane));
                    }
                }
                const int32_t cols = yc + c * 32;
                if (yr >= p.rows || cols >= p.cols)
                    return;
                fp8_store_chunk<kTransposed>(v, staging, lane, fp32, &tmD, yr, cols, p);
            };

            if constexpr (kLong) {
                // The tensor core's additions lose up to a unit of the accumulator
                // each, toward zero: 3e-6 of a sum over K = 32768.  bf16 hides that;
                // for an fp32 D the accumulator takes a segment of k-blocks (2e-7
                // with kFp8Segment of them) and the sums are added up here, in
                // registers: so a tile is at most kFp8MaxLongWidth columns wide.
                constexpr int kOwn = kFp8MaxLongWidth / 64;  // chunks of a warp
                uint32_t run[kOwn][32];
#pragma unroll
                for (int i = 0; i < kOwn; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        run[i][j] = 0u;
                for (int32_t cut = w.kb0; ok && cut < w.kb1;) {
                    cut = fp8_segment_end(cut);
                    if (!(ok = accumulated()))
                        break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int i = 0; i < kOwn; ++i)
                        if (half + 2 * i < nchunks)
                            tmem_add_32x32(tmem_base + ((uint32_t)(q * 32) << 16) +
                                               (uint32_t)(acc * kFp8MaxWidth + (half + 2 * i) * 32),
                                           run[i]);
                    hand_back();
                    acc ^= 1;
                    acc_ph ^= acc == 0 ? 1u : 0u;
                }
                if (!ok)
                    break;
                collect();
#pragma unroll
                for (int i = 0; i < kOwn; ++i)
                    if (half + 2 * i < nchunks)
                        finish(half + 2 * i, run[i]);
            } else {
                if (!accumulated())
                    break;
                tc_fence_after_sync();
                if (half >= nchunks) {  // a tile of one chunk: the second group reads nothing
                    hand_back();
                    collect();
                }
                int c = half;
                if (!kTransposed && !fp32 && !contributor && !owner) {
                    // whole tiles of bf16, most of the work: two chunks at a time
                    for (; c + 2 < nchunks; c += 4) {
                        uint32_t v0[32], v1[32];
                        load_chunk(c, v0);
                        load_chunk(c + 2, v1);
                        if (c + 4 >= nchunks)
                            hand_back();
                        if (yr >= p.rows || yc + c * 32 >= p.cols)
                            continue;
                        fp8_staging_free(lane);
                        fp8_stage_bf16(v0, staging, lane);
                        fp8_stage_bf16(v1, staging + kFp8PieceBytes, lane);
                        fp8_store_pieces(staging, lane, &tmD, 2, yc + c * 32, yr, yc + c * 32 + 64, yr, false, p);
                    }
                }
                for (; c < nchunks; c += 2) {
                    uint32_t v[32];
                    load_chunk(c, v);
                    if (c + 2 >= nchunks)
                        hand_back();
                    if (c == half && owner)
                        collect();  // after this piece's own sums have been read
                    finish(c, v);
                }
                acc ^= 1;
                acc_ph ^= acc == 0 ? 1u : 0u;
            }
            if (spread) {
                // Every rank's sums lie in its own shared memory: once all have
                // arrived, each adds up its share of the tile's float4s, from all
                // ranks at once and in their order.  (Rank 0 alone takes a round
                // trip a piece: 50x146x12439 9.8 us that way, 8.5 this; 241x448x16859
                // 13 and 12, 10.8 with the clusters chosen for it.  With four ranks
                // 939x480x5185 loses 0.3 us by it.)
                __syncwarp();  // the warp's stores come before its lanes' releases
                if (lane < p.cluster)
                    mbar_arrive_cluster(mapa_shared(ready_bar, (uint32_t)lane));
                uint32_t got = 1u;
                if (lane == 0)
                    got = ctl.wait<true>(ready_bar, 0u, kRoleFixup, (uint32_t)ew) ? 1u : 0u;
                __syncwarp();  // lane 0's acquire comes before the lanes' loads
                if (__shfl_sync(0xFFFFFFFFu, got, 0) == 0u)
                    break;
                fp8_add_spread<kTransposed>(p, stage0, tc.mb * kFp8RowsPerCta, yc, nchunks, ew, lane);
            } else if (contributor) {
                __syncwarp();  // the warp's stores come before lane 0's release
                if (lane == 0 && shared_tile)
                    mbar_arrive_cluster(mapa_shared(ready_bar + 8u * (uint32_t)ew, 0u));
                else if (lane == 0)
                    st_release_gpu_u32(p.flags + cta * kFp8EpiWarps + ew, 1u);
            }
        }
        // the staging buffers have been read before the CTA exits
        if (lane == 0)
            bulk_wait_read_all();
        __syncwarp();
    }

    // ---------------- teardown ----------------
    tc_fence_before_sync();
    __syncthreads();
    if (kCluster || shared_tile)
        cluster_arrive_wait();  // the peer is done with this CTA's memory
    if (warp == 2) {
        tc_fence_after_sync();
        tmem_dealloc<CG>(tmem_base, 512);
    }
}

}  // namespace wstma
