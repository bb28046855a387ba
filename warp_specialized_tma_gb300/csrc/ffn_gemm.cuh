// The bf16 products of a feed-forward block, with what follows them in the epilogue.
//
//   plain   S = sum over k of A B (or of two products, added up); D0 = act(S + bias) + residual, D1 = S + bias
//   gated   S = x Wg^T and S2 = x Wu^T over the same x; D0 = act(S) S2, and S and S2 kept in bf16 or 8 bits
//   grad    S = dh = dy Wd, with g and u: D0 = dh u act'(g), D1 = dh act(g), D2 = act(g) u
//
// Either operand may be contiguous along k or along its rows, so a forward product, an input's
// gradient (the weight is contiguous along the columns of the result) and a weight's gradient
// (both operands are contiguous along their rows) are the same kernel: tcgen05.mma reads
// both forms from shared memory, by the descriptors' strides and a bit of the instruction
// descriptor, and nothing is transposed in memory.
//
// One operand is on the MMA's row side (128 rows to a CTA, 256 to an SM pair), the other on
// its column side (`width` columns to a tile).  For few tokens the weights take the row side,
// and the accumulator holds the result transposed.  A gated tile keeps two accumulators: next
// to each other as one MMA of 256 columns, 128 of each weight, or, transposed, one per weight
// and 128 rows of it, so that either way one thread holds both sums of an element.
//
// Roles (384 threads, one CTA per SM):
//   warps 0, 2, 3    TMA producers, in turn: per two k-blocks wait "empty", load the tiles;
//                    warp 2 also allocates and frees tensor memory
//   warp 1           MMA issuer (leader CTA only in pairs), one elected lane
//   warps 4..11      epilogue: tensor memory -> registers -> results
//
// Work: tiles [0, sk_tiles) are split along k, their (tile, k-block) units cut into one
// contiguous range per cluster; the other tiles are walked whole.  The pieces of a split tile
// meet as fp32 through global memory, or, where the CTAs of a thread-block cluster share a
// tile, through distributed shared memory; they are added in range order by the piece that
// holds k-block 0, so the result is the same every time.  Every wait is bounded by the
// watchdog (WaitCtl in ptx.cuh).
//
// Measured (us in a burst, from a graph; the operations' or, for few tokens, the bytes' time):
//   linear 8192^3, silu, bias, residual                565 (572): tensor pipe 91 % active, at the power cap's clock
//   gated 4096 x 4096 x 16384, g and u kept in bf16    561 (572): the same
//   linear 64 x 8192 x 8192, bias, residual            28.5 (20.3): HBM; a launch's start, first loads and last epilogue
//   dx and dW of 4096^3 in one launch                  144 (143, under the profiler): tensor pipe 83 %, 3.4 waves
//   dg, du, h of 8192 x 2048 x 8192 from 8 bits        204 (143): the epilogue, 11.7 us a tile beside 8.6 of MMAs
//   dW of 8192 x 8192 from 64 tokens                   25.4 (20.2): the epilogue's chain; stores at 5.3 TB/s
// 256 x 256 tiles of an SM pair have the most MMAs a byte loaded, and are what long sums get.
#pragma once

#include <stdint.h>

#include "ffn_kernels.h"
#include "ffn_math.cuh"
#include "fp8_ptx.cuh"
#include "gemm_common.cuh"

namespace wstma {

// Copies and MMAs in flight are waited for at a CTA's end however short the watchdog's limit is.
constexpr uint64_t kFfnDrainNs = 20000000;

struct FfnItem {
    int32_t tile, kb0, kb1;
    int32_t product;  // of the launch
};

__host__ __device__ __forceinline__ int64_t ffn_range_begin(int64_t units, int32_t clusters, int32_t c)
{
    return (int64_t)c * units / clusters;
}

__host__ __device__ __forceinline__ bool ffn_range_holds(int64_t units, int32_t clusters, int32_t c)
{
    return ffn_range_begin(units, clusters, c) < ffn_range_begin(units, clusters, c + 1);
}

// The range that holds unit u.
__host__ __device__ __forceinline__ int32_t ffn_range_of(int64_t units, int32_t clusters, int64_t u)
{
    return (int32_t)(((u + 1) * clusters + units - 1) / units) - 1;
}

// End of the segment that k-block kb belongs to (kLong).
__host__ __device__ __forceinline__ int32_t ffn_segment_end(int32_t kb, int32_t segment)
{
    return kb / segment * segment + segment;
}

// Which range is cluster c's, and whose range c is: the last cluster has the first one.  A tile's owner
// waits for the ranges behind its own, so for clusters with lower indices, which the GPU places
// before it: whatever else runs there, another stream's split tiles say, no cluster that is waited for still
// needs a place.  (The CTAs of a cluster that share a tile have their places together.)
__host__ __device__ __forceinline__ int32_t ffn_range_at(const FfnParams &p, int32_t clusters, int32_t c)
{
    return p.cluster > 1 ? c : clusters - 1 - c;
}

// A cluster's items in order: its range of the split tiles' units (a piece of each tile that it
// touches), then every clusters-th whole tile.  Only a range's first piece may start inside a tile (it
// then leaves a partial); a piece that starts at k-block 0 and does not reach the tile's end is the
// last of its range.  So no cluster waits for a partial before it has left its own.
struct FfnWork {
    int64_t u, u_end;
    int32_t dp, C, T, KB;

    __host__ __device__ __forceinline__ void init(const FfnParams &p, int32_t cluster, int32_t clusters)
    {
        KB = p.num_k_blocks;
        C = clusters;
        T = p.num_tiles;
        dp = p.sk_tiles + cluster;
        const int32_t range = ffn_range_at(p, clusters, cluster);
        u = ffn_range_begin(p.sk_units, clusters, range);
        u_end = ffn_range_begin(p.sk_units, clusters, range + 1);
    }

    __host__ __device__ __forceinline__ bool next(FfnItem &w)
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

// The items of a cluster: of one product, or every clusters-th tile of several.
template <int kN>
struct FfnWalk {
    FfnWork one;
    int32_t t, step;

    __host__ __device__ __forceinline__ void init(const FfnArgs<kN> &a, int32_t cluster, int32_t clusters)
    {
        if constexpr (kN == 1)
            one.init(a.p[0], cluster, clusters);
        t = cluster;
        step = clusters;
    }

    __host__ __device__ __forceinline__ bool next(const FfnArgs<kN> &a, FfnItem &w)
    {
        w.product = 0;
        if constexpr (kN == 1) {
            return one.next(w);
        } else {
            if (t >= a.first[kN])
                return false;
            while (t >= a.first[w.product + 1])
                ++w.product;
            w.tile = t - a.first[w.product];
            w.kb0 = 0;
            w.kb1 = a.p[w.product].num_k_blocks;
            t += step;
            return true;
        }
    }
};

struct FfnTile {
    int32_t row, col;
};

// Tile -> (row tile, column tile): bands of raster_group row tiles, walked column by column, odd
// bands right to left, so that tiles running at the same time share operands in L2.
__host__ __device__ __forceinline__ FfnTile ffn_tile_coord(int32_t t, const FfnParams &p)
{
    const uint32_t band = (uint32_t)t / p.band_tiles;
    const int32_t first = (int32_t)band * p.raster_group;
    const int32_t rows = p.num_row_tiles - first < p.raster_group ? p.num_row_tiles - first : p.raster_group;
    const uint32_t r = (uint32_t)t - band * p.band_tiles;
    const int32_t col = (int32_t)(r / (uint32_t)rows);
    return {first + (int32_t)r - col * rows, (band & 1u) ? p.num_col_tiles - 1 - col : col};
}

// ---------------------------------------------------------------- PTX of this kernel
// Shared-memory descriptor of an operand that is contiguous along its rows, as TMA lays it out
// with 128-byte swizzling: chunks of 64 rows x 64 k, a k of a chunk in 128 bytes, 8 k's in 1024
// (the stride offset), chunks 8192 bytes apart (the leading offset).  The other fields are as
// in smem_desc_sw128.  Advancing k by 16 adds 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(8192u >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// D[tmem] (+)= R C^T over a block of 64 elements of k, as four MMAs of 16 whose operands are
// rstep and cstep (in 16 bytes) apart.  Probes the barrier of the next block on the way, so that
// the probe's latency passes while the MMAs issue: 1 if its phase has completed.
template <int CG>
__device__ __forceinline__ uint32_t mma_bf16_block(uint32_t d_tmem, uint64_t rdesc, uint64_t cdesc, uint32_t idesc,
                                                   uint64_t rstep, uint64_t cstep, uint32_t accumulate,
                                                   uint32_t leader, uint32_t next_bar, uint32_t next_parity)
{
    uint32_t ready;
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q, w;\n\t.reg .u64 a, b;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 w, [%9], %10;\n\t"
            "setp.ne.b32 p, %7, 0;\n\t"
            "setp.ne.b32 q, %8, 0;\n\t"
            "mov.u64 a, %2;\n\tmov.u64 b, %3;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, p;\n\t"
            "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
            "setp.ne.b32 p, 1, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, p;\n\t"
            "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, p;\n\t"
            "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, p;\n\t"
            "selp.u32 %0, 1, 0, w;\n\t}"
            : "=r"(ready)
            : "r"(d_tmem), "l"(rdesc), "l"(cdesc), "r"(idesc), "l"(rstep), "l"(cstep), "r"(accumulate), "r"(leader),
              "r"(next_bar), "r"(next_parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q, w;\n\t.reg .u64 a, b;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 w, [%9], %10;\n\t"
            "setp.ne.b32 p, %7, 0;\n\t"
            "setp.ne.b32 q, %8, 0;\n\t"
            "mov.u64 a, %2;\n\tmov.u64 b, %3;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%1], a, b, %4, p;\n\t"
            "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
            "setp.ne.b32 p, 1, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%1], a, b, %4, p;\n\t"
            "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%1], a, b, %4, p;\n\t"
            "add.u64 a, a, %5;\n\tadd.u64 b, b, %6;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%1], a, b, %4, p;\n\t"
            "selp.u32 %0, 1, 0, w;\n\t}"
            : "=r"(ready)
            : "r"(d_tmem), "l"(rdesc), "l"(cdesc), "r"(idesc), "l"(rstep), "l"(cstep), "r"(accumulate), "r"(leader),
              "r"(next_bar), "r"(next_parity)
            : "memory");
    return ready;
}

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}

__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

// One probe: 1 if the phase with this parity has completed.
__device__ __forceinline__ uint32_t mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok;
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// All but the newest committed bulk store of this thread have finished reading shared memory.
__device__ __forceinline__ void bulk_wait_read_all_but_one()
{
    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

// ---------------------------------------------------------------- results through shared memory
// A piece of a result, staged in shared memory as 32 rows of 64 bytes (32 columns of bf16, 16 of
// fp32) in the TMA swizzle of that row size: byte offset of byte `byte` of row r.
__device__ __forceinline__ uint32_t ffn_piece_offset(uint32_t r, uint32_t byte)
{
    return r * 64u + (((byte >> 4) ^ ((r >> 1) & 3u)) << 4) + (byte & 15u);
}

// A warp's two staging buffers, used in turn; every use ends with a commit, so that all but the
// newest group is what used the buffer that comes next.
struct FfnStager {
    uint32_t base;
    int lane;
    uint32_t slot;

    __device__ __forceinline__ uint32_t acquire()
    {
        if (lane == 0)
            bulk_wait_read_all_but_one();
        __syncwarp();
        const uint32_t at = base + slot * kFfnPieceBytes;
        slot ^= 1u;
        return at;
    }
};

// Stores a staged piece at out[y..y+31][x..] by a TMA store, or, where the layout or the last
// columns do not allow one (a TMA store writes whole 16-byte groups), by the warp, a row at a
// time, an element a lane.
__device__ __forceinline__ void ffn_store_piece(uint32_t at, int lane, const CUtensorMap *map, const FfnOut &out,
                                                int32_t x, int32_t y, bool fp32, int32_t D_rows, int32_t D_cols)
{
    const int32_t wide = fp32 ? 16 : 32;
    if (out.tma && (x + wide <= D_cols || D_cols % (fp32 ? 4 : 8) == 0)) {
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (x < D_cols && y < D_rows)
                tma_store_2d(map, at, x, y);
            bulk_commit_group();
        }
        return;
    }
    __syncwarp();
    const int32_t rows = D_rows - y < 32 ? D_rows - y : 32;
    if (fp32) {
        // half a warp a row
        const int32_t c = lane & 15;
        if (x + c < D_cols) {
            float *dst = static_cast<float *>(out.p) + (int64_t)y * out.ld + x + c;
            for (int32_t r = lane >> 4; r < rows; r += 2)
                dst[r * out.ld] = __uint_as_float(ld_shared_u32(at + ffn_piece_offset((uint32_t)r, 4u * (uint32_t)c)));
        }
    } else if (x + lane < D_cols) {
        uint16_t *dst = static_cast<uint16_t *>(out.p) + (int64_t)y * out.ld + x + lane;
        for (int32_t r = 0; r < rows; r += 8) {  // eight rows' loads come before their stores
            uint16_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                asm volatile("ld.shared.u16 %0, [%1];"
                             : "=h"(w[k])
                             : "r"(at + ffn_piece_offset((uint32_t)(r + k), 2u * (uint32_t)lane))
                             : "memory");
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (r + k < rows)
                    *dst = w[k];
                dst += out.ld;
            }
        }
    }
    __syncwarp();
    if (lane == 0)
        bulk_commit_group();
}

// Stores a chunk of 32 x 32 results: w holds pairs of bf16.  Not transposed: thread = row `row`
// + lane, pairs along the columns from `col`.  Transposed: thread = column `col` + lane, pairs
// along the rows.
template <bool kT>
__device__ __forceinline__ void ffn_store_bf16(const uint32_t (&w)[16], FfnStager &st, const CUtensorMap *map,
                                               const FfnOut &out, int32_t row, int32_t col, const FfnParams &p)
{
    const uint32_t at = st.acquire();
    if constexpr (kT) {
        const int32_t live = p.D_rows - row;
#pragma unroll
        for (uint32_t i = 0; i < 16; ++i) {
            if ((int32_t)(2 * i) >= live)
                break;
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + ffn_piece_offset(2 * i, 2u * (uint32_t)st.lane)),
                         "h"((uint16_t)w[i])
                         : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + ffn_piece_offset(2 * i + 1, 2u * (uint32_t)st.lane)),
                         "h"((uint16_t)(w[i] >> 16))
                         : "memory");
        }
    } else {
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u)
            st_shared_v4(at + ffn_piece_offset((uint32_t)st.lane, 16u * u), w[4 * u], w[4 * u + 1], w[4 * u + 2],
                         w[4 * u + 3]);
    }
    ffn_store_piece(at, st.lane, map, out, col, row, false, p.D_rows, p.D_cols);
}

// Stores two chunks of 32 rows x 32 columns, 64 columns apart, with one fence and one wait.  A group for
// each buffer, as acquire() counts them: the first is free before the second.
__device__ __forceinline__ void ffn_store_two(const uint32_t (&w)[2][16], FfnStager &st, const CUtensorMap *map,
                                              const FfnOut &out, int32_t row, int32_t col, const FfnParams &p)
{
    if (st.lane == 0)
        bulk_wait_read_all();
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u)
            st_shared_v4(st.base + h * kFfnPieceBytes + ffn_piece_offset((uint32_t)st.lane, 16u * u), w[h][4 * u],
                         w[h][4 * u + 1], w[h][4 * u + 2], w[h][4 * u + 3]);
    if (out.tma && (col + 96 <= p.D_cols || p.D_cols % 8 == 0)) {
        fence_proxy_async_shared();
        __syncwarp();
        if (st.lane == 0) {
            tma_store_2d(map, st.base, col, row);
            bulk_commit_group();
            if (col + 64 < p.D_cols)
                tma_store_2d(map, st.base + kFfnPieceBytes, col + 64, row);
            bulk_commit_group();
        }
    } else {
        ffn_store_piece(st.base, st.lane, map, out, col, row, false, p.D_rows, p.D_cols);
        if (col + 64 < p.D_cols)
            ffn_store_piece(st.base + kFfnPieceBytes, st.lane, map, out, col + 64, row, false, p.D_rows, p.D_cols);
        else if (st.lane == 0)
            bulk_commit_group();
    }
    st.slot = 0u;
}

template <bool kT>
__device__ __forceinline__ void ffn_store_fp32(const float (&v)[32], FfnStager &st, const CUtensorMap *map,
                                               const FfnOut &out, int32_t row, int32_t col, const FfnParams &p)
{
    if constexpr (kT) {
        // lanes 0-15 fill one piece, 16-31 the other: both buffers are free first
        const uint32_t first = st.acquire();
        if (st.lane == 0)
            bulk_wait_read_all();
        __syncwarp();
        const uint32_t second = first == st.base ? st.base + kFfnPieceBytes : st.base;
        const uint32_t mine = st.lane < 16 ? first : second;
        const int32_t live = p.D_rows - row;
#pragma unroll
        for (uint32_t i = 0; i < 32; ++i) {
            if ((int32_t)i >= live)
                break;
            st_shared_u32(mine + ffn_piece_offset(i, 4u * ((uint32_t)st.lane & 15u)), __float_as_uint(v[i]));
        }
        ffn_store_piece(first, st.lane, map, out, col, row, true, p.D_rows, p.D_cols);
        st.slot ^= 1u;
        ffn_store_piece(second, st.lane, map, out, col + 16, row, true, p.D_rows, p.D_cols);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = st.acquire();
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u)
                st_shared_v4(at + ffn_piece_offset((uint32_t)st.lane, 16u * u), __float_as_uint(v[16 * h + 4 * u]),
                             __float_as_uint(v[16 * h + 4 * u + 1]), __float_as_uint(v[16 * h + 4 * u + 2]),
                             __float_as_uint(v[16 * h + 4 * u + 3]));
            ffn_store_piece(at, st.lane, map, out, col + 16 * h, row, true, p.D_rows, p.D_cols);
        }
    }
}

// ---------------------------------------------------------------- what an epilogue reads
// Raw words of a chunk of an FfnAux for this thread: 32 bf16 as 16 words, or 32 codes as 8 words
// and their scale's byte.
struct FfnRaw {
    uint32_t w[16];
};

__device__ __forceinline__ void load_32_bytes(uint32_t *w, const void *p)
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

// Not transposed: 32 columns of this thread's row.  Rows that start at multiples of 32 bytes come a
// sector a load.  Asynchronous to what follows until the words are used.
__device__ __forceinline__ void ffn_load_rows(FfnRaw &x, const FfnAux &a, int32_t row, int32_t col, const FfnParams &p)
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        x.w[i] = 0u;
    if (row >= p.D_rows || col >= p.D_cols)
        return;
    if (a.scales) {
        const uint8_t *const src = static_cast<const uint8_t *>(a.p) + (int64_t)row * a.ld + col;
        if (a.sectors && col + 32 <= p.D_cols) {
            load_32_bytes(x.w, src);
        } else {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (col + 16 * u < p.D_cols) {  // rows are whole groups of 16
                    const uint4 q = *reinterpret_cast<const uint4 *>(src + 16 * u);
                    x.w[4 * u] = q.x, x.w[4 * u + 1] = q.y, x.w[4 * u + 2] = q.z, x.w[4 * u + 3] = q.w;
                }
        }
        x.w[8] = a.scales[((int64_t)(col >> 9) * p.D_rows + row) * 4 + ((col >> 7) & 3)];
        return;
    }
    const uint16_t *const src = static_cast<const uint16_t *>(a.p) + (int64_t)row * a.ld + col;
    if (a.sectors && col + 32 <= p.D_cols) {
        load_32_bytes(x.w, src);
        load_32_bytes(x.w + 8, src + 16);
        return;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if (col + 8 * u + 8 <= p.D_cols) {
            const uint4 q = *reinterpret_cast<const uint4 *>(src + 8 * u);
            x.w[4 * u] = q.x, x.w[4 * u + 1] = q.y, x.w[4 * u + 2] = q.z, x.w[4 * u + 3] = q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + 8 * u + i < p.D_cols)
                    x.w[4 * u + (i >> 1)] |= (uint32_t)src[8 * u + i] << (16 * (i & 1));
        }
    }
}

// Transposed: column `col` (this thread's) of rows row .. row+31, as fp32.
__device__ __forceinline__ void ffn_load_column(float (&v)[32], const FfnAux &a, int32_t row, int32_t col,
                                                const FfnParams &p)
{
    const int32_t live = col < p.D_cols ? p.D_rows - row : 0;
    if (a.scales) {
        const uint8_t *const src = static_cast<const uint8_t *>(a.p) + (int64_t)row * a.ld + col;
        const uint8_t *const sc = a.scales + ((int64_t)(col >> 9) * p.D_rows + row) * 4 + ((col >> 7) & 3);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            v[i] = 0.0f;
            if (i < live) {
                float hi;
                f32x2_parts(pair_of_e4m3(src[i * a.ld]).v, v[i], hi);
                v[i] *= ffn_scale(sc[4 * i]);
            }
        }
        return;
    }
    const uint16_t *const src = static_cast<const uint16_t *>(a.p) + (int64_t)row * a.ld + col;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = i < live ? __uint_as_float((uint32_t)src[i * a.ld] << 16) : 0.0f;
}

// Values 2 i and 2 i + 1 of a chunk's words (`scale`: what codes are multiplied by).
__device__ __forceinline__ Pair ffn_raw_pair(const FfnRaw &x, int i, bool codes, float scale)
{
    return codes ? pair_of_e4m3(x.w[i >> 1] >> (16 * (i & 1))) * both(scale) : pair_of_bf16(x.w[i]);
}

// Adds bias[at] (kT: one value, this thread's column) or bias[at .. at+31] to the sums.
template <bool kT>
__device__ __forceinline__ void ffn_add_bias(float (&v)[32], int32_t at, const FfnParams &p)
{
    if (p.bias == nullptr)
        return;
    if constexpr (kT) {
        float b = 0.0f;
        if (at < p.D_cols)
            b = p.bias_fp32 ? static_cast<const float *>(p.bias)[at]
                            : __uint_as_float((uint32_t) static_cast<const uint16_t *>(p.bias)[at] << 16);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] += b;
    } else if (p.bias_fp32) {
        const float *const b = static_cast<const float *>(p.bias) + at;
        if (at + 32 <= p.D_cols && (reinterpret_cast<uintptr_t>(b) & 15u) == 0) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float4 q = reinterpret_cast<const float4 *>(b)[u];
                v[4 * u] += q.x, v[4 * u + 1] += q.y, v[4 * u + 2] += q.z, v[4 * u + 3] += q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (at + i < p.D_cols)
                    v[i] += b[i];
        }
    } else {
        const uint16_t *const b = static_cast<const uint16_t *>(p.bias) + at;
        if (at + 32 <= p.D_cols && (reinterpret_cast<uintptr_t>(b) & 15u) == 0) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint4 q = reinterpret_cast<const uint4 *>(b)[u];
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[8 * u + 2 * i] += bf16_low(w[i]);
                    v[8 * u + 2 * i + 1] += bf16_high(w[i]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (at + i < p.D_cols)
                    v[i] += __uint_as_float((uint32_t)b[i] << 16);
        }
    }
}

__device__ __forceinline__ void ffn_pack(uint32_t (&w)[16], const float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
}

__device__ __forceinline__ float *ffn_partial(float *partials, int32_t cta, int ew, int slot, int lane)
{
    return partials + (size_t)cta * kFfnPartialFloats + (size_t)((((ew * 4 + slot) * 8) * 32 + lane) * 4);
}

// v += the 32 fp32 columns of tensor memory at taddr (this warp's 32 lanes), kAtOnce loaded at a time.
template <int kAtOnce>
__device__ __forceinline__ void ffn_add_chunk(uint32_t taddr, uint32_t (&v)[32])
{
#pragma unroll
    for (int h = 0; h < 32; h += kAtOnce) {
        uint32_t t[kAtOnce];
        if constexpr (kAtOnce == 32)
            tmem_load_32x32(taddr, t);
        else
            tmem_load_32x16(taddr + (uint32_t)h, t);
        tmem_load_wait();
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            asm volatile("" : "+r"(t[i])::"memory");
#pragma unroll
        for (int i = 0; i < kAtOnce; i += 2) {
            float lo, hi;
            f32x2_parts((pair(__uint_as_float(v[h + i]), __uint_as_float(v[h + i + 1])) +
                         pair(__uint_as_float(t[i]), __uint_as_float(t[i + 1]))).v,
                        lo, hi);
            v[h + i] = __float_as_uint(lo);
            v[h + i + 1] = __float_as_uint(hi);
        }
    }
}

// ---------------------------------------------------------------- the kernel
// kLong: sums are added up in segments.  The tensor core's additions lose up to a unit of the accumulator each,
// toward zero: a sum over 16384 was off by 1.9e-5 of its size, growing with its length.  bf16 hides that; for a
// result in fp32, and for the codes of 8 bits (of which 8e-4 then rounded to the other side, by up to an eighth),
// the accumulator takes p.segment k-blocks and the sums are added up in the epilogue's registers, rounded to
// nearest: fp32 results are off by 4.8e-7 at any length with segments of 8 (1.0e-6 with 16, 2.1e-6 with 32; products
// in plain fp32 by 2 to 4e-7), and of the codes 4e-5 round to the other side with segments of 16, as after plain fp32
// sums.  Measured (us, with one accumulation and in segments): fp32 linear 4096^3 80.7 and 87.0, 64 x 8192 x 8192
// 27.8 and 29.4, gradients of 4096^3 147.7 and 146.8; gated 8192 x 2048 x 8192 to 8 bits 290 and 287 (331 with
// segments of 8: what follows a tile's sums must pass while the next tile's first two segments do).
template <int CG, bool kT, int kEpi, int kN = 1, bool kLong = false>
__global__ void __launch_bounds__(kFfnThreads, 1) ffn_gemm_kernel(const __grid_constant__ FfnArgs<kN> args)
{
    constexpr bool kPair = CG == 2;
    constexpr bool kDual = kEpi == kFfnGated;
    constexpr int kAccs = kDual ? 2 : 1;  // accumulators of an element
    constexpr bool kCodes = kDual && kLong;  // the gated pair to 8 bits
    static_assert(!kLong || kEpi == kFfnPlain || (kDual && !kT), "forms that segments are made for");
    constexpr uint32_t kTileRBytes = (uint32_t)kFfnRowsPerCta * 128u;
    static_assert(kN == 1 || (kEpi == kFfnPlain && !kT), "several products in one launch are plain ones");
    const FfnParams &p0 = args.p[0];  // what all products share
    const uint32_t stage_bytes = (uint32_t)p0.stage_bytes;  // a multiple of 1024
    // Of 64 rows only these are loaded: the MMA takes what lies behind them for the other 64, whose sums
    // nothing reads.
    auto r_bytes_of = [](const FfnParams &p) { return (uint32_t)p.r_rows * 128u * (kDual && kT ? 2u : 1u); };

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int S = p0.stages;  // even: stages are released in pairs
    const uint32_t stage0 = base;
    const uint32_t staging0 = base + (uint32_t)S * stage_bytes;
    const uint32_t full_bar = staging0 + kFfnEpiWarps * kFfnStagingBytes;
    const uint32_t empty_bar = full_bar + 8u * S;
    const uint32_t accf_bar = empty_bar + 8u * S;
    const uint32_t acce_bar = accf_bar + 16u;
    const uint32_t done_bar = acce_bar + 16u;
    const uint32_t tmem_slot = done_bar + 8u;
    const uint32_t abort_flag = tmem_slot + 4u;
    const uint32_t ready_bar = abort_flag + 4u;  // cluster form: one per epilogue warp of rank 0;
                                                 // behind its eight, one that nothing waits for
    const uint32_t go_words = ready_bar + 72u;   // kCodes: whether the epilogue's wait succeeded, two in turn,
    const uint32_t block_bytes = full_bar + kFfnBarrierBytes;  // and the epilogue warps' scales, 512 bytes twice

    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);  // uniform, and known to be
    const int lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;  // in an SM pair
    const bool shared_tile = kN == 1 && !kPair && p0.cluster > 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar + 8u * s, 1);
            mbar_init(empty_bar + 8u * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(accf_bar + 8u * a, 1);
            mbar_init(acce_bar + 8u * a, kFfnEpiWarps * CG);
        }
        mbar_init(done_bar, 1);
        mbar_init(ready_bar + 64u, 1);
        if (shared_tile)
            for (int e = 0; e < kFfnEpiWarps; ++e)
                mbar_init(ready_bar + 8u * e, (uint32_t)p0.cluster - 1u);  // that warp of every other rank
        st_shared_u32(abort_flag, 0u);
        fence_mbarrier_init();
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < kN; ++i) {
            if (args.p[i].num_k_blocks) {  // an empty sum's operands have no maps
                prefetch_tensormap(&args.maps[i].R[0]);
                prefetch_tensormap(&args.maps[i].C[0]);
            }
            if (args.p[i].D[0].tma)
                prefetch_tensormap(&args.maps[i].D[0]);
        }
    }
    // all CTAs of a cluster have initialised their barriers before any cross-CTA
    // arrive, TMA completion or the paired allocation
    if (kPair || shared_tile) {
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
    ctl.peer_abort_flag = kPair ? mapa_shared(abort_flag, rank ^ 1u) : 0u;
    ctl.err = p0.err;
    ctl.set_limit(p0.watchdog_ns);

    const int32_t cluster_id = (int32_t)blockIdx.x / CG;
    const int32_t num_clusters = (int32_t)gridDim.x / CG;
    FfnWalk<kN> wi;
    wi.init(args, cluster_id, num_clusters);
    FfnItem w;

    if (warp < 4) {
        if (warp != 1) {
            // ---------------- TMA producers ----------------
            // Waiting for a stage, announcing its bytes and issuing its loads take one warp 427
            // clocks a k-block (and 55 more for each load beyond two), as long as 100 columns'
            // MMAs: so the groups of two stages go round the producers.  The stages are released in
            // order, so a producer that has waited for its group before knows that every group two
            // laps behind its next one has been released, as long as there are no more producers
            // than groups in the ring: no parity is mistaken for that of two phases before.
            const int producers = S / 2 < 3 ? S / 2 : 3, me = warp == 0 ? 0 : warp - 1;
            int turn = producers - 1;  // whose group this is
            const uint32_t full_target = kPair ? mapa_shared(full_bar, 0u) : full_bar;
            const uint32_t leader = elect_one();
            int s = 0;
            uint32_t ph = 0;
            int32_t it = 0;
            bool ok = me < producers;
            grid_dependency_wait();
            while (ok && wi.next(args, w)) {
                const FfnParams &p = args.p[w.product];
                const FfnMaps &maps = args.maps[w.product];
                const int32_t width = p.width;
                const uint32_t r_bytes = r_bytes_of(p), loaded = (r_bytes + (uint32_t)p.c_rows * 128u) * CG;  // of a stage
                const FfnTile tc = ffn_tile_coord(w.tile, p);
                const bool other = tc.row >= p.row_split;  // tiles of the second row operand
                const int32_t yr =
                    ((other ? tc.row - p.row_split : tc.row) * CG + (int32_t)rank) * kFfnRowsPerCta;
                const int32_t yc = kDual && !kT ? tc.col * kFfnDualWidth
                                                : tc.col * width + (int32_t)rank * (width / CG);
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    if (ring_group_first(s, 1u)) {
                        turn = turn + 1 == producers ? 0 : turn + 1;
                        const uint32_t bar = empty_bar + 8u * ring_group(s, 1u), parity = ring_empty_parity(ph);
                        if (turn == me && !__all_sync(0xFFFFFFFFu, mbar_wait_tries(bar, parity, ctl.suspend_ns, 1u)) &&
                            !warp_wait<false>(ctl, bar, parity, kRoleProducer, (uint32_t)s, lane)) {
                            ok = false;
                            break;
                        }
                    }
                    if (turn == me && it != p0.fault_skip_it) {
                        if (rank == 0)
                            expect_tx_elected(full_bar + 8u * s, loaded, leader);
                        const uint32_t fb = full_target + 8u * s;
                        const uint32_t sa = stage0 + (uint32_t)s * stage_bytes;
                        const bool second = kb >= p.k_split;
                        const int32_t k = (second ? kb - p.k_split : kb) * kFfnBlockK;
                        if constexpr (kDual && kT) {
                            tma_load_2d_elected<CG>(sa, &maps.R[0], k, yr, fb, leader);
                            tma_load_2d_elected<CG>(sa + kTileRBytes, &maps.R[1], k, yr, fb, leader);
                        } else {
                            const CUtensorMap *mr = second || other ? &maps.R[1] : &maps.R[0];
                            if (p.r_mn) {
                                tma_load_2d_elected<CG>(sa, mr, yr, k, fb, leader);
                                tma_load_2d_elected<CG>(sa + 8192u, mr, yr + 64, k, fb, leader);
                            } else {
                                tma_load_2d_elected<CG>(sa, mr, k, yr, fb, leader);
                            }
                        }
                        const uint32_t sc = sa + r_bytes;
                        if constexpr (kDual && !kT) {
                            if constexpr (CG == 2) {
                                // the pair's MMA takes its first 128 columns from rank 0, the rest from rank 1
                                tma_load_2d_elected<CG>(sc, rank == 0 ? &maps.C[0] : &maps.C[1], k, yc, fb, leader);
                            } else {
                                tma_load_2d_elected<CG>(sc, &maps.C[0], k, yc, fb, leader);
                                tma_load_2d_elected<CG>(sc + kTileRBytes, &maps.C[1], k, yc, fb, leader);
                            }
                        } else {
                            const CUtensorMap *mc = second ? &maps.C[1] : &maps.C[0];
                            if (p.c_mn) {
                                for (int32_t j = 0; j < p.c_rows; j += 64)
                                    tma_load_2d_elected<CG>(sc + (uint32_t)j * 128u, mc, yc + j, k, fb, leader);
                            } else {
                                tma_load_2d_elected<CG>(sc, mc, k, yc, fb, leader);
                            }
                        }
                    }
                    ++it;
                    ring_advance(s, ph, S);
                }
            }
            grid_launch_dependents();
            // Teardown: the last S loads may still be in flight if a role gave up.
            if (lane == 0 && rank == 0) {
                ctl.limit_ns = max(ctl.limit_ns, kFfnDrainNs);
                const int32_t n = it < S ? it : S;
                for (int32_t d = 1; d <= n; ++d) {
                    const int32_t j = it - d;
                    if (j == p0.fault_skip_it || (j >> 1) % producers != me)
                        continue;
                    // one that runs out has outlasted the others' loads too
                    if (!ctl.wait_drain<kPair>(full_bar + 8u * (uint32_t)ring_stage_of(j, S), ring_parity_of(j, S),
                                               (uint32_t)ring_stage_of(j, S)))
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
        } else if (rank == 0) {
            // ---------------- MMA issuer ----------------
            const uint32_t step = stage_bytes >> 4;
            const uint32_t leader = elect_one();
            // A wait that runs out does not leave the k loop: it records the fact, and the rest
            // of the item runs with short single probes and tells nobody.  Above all it releases
            // no stage: one filled again before its first load has landed would count arrivals
            // into a phase that has all of them, which faults.
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
            uint32_t drained = 0u;
            while (wi.next(args, w)) {
                const FfnParams &p = args.p[w.product];
                const uint64_t rdesc0 = p.r_mn ? smem_desc_mn_sw128(stage0) : smem_desc_sw128(stage0);
                const uint32_t r_bytes = r_bytes_of(p);
                const uint64_t cdesc0 =
                    p.c_mn ? smem_desc_mn_sw128(stage0 + r_bytes) : smem_desc_sw128(stage0 + r_bytes);
                const uint64_t rstep = p.r_mn ? 2048u >> 4 : 32u >> 4, cstep = p.c_mn ? 2048u >> 4 : 32u >> 4;
                const int32_t mma_n = kDual && !kT ? 2 * kFfnDualWidth : p.width;
                const uint32_t idesc = idesc_bf16_f32(kFfnRowsPerCta * CG, 0) | ((uint32_t)(mma_n >> 3) << 17) |
                                       (p.r_mn ? 1u << 15 : 0u) | (p.c_mn ? 1u << 16 : 0u);
                wait(acce_bar + 8u * acc, acc_ph ^ 1u, kRoleMmaAcc, (uint32_t)acc);
                tc_fence_after_sync();
                uint32_t d_tmem = tmem_base + (uint32_t)(acc * kFfnMaxWidth);
                int32_t first = w.kb0;  // of the accumulator's k-blocks
                int32_t cut = kLong ? ffn_segment_end(first, p.segment) : 0;
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    if (kLong && kb == cut) {
                        mma_commit_elected<CG>(bad ? nobody_bar : accf_bar + 8u * acc, leader);
                        acc ^= 1;
                        acc_ph ^= acc == 0 ? 1u : 0u;
                        if (!__all_sync(0xFFFFFFFFu, drained))
                            wait(acce_bar + 8u * acc, acc_ph ^ 1u, kRoleMmaAcc, (uint32_t)acc);
                        tc_fence_after_sync();
                        d_tmem = tmem_base + (uint32_t)(acc * kFfnMaxWidth);
                        first = kb;
                        cut += p.segment;
                    }
                    if (!__all_sync(0xFFFFFFFFu, ready))
                        wait(full_bar + 8u * s, ring_full_parity(ph), kRoleMmaFull, (uint32_t)s);
                    tc_fence_after_sync();
                    const uint64_t off = (uint64_t)((uint32_t)s * step);
                    int s1 = s;
                    uint32_t ph1 = ph;
                    ring_advance(s1, ph1, S);
                    const uint32_t add = kb > (kLong ? first : w.kb0) ? 1u : 0u;
                    if constexpr (kDual && kT)
                        mma_bf16_block<CG>(d_tmem + kFfnDualWidth, rdesc0 + off + (kTileRBytes >> 4), cdesc0 + off,
                                           idesc, rstep, cstep, add, leader, full_bar + 8u * s1, ring_full_parity(ph1));
                    ready = mma_bf16_block<CG>(d_tmem, rdesc0 + off, cdesc0 + off, idesc, rstep, cstep, add, leader,
                                               full_bar + 8u * s1, ring_full_parity(ph1));
                    if (kLong && kb + 1 == cut)  // the other accumulator's barrier, as the next stage's
                        drained = mbar_test(acce_bar + 8u * (acc ^ 1), (acc == 1 ? acc_ph ^ 1u : acc_ph) ^ 1u);
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
                ctl.limit_ns = max(ctl.limit_ns, kFfnDrainNs);
                ctl.wait_drain<kPair>(done_bar, 0u, 0xFFFu);
            }
            __syncwarp();
        }
    } else {
        // ---------------- epilogue ----------------
        grid_dependency_wait();
        const int ew = warp - 4;
        const int q = warp & 3;    // tensor-memory lane quadrant
        const int half = ew >> 2;  // takes chunks half, half + 2, ... of 32 columns
        FfnStager st = {staging0 + (uint32_t)ew * kFfnStagingBytes, lane, 0u};
        const uint32_t acce_target = kPair ? mapa_shared(acce_bar, 0u) : acce_bar;
        const int32_t cta = cluster_id * CG + (int32_t)rank;
        // the CTA of this rank that a range is of, where tiles meet through global memory
        auto cta_of = [&](int32_t range) { return (num_clusters - 1 - range) * CG + (int32_t)rank; };
        int acc = 0;
        uint32_t acc_ph = 0;
        const bool dense = p0.sk_units >= num_clusters;  // every range holds a unit
        uint32_t go_parity = 0u, block_parity = 0u;
        // each warp for itself: the warps of a tile need not keep step.  But where warps exchange block maxima
        // (kCodes) one thread waits and posts the outcome, so that all take the same branch; the word
        // alternates.
        auto accumulated = [&]() {
            if constexpr (kCodes) {
                const uint32_t go = go_words + 4u * go_parity;
                go_parity ^= 1u;
                if (threadIdx.x == 128)
                    st_volatile_shared_u32(
                        go, ctl.wait<kPair>(accf_bar + 8u * acc, acc_ph, kRoleEpilogue, (uint32_t)acc) ? 1u : 0u);
                named_barrier_sync(1u, kFfnEpiWarps * 32u);
                return ld_volatile_shared_u32(go) != 0u;
            } else {
                return warp_wait<kPair>(ctl, accf_bar + 8u * acc, acc_ph, kRoleEpilogue, (uint32_t)acc, lane);
            }
        };
        // this warp has read its part of the accumulator: hand it back
        auto hand_back = [&]() {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kPair)
                    mbar_arrive_cluster_handoff(acce_target + 8u * acc);
                else
                    mbar_arrive(acce_bar + 8u * acc);
            }
        };
        auto chunk_at = [&](int a, int c) {
            return tmem_base + ((uint32_t)(q * 32) << 16) +
                   (uint32_t)(acc * kFfnMaxWidth + a * kFfnDualWidth + c * 32);
        };
        auto load_chunk = [&](int a, int c, uint32_t(&v)[32]) { tmem_load_32x32(chunk_at(a, c), v); };
        while (wi.next(args, w)) {
            const FfnParams &p = args.p[w.product];
            const FfnMaps &maps = args.maps[w.product];
            const int32_t KB = p.num_k_blocks, width = p.width;
            const int nchunks = (width + 31) / 32;
            const FfnTile tc = ffn_tile_coord(w.tile, p);
            const bool other = tc.row >= p.row_split;
            // the accumulator's rows and columns of this warp
            const int32_t yr =
                ((other ? tc.row - p.row_split : tc.row) * CG + (int32_t)rank) * kFfnRowsPerCta + q * 32;
            const int32_t yc = tc.col * width;
            const bool contributor = kN == 1 && w.kb0 > 0;
            const bool owner = kN == 1 && w.kb0 == 0 && w.kb1 < KB;
            // the ranges that start inside this tile, up to the last, owner only; a range may be empty
            // (fewer units than clusters), and then leaves nothing
            const int32_t range = num_clusters - 1 - cluster_id;
            int32_t last = range;
            bool parts = owner;
            auto collect = [&]() {
                if (owner && shared_tile) {
                    uint32_t got = 1u;
                    if (lane == 0)
                        got = ctl.wait<true>(ready_bar + 8u * (uint32_t)ew, 0u, kRoleFixup, (uint32_t)ew) ? 1u : 0u;
                    __syncwarp();  // lane 0's acquire comes before the lanes' loads
                    parts = __shfl_sync(0xFFFFFFFFu, got, 0) != 0u;
                } else if (owner) {
                    last = ffn_range_of(p.sk_units, num_clusters, (int64_t)(w.tile + 1) * KB - 1);
                    for (int32_t j2 = range + 1; parts && j2 <= last; ++j2)
                        if (dense || ffn_range_holds(p.sk_units, num_clusters, j2))
                            // a give-up stores the tile unsummed, and the status says so
                            parts = warp_wait_flag(ctl, p.flags + cta_of(j2) * kFfnEpiWarps + ew, 1u, lane);
                    __syncwarp();  // lane 0's acquires come before the lanes' loads
                }
            };
            // one chunk's sums of one accumulator: left for the tile's owner, or completed; false if left
            auto complete = [&](int a, int c, uint32_t(&v)[32]) {
                const int slot = (c >> 1) + 2 * a;
                // The cluster form keeps a partial in the CTA's own ring: a
                // contributor's only item has consumed all of its loads by now.
                const uint32_t local = stage0 + (uint32_t)((((ew * 4 + slot) * 8) * 32 + lane) * 16);
                // (of a transposed result, only its rows' columns, four at a time)
                const int live = kT ? min(8, (p.cols - (yc + c * 32) + 3) >> 2) : 8;
                if (contributor && shared_tile) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < live)
                            st_shared_v4(local + 512u * j, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    return false;
                }
                if (contributor) {
                    float4 *const part = reinterpret_cast<float4 *>(ffn_partial(p.partials, cta, ew, slot, lane));
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < live)
                            __stcg(part + j * 32, make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                                              __uint_as_float(v[4 * j + 2]),
                                                              __uint_as_float(v[4 * j + 3])));
                    return false;
                }
                if (parts && shared_tile) {
                    for (int32_t rk = 1; rk < p.cluster; ++rk) {
                        const uint32_t remote = mapa_shared(local, (uint32_t)rk);
                        uint32_t x[32];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < live)
                                ld_shared_cluster_v4(remote + 512u * j, x[4 * j], x[4 * j + 1], x[4 * j + 2],
                                                     x[4 * j + 3]);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < live)
#pragma unroll
                                for (int e = 4 * j; e < 4 * j + 4; ++e)
                                    v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(x[e]));
                    }
                } else if (parts) {
                    for (int32_t j2 = range + 1; j2 <= last; ++j2) {
                        if (!dense && !ffn_range_holds(p.sk_units, num_clusters, j2))
                            continue;
                        const float4 *const part = reinterpret_cast<const float4 *>(
                            ffn_partial(p.partials, cta_of(j2), ew, slot, lane));
                        float4 f[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < live)
                                f[j] = __ldcg(part + j * 32);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < live) {
                                v[4 * j] = __float_as_uint(__uint_as_float(v[4 * j]) + f[j].x);
                                v[4 * j + 1] = __float_as_uint(__uint_as_float(v[4 * j + 1]) + f[j].y);
                                v[4 * j + 2] = __float_as_uint(__uint_as_float(v[4 * j + 2]) + f[j].z);
                                v[4 * j + 3] = __float_as_uint(__uint_as_float(v[4 * j + 3]) + f[j].w);
                            }
                    }
                }
                return true;
            };
            // where chunk c lies in the results, for this thread or (kT) this warp's first row
            const int32_t d_row0 = kT ? yc : yr;
            const int32_t d_col0 = kT ? yr : yc;
            constexpr int kAux = kEpi == kFfnGrad ? 2 : kEpi == kFfnPlain ? 1 : 0;
            // rows are asked for ahead of their use
            FfnRaw raw[kAux > 0 ? kAux : 1];
            auto ahead = [&](int c) {
                if constexpr (!kT && kAux > 0) {
#pragma unroll
                    for (int i = 0; i < kAux; ++i)
                        if (p.aux[i].p)
                            ffn_load_rows(raw[i], p.aux[i], yr + lane, yc + c * 32, p);
                }
            };
            // transposed, a residual's first chunk: a column, an element a load, all of them ahead too (64 x
            // 8192 x 8192 with a residual and a bias 34.7 us without)
            constexpr bool kEarly = kT && kEpi == kFfnPlain && !kLong;
            static_assert(kFfnEarlyColumns == 2 * 32, "the two halves' first chunks");
            uint16_t early[kEarly ? 32 : 1];
            auto ahead_column = [&]() {
                if constexpr (kEarly) {
                    const int32_t row = yc + half * 32, live = yr + lane < p.D_cols ? p.D_rows - row : 0;
                    const uint16_t *const src = static_cast<const uint16_t *>(p.aux[0].p) + (int64_t)row * p.aux[0].ld + yr + lane;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        early[e] = e < live ? src[e * p.aux[0].ld] : (uint16_t)0;
                }
            };
            auto aux_pairs = [&](int i, int c, Pair(&f)[16]) {
                if (kEarly && c == half) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        f[e] = pair(__uint_as_float((uint32_t)early[kEarly ? 2 * e : 0] << 16),
                                    __uint_as_float((uint32_t)early[kEarly ? 2 * e + 1 : 0] << 16));
                } else if constexpr (kT) {
                    float v[32];
                    ffn_load_column(v, p.aux[i], yc + c * 32, yr + lane, p);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        f[e] = pair(v[2 * e], v[2 * e + 1]);
                } else {
                    const bool codes = p.aux[i].scales != nullptr;
                    const float scale = codes ? ffn_scale(raw[i].w[8]) : 1.0f;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        f[e] = ffn_raw_pair(raw[i], e, codes, scale);
                }
            };
            if (!kLong && !contributor && half < nchunks) {
                ahead(half);
                if (kEarly && p.aux[0].p)
                    ahead_column();
            }
            if constexpr (kT && kAux > 0) {
                // columns are read where they are used, from L2 by then: a line a lane
                if (!contributor && d_col0 < p.D_cols)
                    for (int c = kEarly ? half + 2 : half; c < nchunks; c += 2)
#pragma unroll
                        for (int i = 0; i < kAux; ++i)
                            if (p.aux[i].p && d_row0 + c * 32 + lane < p.D_rows)
                                prefetch_l2(static_cast<const uint8_t *>(p.aux[i].p) +
                                            ((int64_t)(d_row0 + c * 32 + lane) * p.aux[i].ld + d_col0) *
                                                (p.aux[i].scales ? 1 : 2));
            }
            float inv[2] = {0.0f, 0.0f};  // kCodes: this thread's row's scales, inverted
            bool infinite = false;        // and whether this warp holds infinities, whose codes are NaN
            // one chunk's sums: left for the tile's owner, or completed and stored
            auto finish = [&](int c, uint32_t(&v)[kAccs][32]) {
                bool whole = true;
#pragma unroll
                for (int a = 0; a < kAccs; ++a)
                    whole = complete(a, c, v[a]);
                const int32_t row = d_row0 + (kT ? c * 32 : 0), col = d_col0 + (kT ? 0 : c * 32);
                if (!whole || row >= p.D_rows || col >= p.D_cols) {
                    if (!kLong && whole && c + 2 < nchunks)
                        ahead(c + 2);
                    return;
                }
                uint32_t pk[16];
                if constexpr (kEpi == kFfnPlain) {
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        f[i] = __uint_as_float(v[0][i]);
                    const FfnOut &out = other ? p.D[1] : p.D[0];
                    const CUtensorMap *const map = other ? &maps.D[1] : &maps.D[0];
                    ffn_add_bias<kT>(f, kT ? col + lane : col, p);
                    if (p.save) {
                        ffn_pack(pk, f);
                        ffn_store_bf16<kT>(pk, st, &maps.D[1], p.D[1], row, col, p);
                    }
                    if (p.act != kActNone)
                        ffn_with_act(p.act, [&](auto tag) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                f32x2_parts(ffn_act<decltype(tag)::value>(pair(f[2 * i], f[2 * i + 1])).v, f[2 * i],
                                            f[2 * i + 1]);
                        });
                    if (p.aux[0].p) {
                        Pair r[16];
                        if constexpr (kLong)
                            ahead(c);  // its words would take registers from the sums before
                        aux_pairs(0, c, r);
                        if (!kLong && c + 2 < nchunks)
                            ahead(c + 2);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            f32x2_parts((pair(f[2 * i], f[2 * i + 1]) + r[i]).v, f[2 * i], f[2 * i + 1]);
                    }
                    if (p.out_fp32) {
                        ffn_store_fp32<kT>(f, st, map, out, row, col, p);
                    } else {
                        ffn_pack(pk, f);
                        ffn_store_bf16<kT>(pk, st, map, out, row, col, p);
                    }
                } else if constexpr (kEpi == kFfnGated) {
                    if (!kCodes && p.save) {
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                pk[i] = pack_bf16x2(v[a][2 * i], v[a][2 * i + 1]);
                            ffn_store_bf16<kT>(pk, st, &maps.D[1 + a], p.D[1 + a], row, col, p);
                        }
                    }
                    if constexpr (kCodes) {
                        if (row + lane < p.D_rows) {
                            // 32 codes of this thread's row, one sector
#pragma unroll
                            for (int a = 0; a < 2; ++a) {
                                uint32_t code[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    float e[4];
#pragma unroll
                                    for (int j = 0; j < 4; ++j) {
                                        e[j] = __uint_as_float(v[a][4 * i + j]);
                                        e[j] = (infinite ? inf_to_nan(e[j]) : e[j]) * inv[a];
                                    }
                                    code[i] = pack_e4m3x4(e[0], e[1], e[2], e[3]);
                                }
                                uint4 *const dst =
                                    reinterpret_cast<uint4 *>(p.codes[a] + (int64_t)(row + lane) * p.ldq[a] + col);
                                dst[0] = make_uint4(code[0], code[1], code[2], code[3]);
                                dst[1] = make_uint4(code[4], code[5], code[6], code[7]);
                            }
                        }
                    }
                    ffn_with_act(p.act, [&](auto tag) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            pk[i] = bf16_pair(
                                ffn_act<decltype(tag)::value>(
                                    pair(__uint_as_float(v[0][2 * i]), __uint_as_float(v[0][2 * i + 1]))) *
                                pair(__uint_as_float(v[1][2 * i]), __uint_as_float(v[1][2 * i + 1])));
                    });
                    ffn_store_bf16<kT>(pk, st, &maps.D[0], p.D[0], row, col, p);
                } else {
                    Pair g[16], u[16];
                    aux_pairs(0, c, g);
                    aux_pairs(1, c, u);
                    if (c + 2 < nchunks)
                        ahead(c + 2);
                    uint32_t pdu[16], ph[16];
                    ffn_with_act(p.act, [&](auto tag) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const Pair dh = pair(__uint_as_float(v[0][2 * i]), __uint_as_float(v[0][2 * i + 1]));
                            Pair a, d;
                            ffn_act_slope<decltype(tag)::value>(g[i], a, d);
                            pk[i] = bf16_pair(dh * u[i] * d);
                            pdu[i] = bf16_pair(dh * a);
                            ph[i] = bf16_pair(a * u[i]);
                        }
                    });
                    ffn_store_bf16<kT>(pk, st, &maps.D[0], p.D[0], row, col, p);
                    ffn_store_bf16<kT>(pdu, st, &maps.D[1], p.D[1], row, col, p);
                    ffn_store_bf16<kT>(ph, st, &maps.D[2], p.D[2], row, col, p);
                }
            };
            if constexpr (kLong) {
                constexpr int kOwn = (kDual ? kFfnDualWidth : ffn_long_width(CG, kT)) / 64;  // chunks of a warp
                uint32_t run[kOwn][kAccs][32];
#pragma unroll
                for (int i = 0; i < kOwn; ++i)
#pragma unroll
                    for (int a = 0; a < kAccs; ++a)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            run[i][a][j] = 0u;
                bool ok = accumulated();
                if (!ok)
                    break;
                tc_fence_after_sync();
                if (KB) {  // an empty sum's accumulator holds nothing
#pragma unroll
                    for (int i = 0; i < kOwn; ++i)
                        if (half + 2 * i < nchunks) {
#pragma unroll
                            for (int a = 0; a < kAccs; ++a)
                                load_chunk(a, half + 2 * i, run[i][a]);
                        }
                    tmem_load_wait();
#pragma unroll
                    for (int i = 0; i < kOwn; ++i)
#pragma unroll
                        for (int a = 0; a < kAccs; ++a)
                            reg_fence(run[i][a]);
                }
                for (int32_t cut = ffn_segment_end(w.kb0, p.segment);; cut += p.segment) {
                    hand_back();
                    acc ^= 1;
                    acc_ph ^= acc == 0 ? 1u : 0u;
                    if (cut >= w.kb1 || !(ok = accumulated()))
                        break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int i = 0; i < kOwn; ++i)
                        if (half + 2 * i < nchunks) {
#pragma unroll
                            for (int a = 0; a < kAccs; ++a)
                                ffn_add_chunk<kOwn * kAccs == 4 ? 16 : 32>(chunk_at(a, half + 2 * i), run[i][a]);
                        }
                }
                if (!ok)
                    break;
                collect();
                if constexpr (kCodes) {
                    // A block of the format is the tile's 128 columns, of which this warp holds half, and another
                    // the other half.
                    float top[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < kOwn; ++i)
#pragma unroll
                        for (int a = 0; a < 2; ++a)
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                top[a] = fmaxf(top[a], fabsf(__uint_as_float(run[i][a][j])));
                    infinite = __any_sync(0xFFFFFFFFu, is_inf(top[0]) || is_inf(top[1]));
                    if (infinite) {  // infinities are no part of it
                        top[0] = top[1] = 0.0f;
#pragma unroll
                        for (int i = 0; i < kOwn; ++i)
#pragma unroll
                            for (int a = 0; a < 2; ++a)
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    top[a] = fmaxf(top[a], finite_abs(__uint_as_float(run[i][a][j])));
                    }
                    // The larger of the two halves' scales: a byte each, in two places used in turn, so that one
                    // barrier does: whoever writes to a place has passed the barrier behind its last reads.
                    uint32_t mine = scale_byte(top[0]) | scale_byte(top[1]) << 8, theirs;
                    const uint32_t at = block_bytes + 512u * block_parity + 2u * (uint32_t)lane;
                    block_parity ^= 1u;
                    st_shared_u16(at + 64u * (uint32_t)ew, mine);
                    named_barrier_sync(2u + (uint32_t)q, 64u);
                    theirs = ld_shared_u16(at + 64u * (uint32_t)(ew ^ 4));
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const uint32_t byte = max(mine >> (8 * a) & 0xFFu, theirs >> (8 * a) & 0xFFu);
                        inv[a] = scale_inverse(byte);
                        const int32_t row = yr + lane, block = tc.col;
                        if (half == a && row < p.D_rows) {
                            uint8_t *const word = p.scales[a] + ((int64_t)(block >> 2) * p.D_rows + row) * 4;
                            word[block & 3] = (uint8_t)byte;
                            if (block == p.num_col_tiles - 1)
                                for (int i = (block & 3) + 1; i < 4; ++i)
                                    word[i] = 127;
                        }
                    }
                }
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
                int c0 = half;
                if constexpr (kEpi == kFfnPlain && !kT) {
                    // whole tiles of bf16, most of the work: two chunks at a time, whose loads, stores and
                    // fences overlap (4096 x 8192 x 128 with relu 23.1 us, and 30.9 one by one)
                    const bool two = KB && !p.out_fp32 && !contributor && !owner;
                    if (two && !p.bias && p.act == kActNone && !p.aux[0].p && !p.save)
                        // the sums as they are, as in every gradient: apart, in little code, since fetching it is
                        // what counts (8192 x 8192 x 64 25.4 us, and 35.3 through the loop below)
                        for (; c0 + 2 < nchunks; c0 += 4) {
                            uint32_t v[2][32], pk[2][16];
                            load_chunk(0, c0, v[0]);
                            load_chunk(0, c0 + 2, v[1]);
                            tmem_load_wait();
                            reg_fence(v[0]);
                            reg_fence(v[1]);
                            if (c0 + 4 >= nchunks)
                                hand_back();
                            const int32_t col = d_col0 + c0 * 32;
                            if (yr >= p.D_rows || col >= p.D_cols)
                                continue;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    pk[h][i] = pack_bf16x2(v[h][2 * i], v[h][2 * i + 1]);
                            ffn_store_two(pk, st, other ? &maps.D[1] : &maps.D[0], other ? p.D[1] : p.D[0], yr, col, p);
                        }
                    else if (two)
                        for (; c0 + 2 < nchunks; c0 += 4) {
                            uint32_t v[2][32];
                            load_chunk(0, c0, v[0]);
                            load_chunk(0, c0 + 2, v[1]);
                            tmem_load_wait();
                            reg_fence(v[0]);
                            reg_fence(v[1]);
                            if (c0 + 4 >= nchunks)
                                hand_back();
                            const int32_t col = d_col0 + c0 * 32;
                            if (yr >= p.D_rows || col >= p.D_cols)
                                continue;
                            float f[2][32];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    f[h][i] = __uint_as_float(v[h][i]);
                                ffn_add_bias<false>(f[h], col + 64 * h, p);
                            }
                            uint32_t pk[2][16];
                            if (p.save) {
                                ffn_pack(pk[0], f[0]);
                                ffn_pack(pk[1], f[1]);
                                ffn_store_two(pk, st, &maps.D[1], p.D[1], yr, col, p);
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (p.act != kActNone)
                                    ffn_with_act(p.act, [&](auto tag) {
#pragma unroll
                                        for (int i = 0; i < 16; ++i)
                                            f32x2_parts(ffn_act<decltype(tag)::value>(pair(f[h][2 * i], f[h][2 * i + 1])).v,
                                                        f[h][2 * i], f[h][2 * i + 1]);
                                    });
                                if (p.aux[0].p) {
                                    Pair r[16];
                                    aux_pairs(0, c0 + 2 * h, r);
                                    if (c0 + 2 * h + 2 < nchunks)
                                        ahead(c0 + 2 * h + 2);
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        f32x2_parts((pair(f[h][2 * i], f[h][2 * i + 1]) + r[i]).v, f[h][2 * i],
                                                    f[h][2 * i + 1]);
                                }
                                ffn_pack(pk[h], f[h]);
                            }
                            ffn_store_two(pk, st, other ? &maps.D[1] : &maps.D[0], other ? p.D[1] : p.D[0], yr, col, p);
                        }
                }
                for (int c = c0; c < nchunks; c += 2) {
                    uint32_t v[kAccs][32];
#pragma unroll
                    for (int a = 0; a < kAccs; ++a)
                        load_chunk(a, c, v[a]);
                    tmem_load_wait();
#pragma unroll
                    for (int a = 0; a < kAccs; ++a) {
                        reg_fence(v[a]);
                        if (KB == 0) {  // an empty sum
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[a][i] = 0u;
                        }
                    }
                    if (c + 2 >= nchunks)
                        hand_back();
                    if (c == half && owner)
                        collect();  // after this piece's own sums have been read
                    finish(c, v);
                }
                acc ^= 1;
                acc_ph ^= acc == 0 ? 1u : 0u;
            }
            if (contributor) {
                __syncwarp();  // the warp's stores come before lane 0's release
                if (lane == 0 && shared_tile)
                    mbar_arrive_cluster(mapa_shared(ready_bar + 8u * (uint32_t)ew, 0u));
                else if (lane == 0)
                    st_release_gpu_u32(p.flags + cta * kFfnEpiWarps + ew, 1u);
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
    if (kPair || shared_tile)
        cluster_arrive_wait();  // the peer is done with this CTA's memory
    if (warp == 2) {
        tc_fence_after_sync();
        tmem_dealloc<CG>(tmem_base, 512);
    }
}

}  // namespace wstma
