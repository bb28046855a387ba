// Host side of the C ABI declared in include/ffn_ops.h: argument checks, plans,
// TMA tensor maps and launches.
#include "ffn_ops.h"

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "ffn_kernels.h"
#include "ffn_overlap.h"

using namespace wstma;

namespace {

constexpr int64_t kMaxDim = 0x7FFFFFFFLL - 1023;  // a tile past the last row still has a 32-bit index
constexpr size_t kWorkAlign = 256;    // of the parts of a workspace
constexpr int64_t kMaxPitch = int64_t(1) << 37;
constexpr int64_t kMaxElements = int64_t(1) << 50;  // of a matrix, pitch and all: a call's sizes and offsets fit 64 bits
constexpr int kNumOptions = 11;
constexpr int kPlans = 64;              // plans a thread remembers
constexpr int kMaxCtas = 1024;          // bounds the workspace of split tiles
constexpr int64_t kMinSplitBlocks = 8;  // k-blocks per cluster below which tiles are not split further

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int from_cuda(cudaError_t e)
{
    if (e == cudaSuccess)
        return FFN_OK;
    cudaGetLastError();
    return FFN_ERR_CUDA;
}

// --------------------------------------------------------------- device
struct Device {
    int index = -1;
    int sms = 0;
    int max_smem = 0;
    int max_pairs = 0;  // SM pairs that are resident at once
};

// The current device, looked up once per device.
int current_device(Device *out)
{
    static Device known[64];
    static std::mutex lock;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return from_cuda(cudaErrorUnknown);
    if (dev >= 64)
        return FFN_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> hold(lock);
    if (known[dev].index < 0) {
        Device d;
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.max_smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
            return from_cuda(cudaErrorUnknown);
        if (major != 10 || minor != 3)
            return FFN_ERR_UNSUPPORTED;
        d.sms = std::min(d.sms, kMaxCtas);
        const void *fn = ffn_plain_fn(2, false);
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        int n = 0;
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(kFfnThreads, 1, 1);
        cfg.dynamicSmemBytes = ffn_smem_bytes(32768, 4);
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, d.max_smem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1)
            return from_cuda(cudaErrorUnknown);
        d.max_pairs = std::min(n, d.sms / 2);
        d.index = dev;
        known[dev] = d;
    }
    *out = known[dev];
    return FFN_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

bool encode_2d(CUtensorMap *m, bool fp32, const void *ptr, int64_t cols, int64_t rows, int64_t row_bytes, int box_cols,
               int box_rows, CUtensorMapSwizzle swizzle)
{
    auto fn = encode_fn();
    if (!fn)
        return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
              const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// --------------------------------------------------------------- a product
// One operand: `rows` (rows or columns of the result) by k, contiguous along k, or (mn) along
// its rows: in memory then k rows of `rows` elements.
struct Operand {
    const void *p = nullptr;
    int64_t ld = 0;
};

enum Form : int32_t {
    kOne = 0,    // A[0] B[0]
    kSum = 1,    // A[0] B[0] + A[1] B[1]
    kStack = 2,  // A[0] B[0] and A[1] B[0], results D[0] and D[1]
    kDual = 3    // A[0] B[0] and A[0] B[1], both sums of an element in one thread
};

struct Product {
    int epilogue = kFfnPlain;
    Form form = kOne;
    int64_t M = 0, N = 0, K = 0;
    bool a_mn = false, b_mn = false;
    Operand A[2], B[2];
    FfnParams p = {};  // what the epilogue needs
    bool own_a = false, own_b = false;  // operands that an earlier step of the call has made
    bool no_split = false, not_transposed = false;
    ffn_matrix D[3] = {};  // results
    bool fp32 = false;     // of D[0], and D[1] of kStack
};

int64_t k_blocks_of(const Product &x) { return ceil_div(x.K, kFfnBlockK) * (x.form == kSum ? 2 : 1); }

struct Options {
    int64_t v[kNumOptions] = {0, 0, 0, 0, 1, 2000000000, -1, 0, 0, 0, 0};
};
thread_local Options options;

// What a plan follows from; compared as bytes.
struct PlanKey {
    int64_t M, N, K;
    int64_t opt[5];
    int32_t device, epilogue, form, flags;
};

struct Plan {
    PlanKey key;
    uint64_t used;
    bool transposed;
    int cta_group, width, c_rows, r_rows, stages, grid, cluster;
    int64_t row_tiles, row_split, col_tiles, tiles, k_blocks, k_split, sk_tiles;
    size_t smem, stage_bytes;
    const void *fn;
    double cost;
};

// Up to kFfnMaxProducts products in one launch, if that takes less time than one after the other.
struct Together {
    PlanKey key[kFfnMaxProducts];
    uint64_t used;
    bool yes;
    Plan plan[kFfnMaxProducts];
};

thread_local Plan plans[kPlans];
thread_local Together togethers[16];
thread_local uint64_t plan_clock = 0;
thread_local Plan last_plan;
thread_local bool have_last_plan = false;
thread_local int32_t last_packed = 0, last_products = 0;

// Sums that go to 8 bits are always added up in segments, those of an fp32 result where there are several.
bool to_codes(const Product &x) { return x.epilogue == kFfnGated && x.p.save == 2; }
bool long_sum(const Product &x) { return x.fp32 && k_blocks_of(x) > kFfnSegment; }

const void *kernel_fn(const Product &x, int cta_group, bool transposed)
{
    return to_codes(x)                ? ffn_gated_codes_fn(cta_group)
           : x.epilogue == kFfnGated  ? ffn_gated_fn(cta_group, transposed)
           : x.epilogue == kFfnGrad   ? ffn_grad_fn(cta_group, transposed)
           : long_sum(x)              ? ffn_plain_segments_fn(cta_group, transposed)
                                      : ffn_plain_fn(cta_group, transposed);
}

// The widest tile of a product on the column side.
int widest_tile(const Product &x, int cta_group, bool transposed)
{
    return x.form == kDual ? kFfnDualWidth : long_sum(x) ? ffn_long_width(cta_group, transposed) : kFfnMaxWidth;
}

// A way to tile a product, and what it costs.
struct Tiling {
    bool transposed = false;
    int cta_group = 0, width = 0;
    // found by tiling_cost()
    int c_rows = 0, r_rows = 0;
    size_t stage_bytes = 0;
    int64_t clusters = 0;  // SM pairs, or CTAs, of the grid
    int64_t sk_tiles = 0;
    int cluster = 1;  // CTAs that share a tile in a cluster
    double tile = 0.0, epilogue = 0.0, hbm = 0.0;
};

struct Sides {
    int64_t rows, cols;  // of the accumulator
    int64_t row_tiles, col_tiles;
    bool c_mn;
};

Sides sides_of(const Product &x, const Tiling &t)
{
    Sides s;
    s.rows = t.transposed ? x.N : x.M;
    s.cols = t.transposed ? x.M : x.N;
    s.row_tiles = ceil_div(s.rows, kFfnRowsPerCta * t.cta_group) * (x.form == kStack ? 2 : 1);
    s.col_tiles = ceil_div(s.cols, t.width);
    s.c_mn = t.transposed ? x.a_mn : x.b_mn;
    return s;
}

int ring_stages(const Device &d, size_t stage_bytes)
{
    int S = kFfnMaxStages;
    while (S > 2 && ffn_smem_bytes(stage_bytes, S) > (size_t)d.max_smem)
        S -= 2;
    return S;
}

// Estimated time of a tiling, in clocks of an SM (1.9 GHz), without what every launch costs:
// the tiles of the longest chain, each its stages (k-blocks: the longest of the MMAs, 4096
// multiply-adds a clock and SM, the loads, 62 bytes a clock and SM and 9231 over all SMs, and a stage's
// handling, 394 clocks, or 345 where half of its rows are loaded) or its epilogue; or the operands' time in HBM and their repeated loads', if longer;
// then the last epilogue and the exchange between a split tile's pieces.  The constants were fitted to 3400
// measured tilings of 51 products in all forms, of which the one of least estimate took at most 11 % longer
// than the best, 0.9 % in the mean.  What came later (stages of half the rows, HBM's own rate, a residual asked for
// ahead) follows kernels that changed: against the same measurements it is 21 % at most and 2.8 % in the mean.
// The products had rows at multiples of 128 bytes: where rows straddle lines the choice can be further off (852 x
// 1328 x 8840 takes 40 us, and 30.5 in pairs of 192 columns).  Fills in how the tiles are shared out.
double tiling_cost(const Device &d, const Product &x, int64_t KB, Tiling &t)
{
    const Sides s = sides_of(x, t);
    const bool dual = x.form == kDual;
    if (dual && !t.transposed)
        t.c_rows = t.cta_group == 2 ? kFfnDualWidth : 2 * kFfnDualWidth;
    else
        t.c_rows = ffn_chunk_rows(s.c_mn, t.width / t.cta_group);
    // Up to 64 tokens on the row side: half the stage, and half again as many of them in flight (64 x 8192 x 8192
    // in tiles of 64 columns 30.6 us, and 27.5 so; with bias and residual 31.6 and 28.5).
    t.r_rows = !t.transposed && !x.a_mn && t.cta_group == 1 && x.M <= 64 ? 64 : kFfnRowsPerCta;
    t.stage_bytes = (size_t)t.r_rows * 128 * (dual && t.transposed ? 2 : 1) + (size_t)t.c_rows * 128;
    const int64_t tiles = s.row_tiles * s.col_tiles;
    const int64_t split = x.no_split ? 0 : options.v[FFN_OPT_SPLIT];
    const int64_t most = t.cta_group == 2 ? d.max_pairs : d.sms;
    const double sums = (dual ? 2.0 : 1.0) * t.width;  // columns of sums a row
    const double l2 = (double)t.stage_bytes * (double)(std::min(tiles, most) * t.cta_group) / 9231.0;
    const double handling = t.r_rows < kFfnRowsPerCta ? 345.0 : 394.0;
    const double stage = std::max({2.0 * sums, handling, (double)t.stage_bytes / 62.5, l2});
    const double once = (double)(x.M + x.N * (dual ? 2 : 1)) * (double)x.K * 2.0;
    const double loads = (double)tiles * (double)KB * (double)t.stage_bytes * t.cta_group;
    // (the measured tilings' operands were in L2 in part; 134 MB of them take HBM's own rate)
    const double read = std::min(once / 3530.0, once / 4661.0 + std::max(0.0, once - 6.4e7) / 7600.0);
    const double hbm = read + std::max(0.0, loads - once) / 40743.0;
    // What an epilogue does with a chunk, in stores of one: a transposed result's rows are read an element
    // at a time (the gradient of 800 x 5256 x 3872 from 8 bits takes 173 us that way, and 75 not transposed).
    const bool grad = x.epilogue == kFfnGrad;
    double results = grad || (dual && x.p.save == 1) ? 3.0 : x.p.save == 1 ? 2.0 : 1.0;
    for (const FfnAux &a : x.p.aux)
        if (a.p && t.transposed)  // of a residual, what the kernel asks for ahead costs little
            results += a.scales ? 14.0 : !grad && !long_sum(x) && t.width <= kFfnEarlyColumns ? 2.0 : 6.4;
    const double epilogue = 15.6 * sums * results;
    const double chunks = grad && !t.transposed ? 90.0 * sums + 4800.0
                                                : (4.0 * sums + 1853.0) * results * (t.transposed ? 1.7 : 1.0);
    // a gradient's epilogue and the loads of the next tile slow each other down
    const double tile =
        std::max((double)KB * stage, chunks) + (grad ? 0.15 * std::min((double)KB * stage, chunks) : 0.0);

    t.tile = tile;
    t.epilogue = epilogue;
    t.hbm = hbm;
    t.clusters = std::min(tiles, most);
    t.sk_tiles = 0;
    t.cluster = 1;
    double best = std::max((double)ceil_div(tiles, t.clusters) * tile, hbm) + epilogue;
    if (split == 1 && t.cta_group == 1) {
        // each tile shared by a cluster of CTAs
        const int64_t c = std::min<int64_t>({most / tiles, kFfnMaxCluster, KB});
        if (c >= 2) {
            const double exchange = 7685.0 + (130.0 + 14.1 * sums) * (double)(c - 1);
            const double cost = std::max((double)ceil_div(KB, c) * stage, hbm) + epilogue + exchange;
            if (cost < best) {
                best = cost;
                t.clusters = tiles * c;
                t.sk_tiles = tiles;
                t.cluster = (int)c;
            }
        }
    }
    // The last, partial wave of tiles (or all, if they do not fill one) shared by all clusters.  (With a wave
    // more of tiles shared, so that few pieces make a tile, nothing was gained: 160 tiles, 84 and 8 of them
    // shared by 76 pairs, 98 and 94 us.)
    const int64_t sk = tiles % most;
    const int64_t C = tiles > most ? most : std::max(tiles, std::min(most, tiles * KB / kMinSplitBlocks));
    const int64_t whole = C ? (tiles - sk) / C : 0;
    // (a gradient's epilogues are what its tiles wait for: 1000 x 3000 x 1000 takes 26 us with its last wave
    // shared, and 20.  Sums held in registers wait with the next tile's segments: fp32 4096^3 98.7 and 87.0, 6143 x
    // 5999 x 4104 216 either way.  An empty sum has no k-blocks to share: its tiles are walked whole.)
    if (split && KB && sk && C > sk && !((grad || long_sum(x)) && whole)) {
        // behind whole tiles the exchange is out of sight for as long as one takes: the split tiles come first
        const double meet = 11435.0 + (59.0 + 25.4 * sums) * (double)C / (double)sk;
        const double exchange = whole ? std::max(6396.0, meet - tile) : meet;
        const double cost =
            std::max((double)whole * tile + (double)ceil_div(sk * KB, C) * stage, hbm) + epilogue + exchange;
        if (cost < best) {
            best = cost;
            t.clusters = C;
            t.sk_tiles = sk;
            t.cluster = 1;
        }
    }
    return best;
}

// How many clusters of c CTAs of a one-SM kernel are resident at once.
int resident_clusters(const Device &d, const void *fn, size_t smem, int c)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int n = 0;
    cfg.gridDim = dim3((unsigned)c, 1, 1);
    cfg.blockDim = dim3(kFfnThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, d.max_smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

// The plan of a tiling, without its ring and grid.
int plan_tiles(const Product &x, const Tiling &t, Plan &pl)
{
    const Sides s = sides_of(x, t);
    pl.transposed = t.transposed;
    pl.cta_group = t.cta_group;
    pl.width = t.width;
    pl.c_rows = t.c_rows;
    pl.r_rows = t.r_rows;
    pl.stage_bytes = t.stage_bytes;
    pl.row_tiles = s.row_tiles;
    pl.row_split = x.form == kStack ? s.row_tiles / 2 : s.row_tiles;
    pl.col_tiles = s.col_tiles;
    pl.tiles = s.row_tiles * s.col_tiles;
    pl.k_blocks = k_blocks_of(x);
    pl.k_split = x.form == kSum ? pl.k_blocks / 2 : pl.k_blocks;
    pl.sk_tiles = 0;
    pl.cluster = 1;
    // pieces of an empty sum are none: its tiles would be nobody's
    return pl.tiles > kMaxDim || pl.k_blocks > kMaxDim || (t.sk_tiles && !pl.k_blocks) ? FFN_ERR_UNSUPPORTED : FFN_OK;
}

// The tiling of least estimate, and how its tiles are shared out; false if the options allow none.
bool choose_tiling(const Device &d, const Product &x, Tiling &best, double &best_cost)
{
    const int64_t *opt = options.v;
    const int64_t KB = k_blocks_of(x);
    best = {false, 0, 0};
    for (int cg = 1; cg <= 2; ++cg)
        for (int tr = 0; tr <= 1; ++tr) {
            if ((opt[FFN_OPT_CTA_GROUP] && cg != opt[FFN_OPT_CTA_GROUP]) ||
                (tr && (x.not_transposed || x.form == kStack)) ||
                (opt[FFN_OPT_TRANSPOSED] && tr + 1 != opt[FFN_OPT_TRANSPOSED] && !x.not_transposed &&
                 x.form != kStack))
                continue;
            const bool fixed = x.form == kDual && !tr;
            const int widest = widest_tile(x, cg, tr != 0);
            // a width that sums in segments do not have stands for the widest that they have
            const int64_t asked = long_sum(x) ? std::min<int64_t>(opt[FFN_OPT_WIDTH], widest) : opt[FFN_OPT_WIDTH];
            for (int wd = fixed ? kFfnDualWidth : 16; wd <= widest; wd += 16) {
                if (asked && wd != asked && !fixed)
                    continue;
                // chunks of 32 columns: a narrower tile must be the only one
                const int64_t cols = tr ? x.M : x.N;
                if (wd % 32 != 0 && (cg == 2 || wd < cols))
                    continue;
                Tiling t = {tr != 0, cg, wd};
                const double cost = tiling_cost(d, x, KB, t);
                if (best.cta_group == 0 || cost < best_cost)
                    best = t, best_cost = cost;
            }
        }
    return best.cta_group != 0;
}

int make_plan(const Device &d, const Product &x, Plan &pl)
{
    Tiling best;
    double best_cost = 0.0;
    if (!choose_tiling(d, x, best, best_cost))
        return FFN_ERR_UNSUPPORTED;
    const int rc = plan_tiles(x, best, pl);
    if (rc != FFN_OK)
        return rc;
    pl.cost = best_cost;
    pl.stages = ring_stages(d, pl.stage_bytes);
    pl.smem = ffn_smem_bytes(pl.stage_bytes, pl.stages);
    pl.fn = kernel_fn(x, pl.cta_group, pl.transposed);
    // All clusters at once: the largest size that the device can place so often.
    if (best.cluster > 1) {
        while (best.cluster > 1 && resident_clusters(d, pl.fn, pl.smem, best.cluster) < pl.tiles)
            --best.cluster;
        best.clusters = pl.tiles * best.cluster;
        best.sk_tiles = best.cluster > 1 ? pl.tiles : 0;
    }
    pl.sk_tiles = best.sk_tiles;
    pl.cluster = best.cluster;
    pl.grid = (int)(best.clusters * best.cta_group);
    return from_cuda(cudaFuncSetAttribute(pl.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, d.max_smem));
}

PlanKey key_of(const Device &d, const Product &x)
{
    PlanKey key;
    std::memset(&key, 0, sizeof(key));
    key.M = x.M, key.N = x.N, key.K = x.K;
    for (int i = FFN_OPT_CTA_GROUP; i <= FFN_OPT_SPLIT; ++i)
        key.opt[i] = options.v[i];
    key.opt[0] = options.v[FFN_OPT_TOGETHER];
    key.device = d.index, key.epilogue = x.epilogue, key.form = x.form;
    key.flags = (x.a_mn ? 1 : 0) | (x.b_mn ? 2 : 0) | (x.no_split ? 4 : 0) | (x.not_transposed ? 8 : 0) |
                (x.p.aux[0].p ? 16 : 0) | (x.p.aux[0].scales ? 32 : 0) | (x.p.save << 6) | (long_sum(x) ? 256 : 0);
    return key;
}

int find_plan(const Device &d, const Product &x, Plan *out)
{
    const PlanKey key = key_of(d, x);
    Plan *slot = &plans[0];
    for (Plan &pl : plans) {
        if (pl.used && std::memcmp(&pl.key, &key, sizeof(key)) == 0) {
            pl.used = ++plan_clock;
            *out = pl;
            return FFN_OK;
        }
        if (pl.used < slot->used)
            slot = &pl;
    }
    Plan pl;
    std::memset(&pl, 0, sizeof(pl));
    const int rc = make_plan(d, x, pl);
    if (rc != FFN_OK)
        return rc;
    pl.key = key;
    pl.used = ++plan_clock;
    *slot = pl;
    *out = pl;
    return FFN_OK;
}

// What each launch costs beyond its estimate: 3.7 us for the least product.
constexpr double kLaunchClocks = 8000.0;

// Whether n plain products, none of which needs another's result, take less time in one launch, and
// their plans there: one kind of tile, the products with the longest tiles first, every cluster taking
// each clusters-th tile of all.  (In one launch and in several, from a graph: linear_backward of 16 x 512 x 512 4.8
// and 9.3 us, of 4096^3 143 and 151 to 155, the same with gelu by tanh and a bias 168 to 171 and 174;
// gated_backward of 4115 x 361 x 888 52 and 70, of 2047 x 2056 x 5999 240 and 252.)
int find_together(const Device &d, Product **xs, const Plan *alone, int n, const Together **out)
{
    PlanKey key[kFfnMaxProducts];
    std::memset(key, 0, sizeof(key));
    for (int i = 0; i < n; ++i)
        key[i] = key_of(d, *xs[i]);
    Together *slot = &togethers[0];
    for (Together &t : togethers) {
        if (t.used && std::memcmp(t.key, key, sizeof(key)) == 0) {
            t.used = ++plan_clock;
            *out = &t;
            return FFN_OK;
        }
        if (t.used < slot->used)
            slot = &t;
    }
    const int64_t *opt = options.v;
    double separate = (n - 1) * kLaunchClocks;
    bool segments = false;
    for (int i = 0; i < n; ++i) {
        separate += alone[i].cost;
        segments = segments || long_sum(*xs[i]);
    }
    Tiling best[kFfnMaxProducts];
    double best_cost = 0.0;
    int best_cg = 0;
    for (int cg = 1; cg <= 2; ++cg)
        for (int wd = 32; wd <= (segments ? ffn_long_width(cg, false) : kFfnMaxWidth); wd += 32) {
            if ((opt[FFN_OPT_CTA_GROUP] && cg != opt[FFN_OPT_CTA_GROUP]) || opt[FFN_OPT_TRANSPOSED] == 2 ||
                (opt[FFN_OPT_WIDTH] && wd != (segments ? std::min<int64_t>(opt[FFN_OPT_WIDTH], ffn_long_width(cg, false))
                                                       : opt[FFN_OPT_WIDTH])))
                continue;
            Tiling t[kFfnMaxProducts];
            const int64_t C = cg == 2 ? d.max_pairs : d.sms;
            double hbm = 0.0, epilogue = 0.0;
            int64_t count[kFfnMaxProducts], total = 0;
            for (int i = 0; i < n; ++i) {
                t[i] = {false, cg, wd};
                tiling_cost(d, *xs[i], k_blocks_of(*xs[i]), t[i]);
                const Sides s = sides_of(*xs[i], t[i]);
                count[i] = s.row_tiles * s.col_tiles;
                total += count[i];
                hbm += t[i].hbm;
                epilogue = std::max(epilogue, t[i].epilogue);
            }
            // the cluster whose tiles take longest
            double chain = 0.0;
            for (int64_t c = 0; c < std::min(C, total); ++c) {
                double sum = 0.0;
                int64_t first = 0;
                for (int i = 0; i < n; ++i) {
                    const auto upto = [&](int64_t end) { return end > c ? (end - c - 1) / C + 1 : 0; };
                    sum += (double)(upto(first + count[i]) - upto(first)) * t[i].tile;
                    first += count[i];
                }
                chain = std::max(chain, sum);
            }
            const double cost = std::max(chain, hbm) + epilogue;
            if (best_cg == 0 || cost < best_cost) {
                best_cg = cg;
                best_cost = cost;
                for (int i = 0; i < n; ++i)
                    best[i] = t[i];
            }
        }
    Together g;
    std::memset(&g, 0, sizeof(g));
    g.yes = best_cg && opt[FFN_OPT_TOGETHER] != 2 && (opt[FFN_OPT_TOGETHER] == 1 || best_cost < separate);
    if (g.yes) {
        size_t stage_bytes = 0;
        int64_t total = 0;
        for (int i = 0; i < n; ++i) {
            const int rc = plan_tiles(*xs[i], best[i], g.plan[i]);
            if (rc != FFN_OK)
                return rc;
            stage_bytes = std::max(stage_bytes, g.plan[i].stage_bytes);
            total += g.plan[i].tiles;
        }
        if (total > kMaxDim)
            return FFN_ERR_UNSUPPORTED;
        for (int i = 0; i < n; ++i) {
            Plan &pl = g.plan[i];
            pl.stage_bytes = stage_bytes;
            pl.stages = ring_stages(d, stage_bytes);
            pl.smem = ffn_smem_bytes(stage_bytes, pl.stages);
            pl.fn = segments ? ffn_together_segments_fn(best_cg) : ffn_together_fn(best_cg);
            pl.grid = (int)std::min<int64_t>(total, best_cg == 2 ? d.max_pairs : d.sms) * best_cg;
        }
        const int rc = from_cuda(
            cudaFuncSetAttribute(g.plan[0].fn, cudaFuncAttributeMaxDynamicSharedMemorySize, d.max_smem));
        if (rc != FFN_OK)
            return rc;
    }
    std::memcpy(g.key, key, sizeof(key));
    g.used = ++plan_clock;
    *slot = g;
    *out = slot;
    return FFN_OK;
}

// --------------------------------------------------------------- workspace
// A call runs twice: once to measure its workspace and to list the operands that it copies, launching
// nothing, then in earnest.  The copies of all its products come first, in one launch, which also
// clears the flags of all their split tiles.  The workspace holds, in this order: what the call's steps
// hand on, the copies, the flags, and the split tiles' partials, which the products share since they
// run one after another.
struct Call {
    Device dev;
    cudaStream_t stream = nullptr;
    uint8_t *base = nullptr;  // null: measuring
    size_t used = 0;          // of the first part
    size_t flags = 0;         // words so far
    FfnPackJobs jobs = {};    // measuring: `dst` is an offset from the first copy
    size_t copies = 0;        // their bytes
    size_t partials = 0;      // measuring: the largest product's bytes; else where they start
    uint32_t *flag_words = nullptr;
    bool measuring() const { return base == nullptr; }

    static size_t whole(size_t bytes) { return (bytes + kWorkAlign - 1) / kWorkAlign * kWorkAlign; }
    size_t bytes() const { return used + copies + whole(flags * sizeof(uint32_t)) + partials; }

    // a part of the workspace for this call's steps: its place (null when measuring)
    void *take(size_t bytes)
    {
        const size_t at = used;
        used += whole(bytes);
        return base ? base + at : nullptr;
    }
};

// Rows that the library makes start at multiples of 128 bytes.
int64_t padded(int64_t cols) { return (cols + 63) / 64 * 64; }

// A matrix's copy: listed when measuring, found later.
void copy_first(Call &c, Operand &o, int64_t mem_rows, int64_t mem_cols);

// An operand's rows as a product reads them: as they are, or copied.  Copied are rows that no tensor
// map describes (not at multiples of 16 bytes), and long operands whose rows are not at multiples of
// 128: each 128-byte row of a box then straddles two lines of L2, a quarter more clocks a k-block.  The
// copy moves the operand twice; that pays from some 3600 `readers`, rows on the other side, on, and
// for some more its launch: 4096 x 4104 x 4104 takes 105 us with both operands copied and 108.5 as they
// are, 2000 x 4104 x 4104 63 and 57, 6143 x 5999 x 4104 196 and 224.  What an earlier step of the call has
// made (`own`) needs none.
void prepare_operand(Call &c, Operand &o, int64_t mem_rows, int64_t mem_cols, int64_t readers, bool own)
{
    if (mem_rows < 1 || mem_cols < 1)
        return;
    const bool describable = aligned(o.p, 16) && (o.ld % 8 == 0 || mem_rows <= 1);
    const bool straddles = mem_rows > 1 && (o.ld % 64 != 0 || !aligned(o.p, 128));
    const int64_t mode = options.v[FFN_OPT_REPACK];
    if (own || (describable && !(straddles && (mode == 1 || (mode == 0 && (double)(readers - 3600) * (double)mem_rows * (double)mem_cols > 8e9))))) {
        if (mem_rows <= 1)
            o.ld = padded(mem_cols);
        return;
    }
    copy_first(c, o, mem_rows, mem_cols);
}

void copy_first(Call &c, Operand &o, int64_t mem_rows, int64_t mem_cols)
{
    const FfnPackJob *found = nullptr;  // two products may read one matrix
    for (int i = 0; i < c.jobs.n; ++i) {
        const FfnPackJob &j = c.jobs.job[i];
        if (j.src == o.p && j.lds == o.ld && j.R == mem_rows && j.C == mem_cols)
            found = &j;
    }
    if (!found) {  // measuring
        FfnPackJob &job = c.jobs.job[c.jobs.n++];
        job.src = static_cast<const uint16_t *>(o.p);
        job.lds = o.ld;
        job.ldd = padded(mem_cols);
        job.dst = reinterpret_cast<uint16_t *>(c.copies);
        c.copies += Call::whole((size_t)(mem_rows * job.ldd) * 2);
        job.R = mem_rows;
        job.C = (int32_t)mem_cols;
        found = &job;
    }
    o.p = found->dst;
    o.ld = found->ldd;
}

void set_out(FfnOut &out, CUtensorMap *map, const ffn_matrix &m, bool fp32, int64_t rows, int64_t cols)
{
    out.p = m.data;
    out.ld = rows > 1 ? m.ld : padded(cols);
    const int esize = fp32 ? 4 : 2;
    out.tma = aligned(m.data, 16) && out.ld * esize % 16 == 0 &&
              encode_2d(map, fp32, m.data, cols, rows, out.ld * esize, 64 / esize, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

FfnAux aux_of(const ffn_matrix &m)
{
    FfnAux a;
    a.p = m.data;
    a.ld = m.ld;
    return a;
}

FfnAux aux_of(const ffn_quantized &q)
{
    FfnAux a;
    a.p = q.codes;
    a.ld = q.ld;
    a.scales = static_cast<const uint8_t *>(q.scales);
    return a;
}

// Whether a product goes to the kernel for few tokens (ffn_stream.cu, with both sides' times): a
// forward product whose operands are as its 16-byte loads need them, and whose rows fit its one pass.
// Up to 8 tokens it is the faster one throughout, up to 16 but for a large gated pair (16 x 16384 x
// 4096 52 us against 47), up to 32 for small weights (4096 x 4096 12.3 us against 13.4, 8192 x 8192
// 36 against 34).  Between these points, and with this kernel's times first: 24 x 4096 x 6144 15.2 and 16.9,
// gated 24 x 6144 x 4096 23.8 and 31.2, gated 12 x 8192 x 8192 48.7 and 58.9, which go to the other one; 12 x 14336 x
// 4096 24.8 and 22.1, which does not.
bool streams(const Call &c, const Product &x)
{
    const bool dual = x.form == kDual;
    if (options.v[FFN_OPT_STREAM] == 2 || x.M > kFfnStreamTokens || x.K < 1 || x.K % 8 != 0 || x.a_mn || x.b_mn ||
        x.N > ffn_stream_rows(c.dev.sms) || !(dual ? x.p.save != 2 : x.form == kOne && x.epilogue == kFfnPlain))
        return false;
    if (!aligned(x.A[0].p, 16) || (x.M > 1 && x.A[0].ld % 8 != 0))
        return false;
    for (int i = 0; i < (dual ? 2 : 1); ++i)
        if (!aligned(x.B[i].p, 16) || (x.N > 1 && x.B[i].ld % 8 != 0))
            return false;
    if (options.v[FFN_OPT_STREAM] == 1 || x.M <= 8)
        return true;
    return x.M <= 16 ? !dual || x.N * x.K <= 1 << 25 : x.N * x.K <= 1 << 24;
}

// Whether a product goes to the kernel for few tokens and weights that are contiguous along the result's
// columns (ffn_stream_back.cu, with both sides' times).  A gated gradient's do up to 8 tokens, and, where the
// weights are of a middling size, up to 16; the whole gradient takes (us, so and without)
//   1024 x 4096     8 tokens 25.4, 38.7;   16 tokens 31.3, 39.7
//   2048 x 8192     8 tokens 52.9, 75.5;   16 tokens 61.8, 75.0
//   4096 x 16384    8 tokens 175, 184;     16 tokens 182, 168
//   512 x 1024      8 tokens 15.1, 15.6;   16 tokens 19.9, 15.7
// The limits lie between those points; close to them the other choice may be the better one (512 x 2048, 12
// tokens, 19.7 and 23.5, goes to the other kernel; 1024 x 2048 23.0 and 28.0 as well).
// A single dx does where its sum is long; shorter ones do better beside dW in one launch:
//   4096 x 4096     8 tokens 23.6, 27.2;   16 tokens 27.1, 26.6
//   12288 x 512     8 tokens 17.0, 20.9;   2048 x 2048  8 tokens 12.5, 9.3
//   8192 x 8192     8 tokens 58.5, 59.0;   16 tokens 65.2, 59.4
//   4096 x 1024    12 tokens 14.6, 18.8;   3584 x 2048  8 tokens 17.3, 21.0: both go to the other kernel
// (253 products of few tokens in all four forms: the choice takes 2.5 % longer than the better of the two in the
// mean, 32 % at most.)
bool streams_back(const Call &c, const Product &x)
{
    if (options.v[FFN_OPT_STREAM] == 2 || x.M > kFfnStreamBackTokens || x.K < 1 || x.a_mn || !x.b_mn || x.fp32 ||
        x.N > ffn_stream_back_columns(c.dev.sms) ||
        !(x.epilogue == kFfnGrad || (x.epilogue == kFfnPlain && (x.form == kOne || x.form == kSum))))
        return false;
    for (int i = 0; i < (x.form == kSum ? 2 : 1); ++i)
        if (!aligned(x.A[i].p, 8) || (x.M > 1 && x.A[i].ld % 4 != 0) || !aligned(x.B[i].p, 16) ||
            (x.K > 1 && x.B[i].ld % 8 != 0))
            return false;
    if (options.v[FFN_OPT_STREAM] == 1)
        return true;
    if (x.epilogue == kFfnGrad || x.form == kSum)
        return x.M <= 8 || (x.N * x.K > 1 << 21 && x.N * x.K <= 1 << 25);
    return x.M <= 8 && x.K >= 4096;
}

void remember(const Call &c, const Plan &pl, int products);

int run_stream_back(Call &c, const Product &x)
{
    if (c.measuring())
        return FFN_OK;
    FfnStreamBackParams p = {};
    p.products = x.form == kSum ? 2 : 1;
    for (int i = 0; i < p.products; ++i) {
        p.d[i] = static_cast<const uint16_t *>(x.A[i].p);
        p.ldd[i] = x.A[i].ld;
        p.w[i] = static_cast<const uint16_t *>(x.B[i].p);
        p.ldw[i] = x.B[i].ld;
    }
    p.M = (int32_t)x.M, p.N = (int32_t)x.K, p.C = (int32_t)x.N;
    p.act = x.p.act;
    for (int i = 0; i < 2; ++i)
        p.aux[i] = x.p.aux[i];
    for (int i = 0; i < 3; ++i) {
        p.D[i].p = x.D[i].data;
        p.D[i].ld = x.D[i].ld;
    }
    Plan none;
    std::memset(&none, 0, sizeof(none));
    remember(c, none, 1);
    return from_cuda((cudaError_t)launch_ffn_stream_back(p, c.dev.index, c.dev.sms, c.stream));
}

int run_stream(Call &c, const Product &x)
{
    if (c.measuring())
        return FFN_OK;
    FfnStreamParams p = {};
    p.x = static_cast<const uint16_t *>(x.A[0].p);
    p.ldx = x.A[0].ld;
    for (int i = 0; i < (x.form == kDual ? 2 : 1); ++i) {
        p.w[i] = static_cast<const uint16_t *>(x.B[i].p);
        p.ldw[i] = x.B[i].ld;
    }
    p.M = (int32_t)x.M, p.N = (int32_t)x.N, p.K = (int32_t)x.K;
    p.act = x.p.act;
    p.bias = x.p.bias;
    p.bias_fp32 = x.p.bias_fp32;
    p.residual = static_cast<const uint16_t *>(x.p.aux[0].p);
    p.ldr = x.p.aux[0].ld;
    for (int i = 0; i < 3; ++i) {
        p.D[i].p = x.D[i].data;
        p.D[i].ld = x.D[i].ld;
    }
    p.out_fp32 = x.fp32 ? 1 : 0;
    p.save = x.p.save;
    Plan none;
    std::memset(&none, 0, sizeof(none));
    remember(c, none, 1);
    return from_cuda((cudaError_t)launch_ffn_stream(p, c.dev.sms, c.stream));
}

// Height of the bands that tiles are walked in: as many row tiles as 32 MB of the row operand hold, so
// that they stay in L2 from one column to the next, but 8 at least, and all if there are no more than 16;
// bands of one height.  Under the power cap, with bands of 8 and of 16 or 32: 4096 x 16384 x 4096 329 and 319
// us, gated 616 and 600, 8192 x 8192 x 2048 gated 312 and 303, 16384 x 8192 x 4096 627 and 620; 8192^3 648 and
// 655 (here 8 hold 32 MB).
int32_t band_of(const Plan &pl, int64_t K)
{
    const int64_t asked = options.v[FFN_OPT_RASTER_GROUP];
    if (asked)
        return (int32_t)std::min(asked, pl.row_tiles);
    const int64_t tile = (int64_t)kFfnRowsPerCta * pl.cta_group * std::max<int64_t>(K, 1);
    const int64_t most = pl.row_tiles <= 16 ? 16 : std::max<int64_t>(8, (int64_t(1) << 24) / tile);
    return (int32_t)ceil_div(pl.row_tiles, ceil_div(pl.row_tiles, most));
}

// A product's operands, and what its epilogue reads, as its kernel takes them: as they are, or copied.
void prepare(Call &c, Product &x, const Plan &pl)
{
    for (int i = 0; i < 2; ++i) {
        const bool has_a = i == 0 || x.form == kSum || x.form == kStack;
        const bool has_b = i == 0 || x.form == kSum || x.form == kDual;
        if (has_a)
            prepare_operand(c, x.A[i], x.a_mn ? x.K : x.M, x.a_mn ? x.M : x.K, x.N, x.own_a);
        if (has_b)
            prepare_operand(c, x.B[i], x.b_mn ? x.K : x.N, x.b_mn ? x.N : x.K, x.form == kStack ? 2 * x.M : x.M,
                            x.own_b);
    }
    // What an epilogue reads a row a thread, it reads by 16 bytes (element by element, through shared
    // memory, the gradient of 2047 x 5999 took 227 us, not 62); a column a thread, as it is.
    for (FfnAux &a : x.p.aux) {
        if (a.p && !a.scales && !pl.transposed && (!aligned(a.p, 16) || (a.ld % 8 != 0 && x.M > 1))) {
            Operand o = {a.p, a.ld};
            copy_first(c, o, x.M, x.N);
            a.p = o.p;
            a.ld = o.ld;
        }
        a.sectors = aligned(a.p, 32) && (a.ld * (a.scales ? 1 : 2) % 32 == 0 || x.M <= 1);
    }
}

// The kernel's view of a product that has been prepared.
int describe(const Product &x, const Plan &pl, FfnMaps &maps, FfnParams &p)
{
    p = x.p;
    const Operand *R = pl.transposed ? x.B : x.A, *C = pl.transposed ? x.A : x.B;
    const int64_t rows = pl.transposed ? x.N : x.M, cols = pl.transposed ? x.M : x.N;
    p.r_mn = pl.transposed ? x.b_mn : x.a_mn;
    p.c_mn = pl.transposed ? x.a_mn : x.b_mn;
    const bool two_r = x.form == kSum || x.form == kStack || (x.form == kDual && pl.transposed);
    const bool two_c = x.form == kSum || (x.form == kDual && !pl.transposed);
    const int c_box = x.form == kDual && !pl.transposed ? kFfnDualWidth : pl.width / pl.cta_group;
    auto encode = [&](CUtensorMap *m, const Operand &o, bool mn, int64_t extent, int box_rows) {
        return mn ? encode_2d(m, false, o.p, extent, x.K, o.ld * 2, 64, kFfnBlockK, CU_TENSOR_MAP_SWIZZLE_128B)
                  : encode_2d(m, false, o.p, x.K, extent, o.ld * 2, kFfnBlockK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (pl.k_blocks) {
        for (int i = 0; i < 2; ++i)
            if ((i < (two_r ? 2 : 1) && !encode(&maps.R[i], R[i], p.r_mn, rows, pl.r_rows)) ||
                (i < (two_c ? 2 : 1) && !encode(&maps.C[i], C[i], p.c_mn, cols, c_box)))
                return FFN_ERR_TENSORMAP;
    }
    for (int i = 0; i < 3; ++i)
        if (x.D[i].data)
            set_out(p.D[i], &maps.D[i], x.D[i], x.fp32 && (i == 0 || x.form == kStack), x.M, x.N);
    p.rows = (int32_t)rows;
    p.cols = (int32_t)cols;
    p.D_rows = (int32_t)x.M;
    p.D_cols = (int32_t)x.N;
    p.num_k_blocks = (int32_t)pl.k_blocks;
    p.k_split = (int32_t)pl.k_split;
    p.num_row_tiles = (int32_t)pl.row_tiles;
    p.num_col_tiles = (int32_t)pl.col_tiles;
    p.num_tiles = (int32_t)pl.tiles;
    p.row_split = (int32_t)pl.row_split;
    p.width = pl.width;
    p.c_rows = pl.c_rows;
    p.r_rows = pl.r_rows;
    p.stage_bytes = (int32_t)pl.stage_bytes;
    p.stages = pl.stages;
    p.raster_group = band_of(pl, x.K);
    p.band_tiles = ffn_band_tiles(p.raster_group, pl.col_tiles);
    p.segment = to_codes(x) ? kFfnCodesSegment : long_sum(x) ? kFfnSegment : 0x7FFFFFFF;
    p.sk_tiles = (int32_t)pl.sk_tiles;
    p.sk_units = pl.sk_tiles * pl.k_blocks;
    p.cluster = pl.cluster;
    p.out_fp32 = x.fp32 ? 1 : 0;
    p.err = ffn_status_word();
    if (!p.err)
        return FFN_ERR_CUDA;
    // a tile's waits grow with K; 2 us a k-block is far above any measured
    p.watchdog_ns = std::max<uint64_t>((uint64_t)options.v[FFN_OPT_WATCHDOG_NS],
                                       options.v[FFN_OPT_FAULT_SKIP_LOAD] >= 0 ? 0 : (uint64_t)pl.k_blocks * 2000u);
    p.fault_skip_it = (int32_t)options.v[FFN_OPT_FAULT_SKIP_LOAD];
    return FFN_OK;
}

int launch(const Call &c, const Plan &pl, void *arg)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)pl.grid, 1, 1);
    cfg.blockDim = dim3(kFfnThreads, 1, 1);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = c.stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    const int together = pl.cta_group * pl.cluster;  // one of the two is 1
    attr[1].val.clusterDim.x = (unsigned)together;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = together > 1 ? 2 : 1;
    void *args[1] = {arg};
    return from_cuda(cudaLaunchKernelExC(&cfg, pl.fn, args));
}

void remember(const Call &c, const Plan &pl, int products)
{
    last_plan = pl;
    last_packed = c.jobs.n;
    last_products = products;
    have_last_plan = true;
}

// Runs one product.
int run_product(Call &c, Product &x)
{
    if (x.M == 0 || x.N == 0)
        return FFN_OK;
    if (streams(c, x))
        return run_stream(c, x);
    if (streams_back(c, x))
        return run_stream_back(c, x);
    Plan pl;
    int rc = find_plan(c.dev, x, &pl);
    if (rc != FFN_OK)
        return rc;
    prepare(c, x, pl);
    const bool meets = pl.sk_tiles && pl.cluster == 1;  // tiles' pieces meet through global memory
    const size_t flags = meets ? (size_t)pl.grid * kFfnEpiWarps : 0, first_flag = c.flags;
    c.flags += flags;
    if (c.measuring()) {
        c.partials = std::max(c.partials, meets ? (size_t)pl.grid * kFfnPartialFloats * sizeof(float) : 0);
        return FFN_OK;
    }
    FfnArgs<1> args;
    std::memset(static_cast<void *>(&args), 0, sizeof(args));
    if ((rc = describe(x, pl, args.maps[0], args.p[0])) != FFN_OK)
        return rc;
    args.p[0].partials = meets ? reinterpret_cast<float *>(c.base + c.partials) : nullptr;
    args.p[0].flags = meets ? c.flag_words + first_flag : nullptr;
    remember(c, pl, 1);
    return launch(c, pl, &args);
}

// Runs plain products, none of which needs another's result: those that stream their weights, then the
// others in one launch or one after the other.
int run_products(Call &c, Product *all, int count)
{
    Product *xs[kFfnMaxProducts];
    int n = 0, rc;
    for (int i = 0; i < count; ++i)
        if (all[i].M > 0 && all[i].N > 0) {
            if (streams_back(c, all[i])) {
                if ((rc = run_stream_back(c, all[i])) != FFN_OK)
                    return rc;
                continue;
            }
            xs[n++] = &all[i];
        }
    const Together *group = nullptr;
    if (n > 1 && options.v[FFN_OPT_TOGETHER] != 2) {
        // those with the longest tiles first, so that the last tiles are short ones
        std::stable_sort(xs, xs + n, [](const Product *a, const Product *b) { return k_blocks_of(*a) > k_blocks_of(*b); });
        Plan alone[kFfnMaxProducts];
        for (int i = 0; i < n; ++i)
            if ((rc = find_plan(c.dev, *xs[i], &alone[i])) != FFN_OK)
                return rc;
        if ((rc = find_together(c.dev, xs, alone, n, &group)) != FFN_OK)
            return rc;
    }
    if (!group || !group->yes) {
        for (int i = 0; i < n; ++i)
            if ((rc = run_product(c, *xs[i])) != FFN_OK)
                return rc;
        return FFN_OK;
    }
    for (int i = 0; i < n; ++i)
        prepare(c, *xs[i], group->plan[i]);
    if (c.measuring())
        return FFN_OK;
    FfnArgs<kFfnMaxProducts> args;
    std::memset(static_cast<void *>(&args), 0, sizeof(args));
    for (int i = 0; i < kFfnMaxProducts; ++i) {
        if (i < n && (rc = describe(*xs[i], group->plan[i], args.maps[i], args.p[i])) != FFN_OK)
            return rc;
        args.first[i + 1] = args.first[i] + args.p[i].num_tiles;
        args.p[0].watchdog_ns = std::max(args.p[0].watchdog_ns, args.p[i].watchdog_ns);
    }
    remember(c, group->plan[0], n);
    return launch(c, group->plan[0], &args);
}

// --------------------------------------------------------------- checks
bool bad_dim(int64_t n) { return n < 0 || n > kMaxDim; }

// A matrix that must be there (if it has elements), with rows that do not overlap.
bool bad_matrix(const ffn_matrix &m, int64_t rows, int64_t cols, int esize = 2)
{
    if (rows == 0 || cols == 0)
        return false;
    return !m.data || !aligned(m.data, (uintptr_t)esize) ||
           (rows > 1 && (m.ld < cols || m.ld > kMaxPitch || rows > kMaxElements / m.ld));
}

int check_quantized(const ffn_quantized &q, int64_t rows, int64_t cols, int64_t step)
{
    if (rows == 0 || cols == 0)
        return FFN_OK;
    if (!q.codes || !q.scales || q.ld < cols || q.ld > kMaxPitch || rows > kMaxElements / q.ld)
        return FFN_ERR_INVALID_ARG;
    return aligned(q.codes, 16) && q.ld % step == 0 && aligned(q.scales, 4) ? FFN_OK : FFN_ERR_ALIGNMENT;
}

bool bad_act(int32_t a) { return a < FFN_ACT_NONE || a > FFN_ACT_GELU_TANH; }
bool bad_type(int32_t t) { return t != FFN_BF16 && t != FFN_FP32; }

Span span(const ffn_matrix &m, int64_t rows, int64_t cols, int esize = 2) { return {m.data, m.ld * esize, cols * esize, rows}; }

// Results lie apart from what is read and from each other.
bool apart(std::initializer_list<Span> writes, std::initializer_list<Span> reads)
{
    for (const Span *w = writes.begin(); w != writes.end(); ++w) {
        for (const Span *o = w + 1; o != writes.end(); ++o)
            if (touch(*w, *o))
                return false;
        for (const Span &r : reads) {
            if (r.same_allowed && w == writes.begin() && r.p == w->p && r.width == w->width &&
                (r.ld == w->ld || r.rows == 1))
                continue;
            if (touch(*w, r))
                return false;
        }
    }
    return true;
}

// Checks the workspace and runs `body` to measure it, then in earnest.
template <typename F>
int run_call(F body, void *workspace, int64_t size, void *stream)
{
    Call c;
    int rc = current_device(&c.dev);
    if (rc != FFN_OK)
        return rc;
    if ((rc = body(c)) != FFN_OK)
        return rc;
    const size_t need = c.bytes();
    if (need && (!workspace || size < (int64_t)need))
        return FFN_ERR_WORKSPACE;
    if (need && !aligned(workspace, kWorkAlign))
        return FFN_ERR_ALIGNMENT;
    Call run;
    run.dev = c.dev;
    run.stream = static_cast<cudaStream_t>(stream);
    static uint8_t none;  // never used: such a call takes nothing
    run.base = need ? static_cast<uint8_t *>(workspace) : &none;
    run.jobs = c.jobs;
    for (int i = 0; i < run.jobs.n; ++i) {
        FfnPackJob &j = run.jobs.job[i];
        j.dst = reinterpret_cast<uint16_t *>(run.base + c.used + reinterpret_cast<size_t>(j.dst));
    }
    run.flag_words = reinterpret_cast<uint32_t *>(run.base + c.used + c.copies);
    run.partials = need - c.partials;
    run.jobs.flags = c.flags ? run.flag_words : nullptr;
    run.jobs.num_flags = (int32_t)c.flags;
    if ((c.jobs.n || c.flags) &&
        (rc = from_cuda((cudaError_t)launch_ffn_pack(run.jobs, run.dev.sms, run.stream))) != FFN_OK)
        return rc;
    return body(run);
}

template <typename F>
int measure_call(F body, int64_t *bytes)
{
    Call c;
    int rc = current_device(&c.dev);
    if (rc != FFN_OK)
        return rc;
    if ((rc = body(c)) == FFN_OK)
        *bytes = (int64_t)c.bytes();
    return rc;
}

// --------------------------------------------------------------- linear
int check_linear(const ffn_linear_args &a)
{
    if (bad_dim(a.M) || bad_dim(a.N) || bad_dim(a.K) || bad_act(a.activation) || bad_type(a.y_type) ||
        (a.bias && bad_type(a.bias_type)))
        return FFN_ERR_INVALID_ARG;
    const int esize = a.y_type == FFN_FP32 ? 4 : 2;
    const bool out = a.M > 0 && a.N > 0;
    if (bad_matrix(a.y, a.M, a.N, esize) || (out && (bad_matrix(a.x, a.M, a.K) || bad_matrix(a.weight, a.N, a.K))) ||
        (a.residual.data && bad_matrix(a.residual, a.M, a.N)) || (a.z.data && bad_matrix(a.z, a.M, a.N)))
        return FFN_ERR_INVALID_ARG;
    const int bsize = a.bias_type == FFN_FP32 ? 4 : 2;
    if (a.bias && !aligned(a.bias, (uintptr_t)bsize))
        return FFN_ERR_ALIGNMENT;
    Span residual = span(a.residual, a.M, a.N);
    residual.same_allowed = true;
    if (!apart({span(a.y, a.M, a.N, esize), span(a.z, a.M, a.N)},
               {span(a.x, a.M, a.K), span(a.weight, a.N, a.K), residual, {a.bias, 0, a.N * bsize, 1}}))
        return FFN_ERR_INVALID_ARG;
    return FFN_OK;
}

int body_linear(Call &c, const ffn_linear_args &a)
{
    Product x;
    x.M = a.M, x.N = a.N, x.K = a.K;
    x.A[0] = {a.x.data, a.x.ld};
    x.B[0] = {a.weight.data, a.weight.ld};
    x.p.act = a.activation;
    x.p.bias = a.bias;
    x.p.bias_fp32 = a.bias_type == FFN_FP32;
    x.p.aux[0] = aux_of(a.residual);
    x.p.save = a.z.data ? 1 : 0;
    x.D[0] = a.y;
    x.D[1] = a.z;
    x.fp32 = a.y_type == FFN_FP32;
    return run_product(c, x);
}

int check_linear_backward(const ffn_linear_backward_args &a)
{
    if (bad_dim(a.M) || bad_dim(a.N) || bad_dim(a.K) || bad_act(a.activation) || bad_type(a.dweight_type))
        return FFN_ERR_INVALID_ARG;
    const int wsize = a.dweight_type == FFN_FP32 ? 4 : 2;
    if (bad_matrix(a.dy, a.M, a.N) || (a.activation && bad_matrix(a.z, a.M, a.N)) ||
        (a.dx.data && (bad_matrix(a.dx, a.M, a.K) || bad_matrix(a.weight, a.N, a.K))) ||
        (a.dweight.data && (bad_matrix(a.dweight, a.N, a.K, wsize) || bad_matrix(a.x, a.M, a.K))) ||
        !aligned(a.dbias, 4))
        return FFN_ERR_INVALID_ARG;
    if (!apart({span(a.dx, a.M, a.K), span(a.dweight, a.N, a.K, wsize), {a.dbias, 0, a.N * 4, 1}},
               {span(a.dy, a.M, a.N), span(a.x, a.M, a.K), span(a.weight, a.N, a.K), span(a.z, a.M, a.N)}))
        return FFN_ERR_INVALID_ARG;
    return FFN_OK;
}

int body_linear_backward(Call &c, const ffn_linear_backward_args &a)
{
    ffn_matrix dz = a.dy;
    const bool products = a.dx.data || a.dweight.data;
    if (a.N > 0 && ((a.activation && products && a.M > 0) || a.dbias)) {
        FfnSlopeParams s = {};
        s.dy = static_cast<const uint16_t *>(a.dy.data);
        s.lddy = a.dy.ld;
        s.R = (int32_t)a.M, s.C = (int32_t)a.N;
        s.vec = aligned(a.dy.data, 16) && (a.dy.ld % 8 == 0 || a.M <= 1);
        s.act = a.activation;
        if (a.activation) {
            s.z = static_cast<const uint16_t *>(a.z.data);
            s.ldz = a.z.ld;
            s.vec = s.vec && aligned(a.z.data, 16) && (a.z.ld % 8 == 0 || a.M <= 1);
            dz.ld = padded(a.N);
            dz.data = c.take((size_t)(a.M * dz.ld) * 2);
            s.dz = static_cast<uint16_t *>(dz.data);
            s.lddz = dz.ld;
        }
        if (a.dbias) {
            s.dbias = a.dbias;
            const int slices = ffn_slope_slices(a.M, a.N, c.dev.sms);
            s.partials = static_cast<float *>(c.take((size_t)slices * (size_t)a.N * sizeof(float)));
        }
        if (!c.measuring()) {
            const int rc = from_cuda((cudaError_t)launch_ffn_slope(s, c.dev.sms, c.stream));
            if (rc != FFN_OK)
                return rc;
        }
    }
    Product xs[2];
    int n = 0;
    if (a.dx.data) {
        Product &x = xs[n++];
        x.M = a.M, x.N = a.K, x.K = a.N;
        x.b_mn = true;
        x.own_a = a.activation != FFN_ACT_NONE;
        x.A[0] = {dz.data, dz.ld};
        x.B[0] = {a.weight.data, a.weight.ld};
        x.D[0] = a.dx;
    }
    if (a.dweight.data) {
        Product &x = xs[n++];
        x.M = a.N, x.N = a.K, x.K = a.M;
        x.a_mn = x.b_mn = true;
        x.own_a = a.activation != FFN_ACT_NONE;
        x.A[0] = {dz.data, dz.ld};
        x.B[0] = {a.x.data, a.x.ld};
        x.D[0] = a.dweight;
        x.fp32 = a.dweight_type == FFN_FP32;
    }
    return run_products(c, xs, n);
}

// --------------------------------------------------------------- gated
int check_gated(const ffn_gated_args &a)
{
    if (bad_dim(a.M) || bad_dim(a.F) || bad_dim(a.C) || bad_act(a.activation))
        return FFN_ERR_INVALID_ARG;
    const bool bf16 = a.g.data || a.u.data, bits8 = a.qg.codes || a.qu.codes;
    if (bad_matrix(a.h, a.M, a.F) || bad_matrix(a.x, a.M, a.C) || bad_matrix(a.w_gate, a.F, a.C) ||
        bad_matrix(a.w_up, a.F, a.C) || (bf16 && bits8) ||
        (bf16 && (!a.g.data || !a.u.data || bad_matrix(a.g, a.M, a.F) || bad_matrix(a.u, a.M, a.F))))
        return FFN_ERR_INVALID_ARG;
    if (bits8) {
        for (const ffn_quantized *q : {&a.qg, &a.qu}) {
            const int rc = check_quantized(*q, a.M, a.F, 128);
            if (rc != FFN_OK)
                return rc;
        }
    }
    const int64_t words = ceil_div(a.F, 512) * a.M * 4;
    // whole rows of codes: bytes behind a row's last code may be written
    if (!apart({span(a.h, a.M, a.F), span(a.g, a.M, a.F), span(a.u, a.M, a.F), {a.qg.codes, a.qg.ld, a.qg.ld, a.M},
                {a.qu.codes, a.qu.ld, a.qu.ld, a.M}, {a.qg.scales, 0, words, 1}, {a.qu.scales, 0, words, 1}},
               {span(a.x, a.M, a.C), span(a.w_gate, a.F, a.C), span(a.w_up, a.F, a.C)}))
        return FFN_ERR_INVALID_ARG;
    return FFN_OK;
}

int body_gated(Call &c, const ffn_gated_args &a)
{
    Product x;
    x.epilogue = kFfnGated;
    x.form = kDual;
    x.M = a.M, x.N = a.F, x.K = a.C;
    x.A[0] = {a.x.data, a.x.ld};
    x.B[0] = {a.w_gate.data, a.w_gate.ld};
    x.B[1] = {a.w_up.data, a.w_up.ld};
    x.p.act = a.activation;
    x.p.save = a.g.data ? 1 : a.qg.codes ? 2 : 0;
    if (x.p.save == 2) {
        // a thread sees a whole block of a row's sums only where rows are on the row side and a
        // tile's sums lie in one CTA
        x.no_split = x.not_transposed = true;
        x.p.codes[0] = static_cast<uint8_t *>(a.qg.codes);
        x.p.codes[1] = static_cast<uint8_t *>(a.qu.codes);
        x.p.scales[0] = static_cast<uint8_t *>(a.qg.scales);
        x.p.scales[1] = static_cast<uint8_t *>(a.qu.scales);
        x.p.ldq[0] = a.qg.ld;
        x.p.ldq[1] = a.qu.ld;
    }
    x.D[0] = a.h;
    x.D[1] = a.g;
    x.D[2] = a.u;
    return run_product(c, x);
}

int check_gated_backward(const ffn_gated_backward_args &a)
{
    if (bad_dim(a.M) || bad_dim(a.F) || bad_dim(a.C) || bad_dim(a.N) || bad_act(a.activation) ||
        bad_type(a.dweight_type))
        return FFN_ERR_INVALID_ARG;
    const int wsize = a.dweight_type == FFN_FP32 ? 4 : 2;
    const bool bf16 = a.g.data || a.u.data, bits8 = a.qg.codes || a.qu.codes;
    if (bf16 && bits8)
        return FFN_ERR_INVALID_ARG;
    if (bits8) {
        for (const ffn_quantized *q : {&a.qg, &a.qu}) {
            const int rc = check_quantized(*q, a.M, a.F, 16);
            if (rc != FFN_OK)
                return rc;
        }
    } else if (bad_matrix(a.g, a.M, a.F) || bad_matrix(a.u, a.M, a.F)) {
        return FFN_ERR_INVALID_ARG;
    }
    if (bad_matrix(a.dy, a.M, a.N) || bad_matrix(a.w_down, a.N, a.F) || !a.dw_gate.data != !a.dw_up.data ||
        (a.dx.data &&
         (bad_matrix(a.dx, a.M, a.C) || bad_matrix(a.w_gate, a.F, a.C) || bad_matrix(a.w_up, a.F, a.C))) ||
        (a.dw_gate.data && (bad_matrix(a.dw_gate, a.F, a.C, wsize) || bad_matrix(a.dw_up, a.F, a.C, wsize) ||
                            bad_matrix(a.x, a.M, a.C))) ||
        (a.dw_down.data && bad_matrix(a.dw_down, a.N, a.F, wsize)))
        return FFN_ERR_INVALID_ARG;
    const int64_t words = ceil_div(a.F, 512) * a.M * 4;
    if (!apart({span(a.dx, a.M, a.C), span(a.dw_gate, a.F, a.C, wsize), span(a.dw_up, a.F, a.C, wsize),
                span(a.dw_down, a.N, a.F, wsize)},
               {span(a.dy, a.M, a.N), span(a.x, a.M, a.C), span(a.g, a.M, a.F), span(a.u, a.M, a.F),
                {a.qg.codes, a.qg.ld, a.F, a.M}, {a.qu.codes, a.qu.ld, a.F, a.M}, {a.qg.scales, 0, words, 1},
                {a.qu.scales, 0, words, 1}, span(a.w_gate, a.F, a.C), span(a.w_up, a.F, a.C), span(a.w_down, a.N, a.F)}))
        return FFN_ERR_INVALID_ARG;
    return FFN_OK;
}

int body_gated_backward(Call &c, const ffn_gated_backward_args &a)
{
    ffn_matrix t[3];  // dg, du, h
    for (ffn_matrix &m : t) {
        m.ld = padded(a.F);
        m.data = c.take((size_t)(a.M * m.ld) * 2);
    }
    int rc;
    {
        Product x;
        x.epilogue = kFfnGrad;
        x.M = a.M, x.N = a.F, x.K = a.N;
        x.b_mn = true;
        x.A[0] = {a.dy.data, a.dy.ld};
        x.B[0] = {a.w_down.data, a.w_down.ld};
        x.p.act = a.activation;
        const bool bits8 = a.qg.codes != nullptr;
        x.p.aux[0] = bits8 ? aux_of(a.qg) : aux_of(a.g);
        x.p.aux[1] = bits8 ? aux_of(a.qu) : aux_of(a.u);
        for (int i = 0; i < 3; ++i)
            x.D[i] = t[i];
        if ((rc = run_product(c, x)) != FFN_OK)
            return rc;
    }
    Product xs[3];
    int n = 0;
    if (a.dx.data) {
        Product &x = xs[n++];
        x.form = kSum;
        x.M = a.M, x.N = a.C, x.K = a.F;
        x.b_mn = x.own_a = true;
        x.A[0] = {t[0].data, t[0].ld};
        x.A[1] = {t[1].data, t[1].ld};
        x.B[0] = {a.w_gate.data, a.w_gate.ld};
        x.B[1] = {a.w_up.data, a.w_up.ld};
        x.D[0] = a.dx;
    }
    if (a.dw_gate.data) {
        Product &x = xs[n++];
        x.form = kStack;
        x.M = a.F, x.N = a.C, x.K = a.M;
        x.a_mn = x.b_mn = x.own_a = true;
        x.A[0] = {t[0].data, t[0].ld};
        x.A[1] = {t[1].data, t[1].ld};
        x.B[0] = {a.x.data, a.x.ld};
        x.D[0] = a.dw_gate;
        x.D[1] = a.dw_up;
        x.fp32 = a.dweight_type == FFN_FP32;
    }
    if (a.dw_down.data) {
        Product &x = xs[n++];
        x.M = a.N, x.N = a.F, x.K = a.M;
        x.a_mn = x.b_mn = x.own_b = true;
        x.A[0] = {a.dy.data, a.dy.ld};
        x.B[0] = {t[2].data, t[2].ld};
        x.D[0] = a.dw_down;
        x.fp32 = a.dweight_type == FFN_FP32;
    }
    return run_products(c, xs, n);
}

}  // namespace

extern "C" {

FFN_API const char *ffn_strerror(int status)
{
    switch (status) {
    case FFN_OK: return "ok";
    case FFN_ERR_INVALID_ARG: return "invalid argument";
    case FFN_ERR_ALIGNMENT: return "alignment of a pointer or a pitch";
    case FFN_ERR_WORKSPACE: return "the workspace is missing or too small";
    case FFN_ERR_CUDA: return "a CUDA runtime call failed";
    case FFN_ERR_TENSORMAP: return "TMA tensor-map encoding failed";
    case FFN_ERR_DEVICE_TIMEOUT: return "device watchdog: a barrier wait ran out and the kernel returned early";
    case FFN_ERR_UNSUPPORTED: return "unsupported device, size or option combination";
    default: return "unknown status";
    }
}

FFN_API const char *ffn_version(void) { return "ffn_ops 1.0 sm_103a"; }

FFN_API int ffn_set_option(int key, int64_t value)
{
    bool ok = false;
    switch (key) {
    case FFN_OPT_CTA_GROUP: ok = value >= 0 && value <= 2; break;
    case FFN_OPT_TRANSPOSED: ok = value >= 0 && value <= 2; break;
    case FFN_OPT_WIDTH: ok = value >= 0 && value <= kFfnMaxWidth && value % 16 == 0; break;
    case FFN_OPT_SPLIT: ok = value >= 0 && value <= 2; break;
    // far above what any load takes to land: the CTAs of a pair that give up at different
    // times count on each other's having landed
    case FFN_OPT_WATCHDOG_NS: ok = value >= 100000 && value <= 60000000000LL; break;
    case FFN_OPT_FAULT_SKIP_LOAD: ok = value >= -1 && value <= 0x7FFFFFFF; break;
    case FFN_OPT_RASTER_GROUP: ok = value >= 0 && value <= 1024; break;
    case FFN_OPT_TOGETHER: ok = value >= 0 && value <= 2; break;
    case FFN_OPT_STREAM: ok = value >= 0 && value <= 2; break;
    case FFN_OPT_REPACK: ok = value >= 0 && value <= 2; break;
    default: break;
    }
    if (!ok)
        return FFN_ERR_INVALID_ARG;
    options.v[key] = value;
    return FFN_OK;
}

FFN_API int ffn_get_option(int key, int64_t *value)
{
    if (!value || key < 1 || key >= kNumOptions)
        return FFN_ERR_INVALID_ARG;
    *value = options.v[key];
    return FFN_OK;
}

FFN_API int ffn_plan_info(ffn_plan_info_t *info)
{
    if (!info || !have_last_plan)
        return FFN_ERR_INVALID_ARG;
    std::memset(info, 0, sizeof(*info));
    info->tiles = last_plan.tiles;
    info->k_blocks = last_plan.k_blocks;
    info->grid_ctas = last_plan.grid;
    info->cta_group = last_plan.cta_group;
    info->transposed = last_plan.transposed ? 1 : 0;
    info->width = last_plan.width;
    info->stages = last_plan.stages;
    info->split_tiles = (int32_t)last_plan.sk_tiles;
    info->cluster = last_plan.cluster;
    info->packed = last_packed;
    info->products = last_products;
    return FFN_OK;
}

#define FFN_ENTRY(name)                                                                                               \
    FFN_API int ffn_##name##_workspace(const ffn_##name##_args *args, int64_t *bytes)                                 \
    {                                                                                                                 \
        if (!args || !bytes)                                                                                          \
            return FFN_ERR_INVALID_ARG;                                                                               \
        *bytes = 0;                                                                                                   \
        const int rc = check_##name(*args);                                                                           \
        return rc != FFN_OK ? rc : measure_call([args](Call &c) { return body_##name(c, *args); }, bytes);            \
    }                                                                                                                 \
    FFN_API int ffn_##name(const ffn_##name##_args *args, void *workspace, int64_t workspace_bytes, void *stream)     \
    {                                                                                                                 \
        if (!args)                                                                                                    \
            return FFN_ERR_INVALID_ARG;                                                                               \
        const int rc = check_##name(*args);                                                                           \
        return rc != FFN_OK                                                                                           \
                   ? rc                                                                                               \
                   : run_call([args](Call &c) { return body_##name(c, *args); }, workspace, workspace_bytes, stream); \
    }

FFN_ENTRY(linear)
FFN_ENTRY(linear_backward)
FFN_ENTRY(gated)
FFN_ENTRY(gated_backward)

FFN_API int ffn_device_status(uint32_t *detail)
{
    if (detail)
        *detail = 0;
    uint32_t *const at = ffn_status_word();
    if (!at)
        return FFN_ERR_CUDA;
    // the whole device: a launch may run again on any stream, from a graph that captured it
    uint32_t word = 0;
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(&word, at, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess)
        return from_cuda(cudaErrorUnknown);
    if (word == 0)
        return FFN_OK;
    if (detail)
        *detail = word;
    const uint32_t none = 0;
    if (cudaMemcpy(at, &none, sizeof(none), cudaMemcpyHostToDevice) != cudaSuccess)
        return from_cuda(cudaErrorUnknown);
    return FFN_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
