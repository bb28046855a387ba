// Host side of the C ABI declared in include/fp8_ops.h: argument checks, the
// product's handle and plans, TMA tensor maps and launches.
#include "fp8_ops.h"

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <new>

#include "fp8_kernels.h"
#include "fp8_overlap.h"

using namespace wstma;

namespace {

constexpr int64_t kMaxDim = 0x7FFFFFFFLL;
constexpr int64_t kMaxRows = kMaxDim - 1023;  // a tile past the last row still has a 32-bit index
constexpr int64_t kMaxPitch = int64_t(1) << 38;
constexpr int kNumOptions = 8;
constexpr int kPlans = 64;          // plans a handle remembers
constexpr int kMaxCtas = 1024;      // bounds the workspace of split tiles
constexpr int64_t kMinSplitBlocks = 4;  // k-blocks per cluster below which tiles are not split further

struct Plan {
    bool valid = false;
    uint64_t used = 0;  // for replacing the plan used longest ago
    int64_t M = 0, N = 0, K = 0, lda = 0, ldb = 0, ldd = 0;
    int out_type = 0;
    int cta_group = 1, width = 32, stages = 2, grid = 0, cluster = 1;
    bool transposed = false;
    int64_t tiles = 0, row_tiles = 0, col_tiles = 0, k_blocks = 0, sk_tiles = 0;
    size_t smem = 0;
    int regs = 0;
    const void *fn = nullptr;
    // tensor maps and the pointers they were made for
    const void *mA = nullptr, *mB = nullptr;
    void *mD = nullptr;
    bool maps = false, d_tma = false;
    CUtensorMap tmR, tmC, tmD;
};

}  // namespace

struct fp8_gemm {
    int device = 0;
    int num_sms = 0;
    size_t max_smem = 0;
    int max_pairs = 0;  // SM pairs that are resident at once
    uint32_t *d_err = nullptr;
    void *workspace = nullptr;  // of split tiles, allocated at its final size by the first fp8_gemm_run that needs it
    int64_t opt[kNumOptions] = {0, 0, 0, 0, 1, 2000000000, -1, 0};
    Plan plans[kPlans];
    Plan *plan = nullptr;
    uint64_t clock = 0;
};

namespace {

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

int encode_2d(CUtensorMap *m, CUtensorMapDataType type, const void *ptr, uint64_t cols, uint64_t rows,
              uint64_t row_bytes, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    auto fn = encode_fn();
    if (!fn)
        return FP8_ERR_TENSORMAP;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(m, type, 2, const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP8_OK : FP8_ERR_TENSORMAP;
}

// Makes `device` current and puts the caller's device back at the end.
class DeviceGuard {
public:
    explicit DeviceGuard(int device)
    {
        if (cudaGetDevice(&before_) != cudaSuccess) {
            cudaGetLastError();
            return;
        }
        ok_ = before_ == device || cudaSetDevice(device) == cudaSuccess;
        changed_ = ok_ && before_ != device;
        if (!ok_)
            cudaGetLastError();
    }
    ~DeviceGuard()
    {
        if (changed_)
            cudaSetDevice(before_);
    }
    bool ok() const { return ok_; }

private:
    int before_ = 0;
    bool ok_ = false, changed_ = false;
};

// Device memory set to zero, also while a stream of this thread is capturing
// (neither the allocation nor the clear belongs to the graph).
int alloc_zeroed(void **out, size_t bytes)
{
    *out = nullptr;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    void *p = nullptr;
    cudaStream_t st = nullptr;
    bool ok = cudaMalloc(&p, bytes) == cudaSuccess &&
              cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking) == cudaSuccess &&
              cudaMemsetAsync(p, 0, bytes, st) == cudaSuccess && cudaStreamSynchronize(st) == cudaSuccess;
    if (st)
        cudaStreamDestroy(st);
    if (!ok) {
        cudaGetLastError();
        if (p)
            cudaFree(p);
    }
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (!ok)
        return FP8_ERR_CUDA;
    *out = p;
    return FP8_OK;
}

// Number of SMs of the current device, looked up once per device.
int current_sms(int *sms)
{
    static int known[64];
    static std::mutex lock;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return FP8_ERR_CUDA;
    }
    std::lock_guard<std::mutex> hold(lock);
    if (dev >= 64 || known[dev] == 0) {
        int n = 0, major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
            cudaGetLastError();
            return FP8_ERR_CUDA;
        }
        if (major != 10 || minor != 3)
            return FP8_ERR_UNSUPPORTED;
        *sms = n;
        if (dev < 64)
            known[dev] = n;
        return FP8_OK;
    }
    *sms = known[dev];
    return FP8_OK;
}

int from_cuda(cudaError_t e)
{
    if (e == cudaSuccess)
        return FP8_OK;
    cudaGetLastError();
    return FP8_ERR_CUDA;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool bad_pitch(int64_t ld, int64_t width) { return ld < width || ld > kMaxPitch; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// --------------------------------------------------------------- plans of the product
struct Tiling {
    bool transposed;
    int cta_group, width;
    // found by tiling_cost()
    int64_t clusters = 0;  // SM pairs, or CTAs, of the grid
    int64_t sk_tiles = 0;
    int cluster = 1;       // CTAs that share a tile in a cluster
};

// An fp32 D of a long sum is accumulated in segments.
bool long_sums(const Plan &pl) { return pl.out_type == FP8_FP32 && pl.k_blocks > kFp8Segment; }

int ring_stages(const fp8_gemm *h, int cta_group, int width)
{
    int S = kFp8MaxStages;
    while (S > 2 && fp8_smem_bytes(cta_group, width, S) > h->max_smem)
        S -= 2;
    return S;
}

cudaError_t configure(const fp8_gemm *h, const void *fn)
{
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)h->max_smem);
}

// How many clusters of c CTAs of a one-SM kernel are resident at once.
int resident_clusters(const fp8_gemm *h, const Plan &pl, const Tiling &t, int c)
{
    const void *fn = fp8_gemm_kernel_fn(1, t.transposed, long_sums(pl));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int n = 0;
    cfg.gridDim = dim3((unsigned)c, 1, 1);
    cfg.blockDim = dim3(kFp8Threads, 1, 1);
    cfg.dynamicSmemBytes = fp8_smem_bytes(1, t.width, ring_stages(h, 1, t.width));
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (configure(h, fn) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

// Estimated time of a tiling, in clocks of an SM (1.9 GHz), without what every
// launch costs: the stages (k-blocks) of the longest chain, each the longest of
// its MMAs (8192 e4m3 multiply-adds a clock and SM), its loads (56 bytes a clock
// and SM with all SMs loading) and what the MMA issuer needs (400 clocks); or the
// operands' time in HBM, if longer; then the epilogue and the exchange between a
// split tile's pieces.  The exchanges' costs are fitted to measurements: through a
// cluster 8x700x1500 loses 0.5 us by saving 8 of 12 stages; through global memory
// 1x8192x8192 spends 4 us, 1000x1000x8000 in four pieces of 224 columns 14 us.  Where all
// ranks of a cluster fetch at once, its size costs little (with the other formula for
// these too 128x1024x4096 takes 9.3 us, not 8.5, 934x174x5658 10.7, not 9.6).
// Fills in how the tiles are shared out.
double tiling_cost(const fp8_gemm *h, const Plan &pl, Tiling &t)
{
    const int64_t rows = t.transposed ? pl.N : pl.M, cols = t.transposed ? pl.M : pl.N;
    const int64_t KB = pl.k_blocks;
    const int64_t tiles = ceil_div(rows, kFp8RowsPerCta * t.cta_group) * ceil_div(cols, t.width);
    const int64_t split = h->opt[FP8_GEMM_OPT_SPLIT];
    const int64_t most = t.cta_group == 2 ? h->max_pairs : h->num_sms;
    const double stage = std::max({2.0 * t.width, 400.0, (double)fp8_stage_bytes(t.cta_group, t.width) / 56.0});
    const double hbm = (double)(pl.M + pl.N) * (double)pl.K / 3500.0;
    const double epilogue = 8.0 * t.width;

    t.clusters = std::min(tiles, most);
    t.sk_tiles = 0;
    t.cluster = 1;
    double best = std::max((double)(ceil_div(tiles, t.clusters) * KB) * stage, hbm) + epilogue;
    if (split == 1 && t.cta_group == 1) {
        // each tile shared by a cluster of CTAs
        const int64_t c = std::min<int64_t>({most / tiles, 8, KB});
        if (c >= 2) {
            // rank 0 fetches the others' pieces in turn, or all ranks fetch at once
            const double exchange = c >= kFp8SpreadFrom && !long_sums(pl)
                                        ? 6500.0 + 12.0 * t.width
                                        : 4500.0 + (400.0 + 8.0 * t.width) * (double)(c - 1);
            const double cost = std::max((double)ceil_div(KB, c) * stage, hbm) + epilogue + exchange;
            if (cost < best) {
                best = cost;
                t.clusters = tiles * c;
                t.sk_tiles = tiles;
                t.cluster = (int)c;
            }
        }
    }
    if (split) {
        // the last, partial wave of tiles (or all, if they do not fill one) shared by all clusters
        const int64_t sk = tiles % most;
        const int64_t C = tiles > most ? most : std::max(tiles, std::min(most, tiles * KB / kMinSplitBlocks));
        if (sk && C > sk) {
            // behind whole tiles the exchange is out of sight: the split tiles come first
            const int64_t whole = (tiles - sk) / C;
            const double exchange = whole ? 3000.0 : 7500.0 + (700.0 + 12.0 * t.width) * (double)C / (double)sk;
            const double cost =
                std::max((double)(whole * KB + ceil_div(sk * KB, C)) * stage, hbm) + epilogue + exchange;
            if (cost < best) {
                best = cost;
                t.clusters = C;
                t.sk_tiles = sk;
                t.cluster = 1;
            }
        }
    }
    return best;
}

int make_plan(fp8_gemm_t h, Plan &pl)
{
    const int64_t want_cg = h->opt[FP8_GEMM_OPT_CTA_GROUP], want_tr = h->opt[FP8_GEMM_OPT_TRANSPOSED];
    const int64_t want_w = h->opt[FP8_GEMM_OPT_WIDTH];
    Tiling best = {false, 0, 0};
    double best_cost = 0.0;
    for (int cg = 1; cg <= 2; ++cg)
        for (int tr = 0; tr <= 1; ++tr)
            for (int wd = 16; wd <= kFp8MaxWidth; wd += 16) {
                if ((want_cg && cg != want_cg) || (want_tr && tr + 1 != want_tr) || (want_w && wd != want_w))
                    continue;
                // chunks of 32 columns: a narrower tile must be the only one
                const int64_t cols = tr ? pl.M : pl.N;
                if (wd % 32 != 0 && (cg == 2 || wd < cols))
                    continue;
                if (wd > kFp8MaxLongWidth && long_sums(pl))
                    continue;
                Tiling t = {tr != 0, cg, wd};
                const double cost = tiling_cost(h, pl, t);
                if (best.cta_group == 0 || cost < best_cost)
                    best = t, best_cost = cost;
            }
    if (best.cta_group == 0)
        return FP8_ERR_UNSUPPORTED;
    const int64_t rows = best.transposed ? pl.N : pl.M, cols = best.transposed ? pl.M : pl.N;
    pl.transposed = best.transposed;
    pl.cta_group = best.cta_group;
    pl.width = best.width;
    pl.row_tiles = ceil_div(rows, kFp8RowsPerCta * best.cta_group);
    pl.col_tiles = ceil_div(cols, best.width);
    pl.tiles = pl.row_tiles * pl.col_tiles;
    if (pl.tiles > kMaxDim)
        return FP8_ERR_UNSUPPORTED;
    // Rank 0 of a cluster waits for the others, so all clusters must be resident:
    // the largest size that the device can place so often.
    if (best.cluster > 1) {
        while (best.cluster > 1 && resident_clusters(h, pl, best, best.cluster) < pl.tiles)
            --best.cluster;
        best.clusters = pl.tiles * best.cluster;
        best.sk_tiles = best.cluster > 1 ? pl.tiles : 0;
    }
    pl.sk_tiles = best.sk_tiles;
    pl.cluster = best.cluster;
    pl.grid = (int)(best.clusters * best.cta_group);
    pl.stages = ring_stages(h, best.cta_group, best.width);
    pl.smem = fp8_smem_bytes(best.cta_group, best.width, pl.stages);
    pl.fn = fp8_gemm_kernel_fn(best.cta_group, best.transposed, long_sums(pl));
    cudaFuncAttributes a;
    if (configure(h, pl.fn) != cudaSuccess || cudaFuncGetAttributes(&a, pl.fn) != cudaSuccess)
        return from_cuda(cudaErrorUnknown);
    pl.regs = a.numRegs;
    return FP8_OK;
}

// A CTA's part of the workspace of split tiles: all partials come first, then all flags.
constexpr size_t kPartialBytes = kFp8PartialFloats * sizeof(float);
constexpr size_t kFlagBytes = kFp8EpiWarps * sizeof(uint32_t);

size_t workspace_bytes(const Plan &pl)
{
    return pl.sk_tiles && pl.cluster == 1 ? (size_t)pl.grid * (kPartialBytes + kFlagBytes) : 0;
}

}  // namespace

extern "C" {

FP8_API const char *fp8_strerror(int status)
{
    switch (status) {
    case FP8_OK: return "ok";
    case FP8_ERR_INVALID_ARG: return "invalid argument";
    case FP8_ERR_ALIGNMENT: return "alignment: codes need 16-byte aligned bases and row pitches";
    case FP8_ERR_NOT_PLANNED: return "not planned: call fp8_gemm_plan first";
    case FP8_ERR_CUDA: return "a CUDA runtime call failed";
    case FP8_ERR_TENSORMAP: return "TMA tensor-map encoding failed";
    case FP8_ERR_DEVICE_TIMEOUT: return "device watchdog: a barrier wait ran out and the kernel returned early";
    case FP8_ERR_UNSUPPORTED: return "unsupported device, size or option combination";
    default: return "unknown status";
    }
}

FP8_API const char *fp8_version(void) { return "fp8_ops 1.0 sm_103a"; }

FP8_API int fp8_gemm_check_problem(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldd,
                                   int out_type)
{
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return FP8_ERR_INVALID_ARG;
    if (out_type != FP8_BF16 && out_type != FP8_FP32)
        return FP8_ERR_INVALID_ARG;
    if (bad_pitch(lda, K) || bad_pitch(ldb, K) || bad_pitch(ldd, N))
        return FP8_ERR_INVALID_ARG;
    if (lda % 16 != 0 || ldb % 16 != 0)
        return FP8_ERR_ALIGNMENT;
    if (M > kMaxRows || N > kMaxRows)
        return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

FP8_API int fp8_gemm_create(int device, fp8_gemm_t *out)
{
    if (!out)
        return FP8_ERR_INVALID_ARG;
    *out = nullptr;
    int dev = device;
    if (dev < 0 && cudaGetDevice(&dev) != cudaSuccess)
        return from_cuda(cudaErrorUnknown);
    int count = 0;
    if (cudaGetDeviceCount(&count) != cudaSuccess || dev >= count)
        return from_cuda(cudaErrorUnknown);
    DeviceGuard guard(dev);
    if (!guard.ok())
        return FP8_ERR_CUDA;
    int sms = 0, optin = 0;
    int rc = current_sms(&sms);
    if (rc != FP8_OK)
        return rc;
    if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
        return from_cuda(cudaErrorUnknown);
    fp8_gemm_t h = new (std::nothrow) fp8_gemm();
    if (!h)
        return FP8_ERR_CUDA;
    h->device = dev;
    h->num_sms = std::min(sms, kMaxCtas);
    h->max_smem = (size_t)optin;
    // SM pairs resident at once: half the SMs, unless some SM has no partner
    {
        const void *fn = fp8_gemm_kernel_fn(2, false, false);
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        int n = 0;
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(kFp8Threads, 1, 1);
        cfg.dynamicSmemBytes = fp8_smem_bytes(2, kFp8MaxWidth, 4);
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, optin) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
            delete h;
            return from_cuda(cudaErrorUnknown);
        }
        h->max_pairs = std::min(n, h->num_sms / 2);
    }
    void *err = nullptr;
    if ((rc = alloc_zeroed(&err, sizeof(uint32_t))) != FP8_OK) {
        delete h;
        return rc;
    }
    h->d_err = static_cast<uint32_t *>(err);
    *out = h;
    return FP8_OK;
}

FP8_API int fp8_gemm_destroy(fp8_gemm_t h)
{
    if (!h)
        return FP8_OK;
    DeviceGuard guard(h->device);
    if (h->d_err)
        cudaFree(h->d_err);
    if (h->workspace)
        cudaFree(h->workspace);
    delete h;
    return FP8_OK;
}

FP8_API int fp8_gemm_set_option(fp8_gemm_t h, int key, int64_t value)
{
    if (!h)
        return FP8_ERR_INVALID_ARG;
    bool ok = false;
    switch (key) {
    case FP8_GEMM_OPT_CTA_GROUP: ok = value >= 0 && value <= 2; break;
    case FP8_GEMM_OPT_TRANSPOSED: ok = value >= 0 && value <= 2; break;
    case FP8_GEMM_OPT_WIDTH: ok = value >= 0 && value <= kFp8MaxWidth && value % 16 == 0; break;
    case FP8_GEMM_OPT_SPLIT: ok = value >= 0 && value <= 2; break;
    // far above what any load takes to land: the CTAs of a pair that give up at different
    // times count on each other's having landed
    case FP8_GEMM_OPT_WATCHDOG_NS: ok = value >= 100000 && value <= 60000000000LL; break;
    case FP8_GEMM_OPT_FAULT_SKIP_LOAD: ok = value >= -1 && value <= 0x7FFFFFFF; break;
    case FP8_GEMM_OPT_RASTER_GROUP: ok = value >= 0 && value <= 1024; break;
    default: break;
    }
    if (!ok)
        return FP8_ERR_INVALID_ARG;
    if (h->opt[key] != value) {
        h->opt[key] = value;
        for (Plan &pl : h->plans)  // plans were made with the old options
            pl.valid = false;
        h->plan = nullptr;
    }
    return FP8_OK;
}

FP8_API int fp8_gemm_get_option(fp8_gemm_t h, int key, int64_t *value)
{
    if (!h || !value || key < 1 || key >= kNumOptions)
        return FP8_ERR_INVALID_ARG;
    *value = h->opt[key];
    return FP8_OK;
}

FP8_API int fp8_gemm_plan(fp8_gemm_t h, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldd,
                          int out_type)
{
    if (!h)
        return FP8_ERR_INVALID_ARG;
    h->plan = nullptr;
    int rc = fp8_gemm_check_problem(M, N, K, lda, ldb, ldd, out_type);
    if (rc != FP8_OK)
        return rc;
    Plan *slot = &h->plans[0];
    for (Plan &pl : h->plans) {
        if (pl.valid && pl.M == M && pl.N == N && pl.K == K && pl.lda == lda && pl.ldb == ldb && pl.ldd == ldd &&
            pl.out_type == out_type) {
            pl.used = ++h->clock;
            h->plan = &pl;
            return FP8_OK;
        }
        if (!pl.valid ? slot->valid : (slot->valid && pl.used < slot->used))
            slot = &pl;
    }
    DeviceGuard guard(h->device);
    if (!guard.ok())
        return FP8_ERR_CUDA;
    Plan pl;
    pl.M = M, pl.N = N, pl.K = K, pl.lda = lda, pl.ldb = ldb, pl.ldd = ldd;
    pl.out_type = out_type;
    pl.k_blocks = ceil_div(K, kFp8BlockK);
    if (M > 0 && N > 0 && K > 0 && (rc = make_plan(h, pl)) != FP8_OK)
        return rc;
    pl.valid = true;
    pl.used = ++h->clock;
    *slot = pl;
    h->plan = slot;
    return FP8_OK;
}

FP8_API int fp8_gemm_plan_info(fp8_gemm_t h, fp8_gemm_plan_info_t *info)
{
    if (!h || !info)
        return FP8_ERR_INVALID_ARG;
    if (!h->plan)
        return FP8_ERR_NOT_PLANNED;
    const Plan &pl = *h->plan;
    std::memset(info, 0, sizeof(*info));
    info->tiles = pl.tiles;
    info->k_blocks = pl.k_blocks;
    info->grid_ctas = pl.grid;
    info->cta_group = pl.cta_group;
    info->transposed = pl.transposed ? 1 : 0;
    info->width = pl.width;
    info->stages = pl.stages;
    info->split_tiles = (int32_t)pl.sk_tiles;
    info->smem_bytes = (int32_t)pl.smem;
    info->regs_per_thread = pl.regs;
    info->cluster = pl.cluster;
    return FP8_OK;
}

FP8_API int fp8_gemm_workspace(fp8_gemm_t h, int64_t *bytes)
{
    if (!h || !bytes)
        return FP8_ERR_INVALID_ARG;
    *bytes = 0;
    if (!h->plan)
        return FP8_ERR_NOT_PLANNED;
    *bytes = (int64_t)workspace_bytes(*h->plan);
    return FP8_OK;
}

FP8_API int fp8_gemm_run(fp8_gemm_t h, const void *A, const void *SA, const void *B, const void *SB, void *D,
                         void *stream)
{
    if (!h)
        return FP8_ERR_INVALID_ARG;
    if (!h->plan)
        return FP8_ERR_NOT_PLANNED;
    const size_t most = (size_t)std::max(h->num_sms, 2 * h->max_pairs) * (kPartialBytes + kFlagBytes);
    if (!h->workspace && workspace_bytes(*h->plan)) {
        DeviceGuard guard(h->device);
        if (!guard.ok())
            return FP8_ERR_CUDA;
        const int rc = alloc_zeroed(&h->workspace, most);
        if (rc != FP8_OK)
            return rc;
    }
    return fp8_gemm_run_in(h, A, SA, B, SB, D, h->workspace, h->workspace ? (int64_t)most : 0, stream);
}

FP8_API int fp8_gemm_run_in(fp8_gemm_t h, const void *A, const void *SA, const void *B, const void *SB, void *D,
                            void *workspace, int64_t size, void *stream)
{
    if (!h)
        return FP8_ERR_INVALID_ARG;
    if (!h->plan)
        return FP8_ERR_NOT_PLANNED;
    Plan &pl = *h->plan;
    const size_t need = workspace_bytes(pl);
    if (need && (!workspace || size < (int64_t)need))
        return FP8_ERR_INVALID_ARG;
    if (need && !aligned(workspace, 16))
        return FP8_ERR_ALIGNMENT;
    if (pl.M == 0 || pl.N == 0)
        return FP8_OK;
    const uintptr_t esize = pl.out_type == FP8_FP32 ? 4 : 2;
    if (!D || (pl.K > 0 && (!A || !SA || !B || !SB)))
        return FP8_ERR_INVALID_ARG;
    if (!aligned(D, esize) || !aligned(A, 16) || !aligned(B, 16) || !aligned(SA, 4) || !aligned(SB, 4))
        return FP8_ERR_ALIGNMENT;
    DeviceGuard guard(h->device);
    if (!guard.ok())
        return FP8_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pl.K == 0)  // an empty sum
        return from_cuda(cudaMemset2DAsync(D, (size_t)pl.ldd * esize, 0, (size_t)pl.N * esize, (size_t)pl.M, st));

    if (!pl.maps || pl.mA != A || pl.mB != B || pl.mD != D) {
        pl.maps = false;
        const void *rp = pl.transposed ? B : A, *cp = pl.transposed ? A : B;
        const int64_t rows = pl.transposed ? pl.N : pl.M, cols = pl.transposed ? pl.M : pl.N;
        const int64_t ldr = pl.transposed ? pl.ldb : pl.lda, ldc = pl.transposed ? pl.lda : pl.ldb;
        int rc = encode_2d(&pl.tmR, CU_TENSOR_MAP_DATA_TYPE_UINT8, rp, (uint64_t)pl.K, (uint64_t)rows, (uint64_t)ldr,
                           kFp8BlockK, kFp8RowsPerCta, CU_TENSOR_MAP_SWIZZLE_128B);
        if (rc == FP8_OK)
            rc = encode_2d(&pl.tmC, CU_TENSOR_MAP_DATA_TYPE_UINT8, cp, (uint64_t)pl.K, (uint64_t)cols, (uint64_t)ldc,
                           kFp8BlockK, (uint32_t)(pl.width / pl.cta_group), CU_TENSOR_MAP_SWIZZLE_128B);
        if (rc != FP8_OK)
            return rc;
        // D by TMA where its rows are 16-byte aligned, else by the threads
        pl.d_tma = aligned(D, 16) && (pl.ldd * (int64_t)esize) % 16 == 0 &&
                   encode_2d(&pl.tmD,
                             esize == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, D,
                             (uint64_t)pl.N, (uint64_t)pl.M, (uint64_t)pl.ldd * esize, (uint32_t)(64 / esize), 32,
                             CU_TENSOR_MAP_SWIZZLE_64B) == FP8_OK;
        if (!pl.d_tma)
            std::memset(&pl.tmD, 0, sizeof(pl.tmD));  // passed, never used
        pl.mA = A, pl.mB = B, pl.mD = D;
        pl.maps = true;
    }

    Fp8GemmParams p;
    p.rows = (int32_t)(pl.transposed ? pl.N : pl.M);
    p.cols = (int32_t)(pl.transposed ? pl.M : pl.N);
    p.num_k_blocks = (int32_t)pl.k_blocks;
    p.num_row_tiles = (int32_t)pl.row_tiles;
    p.num_col_tiles = (int32_t)pl.col_tiles;
    p.num_tiles = (int32_t)pl.tiles;
    p.raster_group = fp8_raster_group(h->opt[FP8_GEMM_OPT_RASTER_GROUP], pl.row_tiles);
    p.width = pl.width;
    p.stages = pl.stages;
    p.sk_tiles = (int32_t)pl.sk_tiles;
    p.sk_units = pl.sk_tiles * pl.k_blocks;
    p.cluster = pl.cluster;
    p.D_rows = (int32_t)pl.M;
    p.D_cols = (int32_t)pl.N;
    p.out_fp32 = pl.out_type == FP8_FP32 ? 1 : 0;
    p.d_tma = pl.d_tma ? 1 : 0;
    p.ldd = pl.ldd;
    p.D = D;
    p.s_rows = static_cast<const uint32_t *>(pl.transposed ? SB : SA);
    p.s_cols = static_cast<const uint32_t *>(pl.transposed ? SA : SB);
    p.partials = need ? static_cast<float *>(workspace) : nullptr;
    p.flags = need ? reinterpret_cast<uint32_t *>(p.partials + (size_t)pl.grid * kFp8PartialFloats) : nullptr;
    p.err = h->d_err;
    // a tile's waits grow with K; 2 us a k-block is far above any measured
    p.watchdog_ns = std::max<uint64_t>((uint64_t)h->opt[FP8_GEMM_OPT_WATCHDOG_NS],
                                       h->opt[FP8_GEMM_OPT_FAULT_SKIP_LOAD] >= 0 ? 0 : (uint64_t)pl.k_blocks * 2000u);
    p.fault_skip_it = (int32_t)h->opt[FP8_GEMM_OPT_FAULT_SKIP_LOAD];

    if (need) {
        const int rc = from_cuda((cudaError_t)launch_fp8_clear(p.flags, pl.grid * kFp8EpiWarps, st));
        if (rc != FP8_OK)
            return rc;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)pl.grid, 1, 1);
    cfg.blockDim = dim3(kFp8Threads, 1, 1);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    const int together = pl.cta_group * pl.cluster;  // one of the two is 1
    attr[1].val.clusterDim.x = (unsigned)together;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = together > 1 ? 2 : 1;
    void *args[4] = {&pl.tmR, &pl.tmC, &pl.tmD, &p};
    return from_cuda(cudaLaunchKernelExC(&cfg, pl.fn, args));
}

FP8_API int fp8_gemm_device_status(fp8_gemm_t h, uint32_t *detail)
{
    if (detail)
        *detail = 0;
    if (!h)
        return FP8_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (!guard.ok())
        return FP8_ERR_CUDA;
    // The whole device: a launch may run again on any stream, from a graph that captured
    // it, and the stream it was first made on may be gone.
    uint32_t word = 0;
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(&word, h->d_err, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess)
        return from_cuda(cudaErrorUnknown);
    if (word == 0)
        return FP8_OK;
    if (detail)
        *detail = word;
    const uint32_t none = 0;
    if (cudaMemcpy(h->d_err, &none, sizeof(none), cudaMemcpyHostToDevice) != cudaSuccess)
        return from_cuda(cudaErrorUnknown);
    return FP8_ERR_DEVICE_TIMEOUT;
}

FP8_API int fp8_quantize(const void *x, int x_type, int64_t ldx, int64_t R, int64_t C, int tile,
                         const float *row_factor, const void *column_factor, int column_type, void *codes, int64_t ldq,
                         void *scales, void *codes_t, int64_t ldqt, void *scales_t, void *stream)
{
    if (R < 0 || C < 0 || R > kMaxDim || C > kMaxDim || bad_pitch(ldx, C))
        return FP8_ERR_INVALID_ARG;
    if ((x_type != FP8_BF16 && x_type != FP8_FP32) || (column_type != FP8_BF16 && column_type != FP8_FP32))
        return FP8_ERR_INVALID_ARG;
    if (R == 0 || C == 0)
        return FP8_OK;
    const bool rows = codes || scales, cols = codes_t || scales_t;
    if (!x || (!rows && !cols) || (rows && (!codes || !scales || bad_pitch(ldq, C))) ||
        (cols && (!codes_t || !scales_t || bad_pitch(ldqt, R))))
        return FP8_ERR_INVALID_ARG;
    const uintptr_t esize = x_type == FP8_FP32 ? 4 : 2;
    if (!aligned(x, esize) || !aligned(row_factor, 4) || !aligned(column_factor, column_type == FP8_FP32 ? 4 : 2))
        return FP8_ERR_ALIGNMENT;
    if (rows && (!aligned(codes, 16) || ldq % 16 != 0 || !aligned(scales, 4)))
        return FP8_ERR_ALIGNMENT;
    if (cols && (!aligned(codes_t, 16) || ldqt % 16 != 0 || !aligned(scales_t, 4)))
        return FP8_ERR_ALIGNMENT;
    if (R > kMaxRows || C > kMaxRows || ceil_div(R, kFp8BlockK) * ceil_div(C, kFp8BlockK) > kMaxDim)
        return FP8_ERR_UNSUPPORTED;
    int sms = 0;
    const int rc = current_sms(&sms);
    if (rc != FP8_OK)
        return rc;
    QuantizeParams p;
    p.x = x;
    p.ldx = ldx;
    p.R = (int32_t)R;
    p.C = (int32_t)C;
    p.x_fp32 = x_type == FP8_FP32 ? 1 : 0;
    p.tile = tile ? 1 : 0;
    p.row_factor = row_factor;
    p.column_factor = column_factor;
    p.column_fp32 = column_type == FP8_FP32 ? 1 : 0;
    p.x_vec = aligned(x, 16) && (ldx * (int64_t)esize) % 16 == 0 ? 1 : 0;
    p.column_vec = aligned(column_factor, 16) ? 1 : 0;
    p.codes = static_cast<uint8_t *>(codes);
    p.ldq = ldq;
    p.scales = static_cast<uint8_t *>(scales);
    p.codes_t = static_cast<uint8_t *>(codes_t);
    p.ldqt = ldqt;
    p.scales_t = static_cast<uint8_t *>(scales_t);
    return from_cuda((cudaError_t)launch_quantize(p, static_cast<cudaStream_t>(stream)));
}

FP8_API int fp8_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                        int weight_type, int64_t R, int64_t C, float eps, void *h, int64_t ldh, void *codes,
                        int64_t ldq, void *scales, float *rstd, void *stream)
{
    if (R < 0 || C < 1 || R > kMaxDim || (weight_type != FP8_BF16 && weight_type != FP8_FP32) || !(eps >= 0.f))
        return FP8_ERR_INVALID_ARG;
    if (C > FP8_NORM_MAX_COLUMNS)
        return FP8_ERR_UNSUPPORTED;
    if (bad_pitch(ldx, C) || bad_pitch(ldq, C) || (residual && (bad_pitch(ldr, C) || bad_pitch(ldh, C))))
        return FP8_ERR_INVALID_ARG;
    if (R == 0)
        return FP8_OK;
    if (!x || !weight || !codes || !scales || (residual && !h))
        return FP8_ERR_INVALID_ARG;
    const uintptr_t wsize = weight_type == FP8_FP32 ? 4 : 2;
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(h, 2) || !aligned(weight, wsize) || !aligned(rstd, 4) ||
        !aligned(codes, 16) || ldq % 16 != 0 || !aligned(scales, 4))
        return FP8_ERR_ALIGNMENT;
    if (residual &&
        (rows_clash(x, 2 * ldx, h, 2 * ldh, R, 2 * C) || rows_clash(residual, 2 * ldr, h, 2 * ldh, R, 2 * C)))
        return FP8_ERR_INVALID_ARG;
    int sms = 0;
    const int rc = current_sms(&sms);
    if (rc != FP8_OK)
        return rc;
    NormParams p;
    p.x = static_cast<const uint16_t *>(x);
    p.ldx = ldx;
    p.residual = static_cast<const uint16_t *>(residual);
    p.ldr = ldr;
    p.weight = weight;
    p.w_fp32 = weight_type == FP8_FP32 ? 1 : 0;
    p.R = (int32_t)R;
    p.C = (int32_t)C;
    p.inv_c = 1.f / (float)p.C;
    p.eps = eps;
    p.w_vec = aligned(weight, 16) ? 1 : 0;
    p.vec = aligned(x, 16) && ldx % 8 == 0 &&
            (!residual || (aligned(residual, 16) && ldr % 8 == 0 && aligned(h, 16) && ldh % 8 == 0));
    p.h = static_cast<uint16_t *>(h);
    p.ldh = ldh;
    p.codes = static_cast<uint8_t *>(codes);
    p.ldq = ldq;
    p.scales = static_cast<uint8_t *>(scales);
    p.rstd = rstd;
    return from_cuda((cudaError_t)launch_rmsnorm(p, sms, static_cast<cudaStream_t>(stream)));
}

FP8_API int fp8_rmsnorm_backward_workspace(int64_t R, int64_t C, int64_t *bytes)
{
    if (!bytes)
        return FP8_ERR_INVALID_ARG;
    *bytes = 0;
    if (R < 0 || C < 1 || R > kMaxDim)
        return FP8_ERR_INVALID_ARG;
    if (C > FP8_NORM_MAX_COLUMNS)
        return FP8_ERR_UNSUPPORTED;
    int sms = 0;
    const int rc = current_sms(&sms);
    if (rc != FP8_OK)
        return rc;
    *bytes = (int64_t)rmsnorm_backward_ctas(R, C, sms) * C * (int64_t)sizeof(float);
    return FP8_OK;
}

FP8_API int fp8_rmsnorm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *weight,
                                 int weight_type, const float *rstd, const void *dresidual, int64_t lddr, void *dx,
                                 int64_t lddx, float *dweight, int64_t R, int64_t C, void *workspace,
                                 int64_t workspace_bytes, void *stream)
{
    if (weight_type != FP8_BF16 && weight_type != FP8_FP32)
        return FP8_ERR_INVALID_ARG;
    int64_t need = 0;
    int rc = fp8_rmsnorm_backward_workspace(R, C, &need);
    if (rc != FP8_OK)
        return rc;
    if (bad_pitch(lddy, C) || bad_pitch(ldh, C) || bad_pitch(lddx, C) || (dresidual && bad_pitch(lddr, C)) || !dweight)
        return FP8_ERR_INVALID_ARG;
    if (!aligned(dweight, 4))
        return FP8_ERR_ALIGNMENT;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (R == 0)  // an empty sum
        return from_cuda(cudaMemsetAsync(dweight, 0, (size_t)C * sizeof(float), st));
    if (!dy || !h || !weight || !rstd || !dx || !workspace || workspace_bytes < need)
        return FP8_ERR_INVALID_ARG;
    if (!aligned(dy, 2) || !aligned(h, 2) || !aligned(weight, weight_type == FP8_FP32 ? 4 : 2) || !aligned(rstd, 4) ||
        !aligned(dresidual, 2) || !aligned(dx, 2) || !aligned(workspace, 16))
        return FP8_ERR_ALIGNMENT;
    if (rows_clash(dy, 2 * lddy, dx, 2 * lddx, R, 2 * C) || rows_clash(h, 2 * ldh, dx, 2 * lddx, R, 2 * C) ||
        (dresidual && rows_clash(dresidual, 2 * lddr, dx, 2 * lddx, R, 2 * C)))
        return FP8_ERR_INVALID_ARG;
    int sms = 0;
    if ((rc = current_sms(&sms)) != FP8_OK)
        return rc;
    NormBackwardParams p;
    p.dy = static_cast<const uint16_t *>(dy);
    p.lddy = lddy;
    p.h = static_cast<const uint16_t *>(h);
    p.ldh = ldh;
    p.weight = weight;
    p.w_fp32 = weight_type == FP8_FP32 ? 1 : 0;
    p.rstd = rstd;
    p.dres = static_cast<const uint16_t *>(dresidual);
    p.lddr = lddr;
    p.dx = static_cast<uint16_t *>(dx);
    p.lddx = lddx;
    p.dw = dweight;
    p.R = (int32_t)R;
    p.C = (int32_t)C;
    p.w_vec = aligned(weight, 16) ? 1 : 0;
    p.vec = aligned(dy, 16) && lddy % 8 == 0 && aligned(h, 16) && ldh % 8 == 0 && aligned(dx, 16) &&
            lddx % 8 == 0 && (!dresidual || (aligned(dresidual, 16) && lddr % 8 == 0));
    p.partials = static_cast<float *>(workspace);
    return from_cuda((cudaError_t)launch_rmsnorm_backward(p, sms, st));
}

}  // extern "C"
