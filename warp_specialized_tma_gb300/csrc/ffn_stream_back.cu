// A few tokens' products with weights that are contiguous along the result's columns: an input's
// gradient dx = d W (or d0 W0 + d1 W1) and the gated gradient's dh = dy Wd with its epilogue.
//
// As in ffn_stream.cu the weights' bytes bound them, and go straight into registers as operands of
// mma.sync.  Here a result's columns are the MMA's rows, and the sum runs down the weights' rows: a lane
// loads 16 bytes, eight columns, of four rows, and pairs of rows are brought together by byte
// permutes.  Eight lanes read 128 bytes of a row, so a warp's unit is 16 rows of 64 columns.  The
// MMA adds up over k in any order: lane t of four stands for rows 4 t .. 4 t + 3 of the unit, in
// both operands alike, so that a token's part is one load of 8 bytes.
//
// The columns are shared out in eights among clusters of CTAs, whose CTAs and warps take every so
// many units of the rows; up to four units a warp are in flight (128 KB an SM; no load in the loop
// depends on a condition).  Sums meet in shared memory, the CTAs' in distributed shared memory, in a
// fixed order.  More CTAs to a cluster for fewer columns: a cluster's share is then wide enough for
// whole lines, which is what bandwidth hangs on (4096 x 4096 in shares of 7 eights and of 3 and a half
// took 15.3 us).  Units of 32 rows, with a token's part in one load for two units, were no faster.
//
// Measured (us, from a graph; in brackets the kernel of ffn_gemm.cuh; the weights' time in HBM):
//   dx of a 8192 x 8192 weight   1 token 24.8 (25.8; 19.8), 8 tokens 26.7 (25.9), 16 tokens 33.9 (26.2)
//   dx of a 4096 x 4096 weight   1 token 10.0 (12.3;  5.0), 8 tokens 11.6 (12.7), 16 tokens 14.9 (13.1)
//   dx of a 13528 x 5048 weight  1 token 24.1 (28.5; 20.2), 8 tokens 25.9 (29.2)
//   dg, du, h of 2 tokens, 584 x 10080   6.7 (13.5; 1.7), of 10 tokens, 8056 x 2168  13.9 (21.8; 5.2)
// One token's are bound by HBM (up to 6.4 TB/s); with more the tokens' words, read from L1 by every warp,
// count.
#include "ffn_math.cuh"
#include "ffn_stream.cuh"
#include "gemm_common.cuh"

#include <algorithm>
#include <mutex>

namespace wstma {

namespace {

constexpr int kBackWarps = 16;
constexpr int kBackRows = 16;  // of a unit
constexpr int kBackColumns = 64;

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float aux_value(const FfnAux &a, int32_t m, int32_t c, int32_t M)
{
    if (a.scales) {
        float lo, hi;
        f32x2_parts(pair_of_e4m3(static_cast<const uint8_t *>(a.p)[(int64_t)m * a.ld + c]).v, lo, hi);
        return lo * ffn_scale(a.scales[((int64_t)(c >> 9) * M + m) * 4 + ((c >> 7) & 3)]);
    }
    return bf16_low(static_cast<const uint16_t *>(a.p)[(int64_t)m * a.ld + c]);
}

__device__ __forceinline__ void store_bf16(const FfnOut &out, int32_t m, int32_t c, float v)
{
    static_cast<uint16_t *>(out.p)[(int64_t)m * out.ld + c] = (uint16_t)bf16_pair(v, 0.0f);
}

// kTiles * 8 tokens.
template <int kTiles, bool kGrad>
__global__ void __launch_bounds__(kBackWarps * 32, 1) ffn_stream_back_kernel(const FfnStreamBackParams p)
{
    constexpr int kDepth = kTiles == 1 ? 4 : 3;           // units in flight
    constexpr int kWarpSums = kBackColumns * 8 * kTiles;  // [column][token]
    extern __shared__ float sums[];                       // [warp], then the CTA's, [token][column]
    float *const total = sums + kBackWarps * kWarpSums;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int32_t S = p.ranks, rank = (int32_t)blockIdx.x % S;
    const int32_t first = (int32_t)blockIdx.x / S * p.share;  // in eights of columns
    const int32_t R = min(p.share, (p.C + 7) / 8 - first);    // of this cluster
    const int wr = warp % p.groups, wk = warp / p.groups, ranges = kBackWarps / p.groups;
    const int32_t all = ranges * S, me = rank * ranges + wk;
    const int32_t full = p.N / kBackRows, units = wk < ranges ? p.products * full : 0;
    const int32_t n = units > me ? (units - me + all - 1) / all : 0;  // of this warp
    grid_launch_dependents();
    grid_dependency_wait();
    // Columns and tokens that are not there are another's: their results are not read, their loads
    // are part of that one's, and no load depends on a condition.
    const int32_t e0 = first + wr * R / p.groups, e1 = first + (wr + 1) * R / p.groups;
    const int64_t col = 8 * (int64_t)max(min(e0 + g, e1 - 1), first);
    uint4 w[kDepth][4];
    uint2 d[kDepth][kTiles];
    float acc[4][kTiles][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int b = 0; b < kTiles; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][b][e] = 0.0f;
    auto load = [&](uint4(&to)[4], uint2(&ds)[kTiles], int32_t i) {
        const int32_t u = me + i * all;
        const int which = u >= full ? 1 : 0;
        const int64_t row = (int64_t)(u - which * full) * kBackRows + 4 * t;
        const uint16_t *const from = p.w[which] + row * p.ldw[which] + col;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            to[r] = load_once(from + r * p.ldw[which]);
#pragma unroll
        for (int b = 0; b < kTiles; ++b)
            ds[b] = load_again_8(p.d[which] + (int64_t)min(g + 8 * b, p.M - 1) * p.ldd[which] + row);
    };
    auto use = [&](uint4(&from)[4], uint2(&ds)[kTiles]) {
        const uint32_t r[4][4] = {{from[0].x, from[0].y, from[0].z, from[0].w},
                                  {from[1].x, from[1].y, from[1].z, from[1].w},
                                  {from[2].x, from[2].y, from[2].z, from[2].w},
                                  {from[3].x, from[3].y, from[3].z, from[3].w}};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = __byte_perm(r[0][i], r[1][i], 0x5410), a1 = __byte_perm(r[0][i], r[1][i], 0x7632);
            const uint32_t a2 = __byte_perm(r[2][i], r[3][i], 0x5410), a3 = __byte_perm(r[2][i], r[3][i], 0x7632);
#pragma unroll
            for (int b = 0; b < kTiles; ++b)
                mma_16x8x16(acc[i][b], a0, a1, a2, a3, ds[b].x, ds[b].y);
        }
    };
    const int32_t rounds = n / kDepth;
    if (rounds > 0) {
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
            load(w[k], d[k], k);
        for (int32_t i = 1; i < rounds; ++i)
#pragma unroll
            for (int k = 0; k < kDepth; ++k) {
                use(w[k], d[k]);
                load(w[k], d[k], i * kDepth + k);
            }
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
            use(w[k], d[k]);
    }
#pragma unroll
    for (int k = 0; k < kDepth; ++k)
        if (rounds * kDepth + k < n)
            load(w[k], d[k], rounds * kDepth + k);
#pragma unroll
    for (int k = 0; k < kDepth; ++k)
        if (rounds * kDepth + k < n)
            use(w[k], d[k]);
    // the rows behind the last whole unit: one warp's a product, zeros where there are none
    for (int which = 0; which < p.products; ++which)
        if (p.N % kBackRows && wk < ranges && me == which % all) {
            const int64_t row = (int64_t)full * kBackRows + 4 * t;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                w[0][r] = row + r < p.N ? load_once(p.w[which] + (row + r) * p.ldw[which] + col) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int b = 0; b < kTiles; ++b) {
                const uint16_t *const from = p.d[which] + (int64_t)min(g + 8 * b, p.M - 1) * p.ldd[which] + row;
                uint32_t v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    v[r] = row + r < p.N ? from[r] : 0u;
                d[0][b] = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
            }
            use(w[0], d[0]);
        }
    float *const mine = sums + warp * kWarpSums;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int b = 0; b < kTiles; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                mine[(8 * g + 2 * i + (e >> 1)) * 8 * kTiles + 8 * b + 2 * t + (e & 1)] = acc[i][b][e];
    __syncthreads();
    const int32_t cols = 8 * R;
    auto of_cta = [&](int32_t m, int32_t c) {
        const int32_t eight = c >> 3;
        int group = eight * p.groups / R;  // the group whose share holds these columns
        while (group + 1 < p.groups && (group + 1) * R / p.groups <= eight)
            ++group;
        const float *const from =
            sums + group * kWarpSums + (8 * (eight - group * R / p.groups) + (c & 7)) * 8 * kTiles + m;
        float s = 0.0f;
        for (int k = 0; k < ranges; ++k)
            s += from[k * p.groups * kWarpSums];
        return s;
    };
    auto finish = [&](int32_t m, int32_t at, float s) {
        const int32_t c = 8 * first + at;
        if (c >= p.C)
            return;
        if constexpr (kGrad) {
            const float gate = aux_value(p.aux[0], m, c, p.M), up = aux_value(p.aux[1], m, c, p.M);
            float a = 0.0f, slope = 0.0f;
            ffn_with_act(p.act, [&](auto tag) {
                Pair both_a, both_d;
                ffn_act_slope<decltype(tag)::value>(pair(gate, gate), both_a, both_d);
                float unused;
                f32x2_parts(both_a.v, a, unused);
                f32x2_parts(both_d.v, slope, unused);
            });
            store_bf16(p.D[0], m, c, s * up * slope);
            store_bf16(p.D[1], m, c, s * a);
            store_bf16(p.D[2], m, c, a * up);
        } else {
            store_bf16(p.D[0], m, c, s);
        }
    };
    // one result a thread: columns fastest, so that a token's results are stored together
    if (S == 1) {
        for (int32_t i = (int32_t)threadIdx.x; i < cols * p.M; i += kBackWarps * 32)
            finish(i / cols, i % cols, of_cta(i / cols, i % cols));
        return;
    }
    for (int32_t i = (int32_t)threadIdx.x; i < cols * p.M; i += kBackWarps * 32)
        total[i] = of_cta(i / cols, i % cols);
    cluster_arrive_wait();
    const uint32_t local = smem_u32(total);
    for (int32_t i = rank * kBackWarps * 32 + (int32_t)threadIdx.x; i < cols * p.M; i += S * kBackWarps * 32) {
        float s = 0.0f;
        for (int32_t k = 0; k < S; ++k)
            s += ld_shared_cluster_f32(mapa_shared(local + 4u * (uint32_t)i, (uint32_t)k));
        finish(i / cols, i % cols, s);
    }
    cluster_arrive_wait();  // the others have read this CTA's sums
}

using Kernel = void (*)(FfnStreamBackParams);

Kernel kernel_of(bool grad, int32_t M)
{
    return M <= 8 ? (grad ? &ffn_stream_back_kernel<1, true> : &ffn_stream_back_kernel<1, false>)
                  : (grad ? &ffn_stream_back_kernel<2, true> : &ffn_stream_back_kernel<2, false>);
}

size_t smem_of(int32_t groups, int32_t M)
{
    const size_t tokens = M <= 8 ? 8 : 16;
    return ((size_t)kBackWarps + (size_t)groups) * kBackColumns * tokens * sizeof(float);
}

void describe(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], unsigned grid, int ranks, size_t smem,
              cudaStream_t stream)
{
    cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kBackWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

// Clusters of each size that are resident at once on the current device; all kernels here take an SM each.
cudaError_t resident(int device, int num_sms, const int **out)
{
    static int known[64][kFfnMaxCluster + 1];
    static std::mutex lock;
    std::lock_guard<std::mutex> hold(lock);
    int *const at = known[device];
    if (at[1] == 0) {
        for (int s = 2; s <= kFfnMaxCluster; ++s) {
            cudaLaunchConfig_t cfg;
            cudaLaunchAttribute attr[2];
            describe(cfg, attr, (unsigned)s, s, smem_of(1, 8), nullptr);
            cfg.numAttrs = 1;
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&at[s], kernel_of(false, 1), &cfg);
            if (e != cudaSuccess)
                return e;
            at[s] = std::min(at[s], num_sms / s);
        }
        at[1] = num_sms;
    }
    *out = at;
    return cudaSuccess;
}

}  // namespace

int launch_ffn_stream_back(FfnStreamBackParams &p, int device, int num_sms, cudaStream_t stream)
{
    const int *places = nullptr;
    cudaError_t e = resident(device, num_sms, &places);
    if (e != cudaSuccess)
        return e;
    // The size of cluster whose warps have the fewest units, of columns shared out by 64 bytes; a unit more
    // for each CTA that exchanges sums.
    const int64_t eights = ((int64_t)p.C + 7) / 8, units = (int64_t)p.products * ((p.N + kBackRows - 1) / kBackRows);
    int64_t best = 0, clusters = 1;
    for (int s = 1; s <= kFfnMaxCluster; ++s) {
        const int64_t most = std::min<int64_t>(places[s], eights);
        if (most < 1)
            continue;
        const int64_t share = ((eights + most - 1) / most + 3) / 4 * 4;
        if (share > 8 * kBackWarps)
            continue;
        const int64_t groups = (share + 7) / 8, warps = kBackWarps / groups * s;
        const int64_t cost = (units + warps - 1) / warps + s - 1;
        if (best == 0 || cost < best) {
            best = cost;
            p.ranks = s;
            p.share = (int32_t)share;
            p.groups = (int32_t)groups;
            clusters = (eights + share - 1) / share;
        }
    }
    const Kernel fn = kernel_of(p.aux[0].p != nullptr, p.M);
    const size_t smem = smem_of(p.groups, p.M);
    if (smem > 48 * 1024 &&
        (e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    describe(cfg, attr, (unsigned)(clusters * p.ranks), p.ranks, smem, stream);
    return cudaLaunchKernelEx(&cfg, fn, p);
}

int64_t ffn_stream_back_columns(int num_sms) { return (int64_t)num_sms * kBackColumns * kBackWarps; }

}  // namespace wstma
