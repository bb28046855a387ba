// The forward products for a few tokens: y = act(x W^T + bias) + residual and
// h = act(x Wg^T) (x Wu^T), with the weights read once, straight into registers.
//
// With so few tokens the weights' bytes bound a product (2 N K of them, 4 F C gated), and what the
// tensor-memory kernel (ffn_gemm.cuh) does before its first MMA and after its last costs as much
// as a small one.  Here a warp's lane loads 16 bytes of a weight's row and 16 bytes of a token's
// at the same k, and these are the operands of two mma.sync: the MMA adds up over k in any order, so
// a lane's eight consecutive k stand for the eight that the fragment layout gives it, in both
// operands alike.  16 rows of the weights are the MMA's rows, 8 tokens its columns.
//
// A CTA (one an SM) has the N / SMs rows that are its share, to within one row, so that all SMs
// read the same bytes; its 16 warps are `groups` of up to 16 of these rows times 16 / groups ranges
// of k, interleaved by 128 bytes.  Up to three chunks of 128 bytes a row are in flight in registers
// (96 KB an SM; HBM's rate times its latency asks for about 40; more spill).  No load in the loop
// depends on a condition: with one each, the warp waited for all loads it had issued, whatever the
// depth (1 x 8192 x 8192 30 us).  The ranges' sums meet in shared memory, in a fixed order.
//
// Measured (us, from a graph; in brackets the kernel of ffn_gemm.cuh; the weights' time in HBM):
//   linear 1 x 8192 x 8192   23.4 (31.7; 19.8), 16 tokens 25.8 (31.7), 32 tokens 36.2 (33.7)
//   linear 1 x 4096 x 4096    8.6 (12.5;  5.0), 16 tokens  9.5 (13.1), 32 tokens 12.3 (13.4)
//   linear 1 x 1024 x 1024    3.0 ( 7.7;  0.3)
//   gated 1 x 16384 x 4096   42.2 (46.4; 39.7), 16 tokens 51.8 (46.6)
//   gated 16 x 4096 x 4096   15.1 (20.8;  9.9), 32 tokens 19.3 (22.9)
// One token's are bound by HBM (5.7 to 6.4 TB/s), small ones by a launch and the first loads'
// latency; from 16 tokens on the tokens' words, read from L1 by every warp, cost as much as the
// weights'.
#include "ffn_math.cuh"
#include "ffn_stream.cuh"
#include "gemm_common.cuh"

#include <algorithm>

namespace wstma {

namespace {

constexpr int kStreamWarps = 16;
constexpr int kStreamK = 64;  // of a chunk: 128 bytes of a row

// Chunks of a warp whose products the MMA adds up before its sums move on, to this thread's places in shared memory
// (kLong: fp32 results of long sums; see ffn_gemm.cuh).
constexpr int kStreamSegment = kFfnSegment;

// kTiles * 8 tokens; kDual: two weights.
template <int kTiles, bool kDual, bool kLong>
__global__ void __launch_bounds__(kStreamWarps * 32, 1) ffn_stream_kernel(const FfnStreamParams p)
{
    constexpr int kW = kDual ? 2 : 1;
    constexpr int kDepth = kTiles == 4 ? 1 : kDual ? 3 - kTiles : 4 - kTiles;  // chunks in flight
    extern __shared__ float sums[];        // [warp][weight][tile][row of 16][token of 8]
    constexpr int kWarpSums = kW * kTiles * 128;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int wr = warp % p.groups, wk = warp / p.groups, ranges = kStreamWarps / p.groups;
    const int32_t first = (int32_t)((int64_t)blockIdx.x * p.N / gridDim.x);
    const int32_t end = (int32_t)((int64_t)(blockIdx.x + 1) * p.N / gridDim.x);
    const int32_t chunks = (p.K + kStreamK - 1) / kStreamK;
    const int32_t n = wk < ranges ? (chunks - wk + ranges - 1) / ranges : 0;  // of this warp
    grid_launch_dependents();
    grid_dependency_wait();
    // its rows, shared out evenly among the groups
    const int32_t R = end - first, r0 = first + wr * R / p.groups;
    // Rows and tokens that are not there are another's: their results are not read, their loads
    // are part of that one's, and no load depends on a condition.
    const uint16_t *wrow[kW][2], *xrow[kTiles];
#pragma unroll
    for (int a = 0; a < kW; ++a)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            wrow[a][r] = p.w[a] + (int64_t)min(r0 + g + 8 * r, end - 1) * p.ldw[a] + 8 * t;
#pragma unroll
    for (int b = 0; b < kTiles; ++b)
        xrow[b] = p.x + (int64_t)min(g + 8 * b, p.M - 1) * p.ldx + 8 * t;
    uint4 w[kDepth][kW][2][2];  // [weight][half of the chunk][row g or g + 8]
    uint4 x[kDepth][kTiles][2];
    float acc[kW][kTiles][4];
#pragma unroll
    for (int a = 0; a < kW; ++a)
#pragma unroll
        for (int b = 0; b < kTiles; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[a][b][e] = 0.0f;
    float *const mine = sums + warp * kWarpSums;
    auto place = [&](int a, int b, int e) { return (a * kTiles + b) * 128 + (g + 8 * (e >> 1)) * 8 + 2 * t + (e & 1); };
    auto move_on = [&]() {
#pragma unroll
        for (int a = 0; a < kW; ++a)
#pragma unroll
            for (int b = 0; b < kTiles; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mine[place(a, b, e)] += acc[a][b][e];
                    acc[a][b][e] = 0.0f;
                }
    };
    if constexpr (kLong)
#pragma unroll
        for (int i = 0; i < kWarpSums / 32; ++i)
            mine[i * 32 + lane] = 0.0f;
    if constexpr (kLong)
        __syncwarp();
    // `whole`: the chunk lies inside the rows
    auto load = [&](uint4(&to)[kW][2][2], uint4(&xs)[kTiles][2], int32_t i, bool whole) {
        const int32_t k = (wk + i * ranges) * kStreamK;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (whole || k + 32 * h + 8 * t < p.K) {
#pragma unroll
                for (int a = 0; a < kW; ++a)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        to[a][h][r] = load_once(wrow[a][r] + k + 32 * h);
#pragma unroll
                for (int b = 0; b < kTiles; ++b)
                    xs[b][h] = load_again_16(xrow[b] + k + 32 * h);
            } else {
#pragma unroll
                for (int a = 0; a < kW; ++a)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        to[a][h][r] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int b = 0; b < kTiles; ++b)
                    xs[b][h] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    };
    auto use = [&](uint4(&from)[kW][2][2], uint4(&xs)[kTiles][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int a = 0; a < kW; ++a) {
                const uint4 lo = from[a][h][0], hi = from[a][h][1];
#pragma unroll
                for (int b = 0; b < kTiles; ++b) {
                    mma_16x8x16(acc[a][b], lo.x, hi.x, lo.y, hi.y, xs[b][h].x, xs[b][h].y);
                    mma_16x8x16(acc[a][b], lo.z, hi.z, lo.w, hi.w, xs[b][h].z, xs[b][h].w);
                }
            }
    };
    // the chunks inside the rows, kDepth in flight; then what is left, one by one
    const int32_t full = p.K % kStreamK && n && (wk + (n - 1) * ranges) == chunks - 1 ? n - 1 : n;
    const int32_t rounds = full / kDepth;
    if (rounds > 0) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            load(w[d], x[d], d, true);
        for (int32_t i = 1; i < rounds; ++i) {
            if (kLong && i % (kStreamSegment / kDepth) == 0)
                move_on();
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                use(w[d], x[d]);
                load(w[d], x[d], i * kDepth + d, true);
            }
        }
        if (kLong)
            move_on();
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            use(w[d], x[d]);
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if (rounds * kDepth + d < n)
            load(w[d], x[d], rounds * kDepth + d, false);
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if (rounds * kDepth + d < n)
            use(w[d], x[d]);
    if constexpr (kLong) {
        move_on();
    } else {
#pragma unroll
        for (int a = 0; a < kW; ++a)
#pragma unroll
            for (int b = 0; b < kTiles; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mine[place(a, b, e)] = acc[a][b][e];
    }
    __syncthreads();
    // one result a thread: rows fastest, so that a token's results are stored together
    for (int32_t i = (int32_t)threadIdx.x; i < R * p.M; i += kStreamWarps * 32) {
        const int32_t m = i / R, row = i - m * R;
        int group = row * p.groups / R;  // the group whose share holds this row
        while (group + 1 < p.groups && (group + 1) * R / p.groups <= row)
            ++group;
        const float *from = sums + group * kWarpSums + (m >> 3) * 128 + (row - group * R / p.groups) * 8 + (m & 7);
        float s[kW];
#pragma unroll
        for (int a = 0; a < kW; ++a) {
            s[a] = 0.0f;
            for (int k = 0; k < ranges; ++k)
                s[a] += from[a * kTiles * 128 + k * p.groups * kWarpSums];
        }
        const int32_t col = first + row;
        if constexpr (kDual) {
            if (p.save) {
                static_cast<uint16_t *>(p.D[1].p)[(int64_t)m * p.D[1].ld + col] = (uint16_t)bf16_pair(s[0], 0.0f);
                static_cast<uint16_t *>(p.D[2].p)[(int64_t)m * p.D[2].ld + col] = (uint16_t)bf16_pair(s[1], 0.0f);
            }
            float h = 0.0f;
            ffn_with_act(p.act, [&](auto tag) { h = ffn_act<decltype(tag)::value>(s[0]) * s[1]; });
            static_cast<uint16_t *>(p.D[0].p)[(int64_t)m * p.D[0].ld + col] = (uint16_t)bf16_pair(h, 0.0f);
        } else {
            float z = s[0];
            if (p.bias)
                z += p.bias_fp32 ? static_cast<const float *>(p.bias)[col]
                                 : bf16_low(static_cast<const uint16_t *>(p.bias)[col]);
            if (p.save)
                static_cast<uint16_t *>(p.D[1].p)[(int64_t)m * p.D[1].ld + col] = (uint16_t)bf16_pair(z, 0.0f);
            float y = z;
            ffn_with_act(p.act, [&](auto tag) { y = ffn_act<decltype(tag)::value>(z); });
            if (p.residual)
                y += bf16_low(p.residual[(int64_t)m * p.ldr + col]);
            if (p.out_fp32)
                static_cast<float *>(p.D[0].p)[(int64_t)m * p.D[0].ld + col] = y;
            else
                static_cast<uint16_t *>(p.D[0].p)[(int64_t)m * p.D[0].ld + col] = (uint16_t)bf16_pair(y, 0.0f);
        }
    }
}

template <int kTiles, bool kDual, bool kLong = false>
cudaError_t run(const FfnStreamParams &p, unsigned grid, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kStreamWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = (size_t)kStreamWarps * kTiles * 128 * (kDual ? 2 : 1) * sizeof(float);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cfg.dynamicSmemBytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(ffn_stream_kernel<kTiles, kDual, kLong>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)cfg.dynamicSmemBytes);
        if (e != cudaSuccess)
            return e;
    }
    return cudaLaunchKernelEx(&cfg, ffn_stream_kernel<kTiles, kDual, kLong>, p);
}

}  // namespace

int launch_ffn_stream(FfnStreamParams &p, int num_sms, cudaStream_t stream)
{
    const unsigned grid = (unsigned)std::min<int64_t>(num_sms, ((int64_t)p.N + 3) / 4);
    const int64_t rows = ((int64_t)p.N + grid - 1) / grid;
    p.groups = (int32_t)((rows + 15) / 16);
    const bool dual = p.w[1] != nullptr;
    const int64_t chunks = ((int64_t)p.K + kStreamK - 1) / kStreamK;
    if (!dual && p.out_fp32 && chunks > (int64_t)kStreamSegment * (kStreamWarps / p.groups))
        return p.M <= 8    ? run<1, false, true>(p, grid, stream)
               : p.M <= 16 ? run<2, false, true>(p, grid, stream)
                           : run<4, false, true>(p, grid, stream);
    if (p.M <= 8)
        return dual ? run<1, true>(p, grid, stream) : run<1, false>(p, grid, stream);
    if (p.M <= 16)
        return dual ? run<2, true>(p, grid, stream) : run<2, false>(p, grid, stream);
    return dual ? run<4, true>(p, grid, stream) : run<4, false>(p, grid, stream);
}

int64_t ffn_stream_rows(int num_sms) { return (int64_t)num_sms * 16 * kStreamWarps; }

}  // namespace wstma
