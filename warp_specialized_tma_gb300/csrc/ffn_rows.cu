// Row kernels around the feed-forward products: the slope of an activation with the bias's
// gradient, the copy of rows that a tensor map cannot describe, the flags of split launches
// and the status word.
#include "ffn_math.cuh"
#include "gemm_common.cuh"

#include <algorithm>
#include <mutex>

namespace wstma {

namespace {

__device__ uint32_t ffn_status[32];  // one word is used; a sector of its own

constexpr int kSlopeWarps = 8;
constexpr int kSlopeColumns = 256;  // of a warp: 8 a lane
constexpr int kSlopeMaxSlices = 128;

// Vector c .. c+7 of a row, whatever its alignment; zero past the row's end.  `live` holds for all
// lanes or none: a lane behind the row's end still loads what its neighbour's vector ends in.
template <bool kVec>
__device__ __forceinline__ uint4 load8_any(const uint16_t *row, int32_t c, int32_t C, bool live)
{
    if constexpr (kVec)
        return live && c < C ? load8_bf16(row, c, C, true) : make_uint4(0u, 0u, 0u, 0u);
    else
        return load8_bf16_shifted(row, c, C, live);
}

// dz = dy act'(z), and its sums over a slice of the rows before it is rounded.  One pass over
// dy and z; a warp takes 256 columns of every eighth row of its slice, two rows at a time, so
// that a row's partial sums stay in registers until the end.  Sums of 8 warps meet in shared
// memory, those of the slices in ffn_column_sum_kernel: in a fixed order.
template <bool kVec, int A>
__global__ void __launch_bounds__(kSlopeWarps * 32) ffn_slope_kernel(const FfnSlopeParams p, int32_t slice_rows)
{
    __shared__ float sums[kSlopeWarps][kSlopeColumns];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t c = (int32_t)blockIdx.x * kSlopeColumns + 8 * lane;
    const int32_t r0 = (int32_t)blockIdx.y * slice_rows;
    const int32_t r1 = min(r0 + slice_rows, p.R);
    Pair sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sum[i] = both(0.0f);
    grid_dependency_wait();
    constexpr int kRows = 2;
    for (int32_t r = r0 + warp; r < r1; r += kRows * kSlopeWarps) {
        uint4 dy[kRows], z[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int32_t row = r + k * kSlopeWarps;
            const bool live = row < r1;
            dy[k] = load8_any<kVec>(p.dy + (int64_t)min(row, r1 - 1) * p.lddy, c, p.C, live);
            if constexpr (A != kActNone)
                z[k] = load8_any<kVec>(p.z + (int64_t)min(row, r1 - 1) * p.ldz, c, p.C, live);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int32_t row = r + k * kSlopeWarps;
            const uint32_t yw[4] = {dy[k].x, dy[k].y, dy[k].z, dy[k].w};
            Pair f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = pair_of_bf16(yw[i]);
            if constexpr (A != kActNone) {
                const uint32_t zw[4] = {z[k].x, z[k].y, z[k].z, z[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Pair a, d;
                    ffn_act_slope<A>(pair_of_bf16(zw[i]), a, d);
                    f[i] = f[i] * d;
                }
                if (row < r1 && c < p.C)  // rows of dz are whole 16-byte groups, of which the last may be padding
                    *reinterpret_cast<uint4 *>(p.dz + (int64_t)row * p.lddz + c) =
                        make_uint4(bf16_pair(f[0]), bf16_pair(f[1]), bf16_pair(f[2]), bf16_pair(f[3]));
            }
            if (row < r1) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[i] = sum[i] + f[i];
            }
        }
    }
    if (p.dbias == nullptr)
        return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f32x2_parts(sum[i].v, sums[warp][8 * lane + 2 * i], sums[warp][8 * lane + 2 * i + 1]);
    __syncthreads();
    const int32_t col = (int32_t)blockIdx.x * kSlopeColumns + (int32_t)threadIdx.x;
    if (col < p.C) {
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < kSlopeWarps; ++k)
            t += sums[k][threadIdx.x];
        if (gridDim.y == 1)
            p.dbias[col] = t;
        else
            p.partials[(int64_t)blockIdx.y * p.C + col] = t;
    }
}

__global__ void __launch_bounds__(256) ffn_column_sum_kernel(const float *partials, float *out, int32_t C, int32_t slices)
{
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int32_t c = (int32_t)blockIdx.x * 32 + lane;
    grid_dependency_wait();
    float t = 0.0f;
    if (c < C)
#pragma unroll 4
        for (int32_t s = part; s < slices; s += 8)
            t += partials[(int64_t)s * C + c];
    sums[part][lane] = t;
    __syncthreads();
    if (part == 0 && c < C) {
#pragma unroll
        for (int k = 1; k < 8; ++k)
            t += sums[k][lane];
        out[c] = t;
    }
}

// What a call's products need before they start: copies of operands at the copy's bandwidth, and the
// flags of split tiles at 0 (not left so by the launch before: one that gave up leaves some set, and
// the next would take old partials for its own).  A warp's unit is 1024 columns of a row,
// four vectors a lane in flight.  Rows that are not 16-byte aligned are read by whole 16-byte
// groups too: every lane takes what its own group lacks from its neighbour.
constexpr int kPackVectors = 4;
__global__ void __launch_bounds__(256) ffn_pack_kernel(const FfnPackJobs jobs)
{
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    if (jobs.n == 0)
        grid_launch_dependents();  // the product's start overlaps the kernel before this one
    grid_dependency_wait();
    if (blockIdx.x == 0)
        for (int32_t i = (int32_t)threadIdx.x; i < jobs.num_flags; i += 256)
            jobs.flags[i] = 0u;
    for (int64_t u0 = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u0 < jobs.units; u0 += step) {
        int64_t u = u0;
        int n = 0;
        while (u >= jobs.job[n].units)
            u -= jobs.job[n++].units;
        const FfnPackJob &j = jobs.job[n];
        const int64_t r = j.blocks == 1 ? u : u / j.blocks;
        const int32_t c = (int32_t)(u - r * j.blocks) * (kPackVectors * kSlopeColumns) + 8 * lane;
        const uint16_t *const from = j.src + r * j.lds;
        uint4 q[kPackVectors];
        if (j.vec) {
#pragma unroll
            for (int k = 0; k < kPackVectors; ++k) {
                const int32_t at = c + k * kSlopeColumns;
                if (at + 8 <= j.C)
                    q[k] = __ldcs(reinterpret_cast<const uint4 *>(from + at));
                else
                    q[k] = load8_bf16(from, at, j.C, false);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kPackVectors; ++k)
                q[k] = load8_bf16_shifted(from, c + k * kSlopeColumns, j.C, true);
        }
#pragma unroll
        for (int k = 0; k < kPackVectors; ++k)
            if (c + k * kSlopeColumns < j.C)
                *reinterpret_cast<uint4 *>(j.dst + r * j.ldd + c + k * kSlopeColumns) = q[k];
    }
    grid_launch_dependents();
}

template <typename... P, typename... A>
cudaError_t launch(void (*fn)(P...), dim3 grid, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <bool kVec>
cudaError_t launch_slope(const FfnSlopeParams &p, dim3 grid, int32_t rows, cudaStream_t st)
{
    switch (p.act) {
    case kActRelu: return launch(ffn_slope_kernel<kVec, kActRelu>, grid, st, p, rows);
    case kActSilu: return launch(ffn_slope_kernel<kVec, kActSilu>, grid, st, p, rows);
    case kActGelu: return launch(ffn_slope_kernel<kVec, kActGelu>, grid, st, p, rows);
    case kActGeluTanh: return launch(ffn_slope_kernel<kVec, kActGeluTanh>, grid, st, p, rows);
    default: return launch(ffn_slope_kernel<kVec, kActNone>, grid, st, p, rows);
    }
}

}  // namespace

int launch_ffn_pack(FfnPackJobs &jobs, int num_sms, cudaStream_t stream)
{
    jobs.units = 0;
    for (int i = 0; i < jobs.n; ++i) {
        FfnPackJob &j = jobs.job[i];
        j.blocks = (j.C + kPackVectors * kSlopeColumns - 1) / (kPackVectors * kSlopeColumns);
        j.vec = (reinterpret_cast<uintptr_t>(j.src) & 15u) == 0 && j.lds % 8 == 0;
        j.units = j.R * j.blocks;
        jobs.units += j.units;
    }
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>((jobs.units + 7) / 8, (int64_t)num_sms * 8));
    return launch(ffn_pack_kernel, dim3((unsigned)ctas), stream, jobs);
}

// Slices of the rows: enough CTAs to fill the GPU four times over, 16 rows a slice at least.
int ffn_slope_slices(int64_t R, int64_t C, int num_sms)
{
    const int64_t blocks = (C + kSlopeColumns - 1) / kSlopeColumns;
    const int64_t want = std::max<int64_t>(1, 4 * (int64_t)num_sms / std::max<int64_t>(blocks, 1));
    return (int)std::max<int64_t>(1, std::min({want, (R + 15) / 16, (int64_t)kSlopeMaxSlices}));
}

int launch_ffn_slope(const FfnSlopeParams &p, int num_sms, cudaStream_t stream)
{
    int slices = ffn_slope_slices(p.R, p.C, num_sms);
    const int32_t rows = (p.R + slices - 1) / slices;
    slices = rows ? (p.R + rows - 1) / rows : 1;
    const dim3 grid((unsigned)((p.C + kSlopeColumns - 1) / kSlopeColumns), (unsigned)std::max(slices, 1));
    cudaError_t e = p.vec ? launch_slope<true>(p, grid, rows, stream) : launch_slope<false>(p, grid, rows, stream);
    if (e == cudaSuccess && p.dbias && slices > 1)
        e = launch(ffn_column_sum_kernel, dim3((unsigned)((p.C + 31) / 32)), stream, (const float *)p.partials, p.dbias,
                   p.C, (int32_t)slices);
    return e;
}

uint32_t *ffn_status_word()
{
    static uint32_t *known[64];
    static std::mutex lock;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) {
        cudaGetLastError();
        return nullptr;
    }
    std::lock_guard<std::mutex> hold(lock);
    if (!known[dev]) {
        // also while a stream of this thread is capturing
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        cudaThreadExchangeStreamCaptureMode(&mode);
        void *at = nullptr;
        if (cudaGetSymbolAddress(&at, ffn_status) == cudaSuccess)
            known[dev] = static_cast<uint32_t *>(at);
        else
            cudaGetLastError();
        cudaThreadExchangeStreamCaptureMode(&mode);
    }
    return known[dev];
}

}  // namespace wstma
