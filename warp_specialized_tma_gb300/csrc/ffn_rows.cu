// Row kernels around the feed-forward products: the slope of an activation with the bias's
// gradient, the copy of rows that a tensor map cannot describe, the flags of split launches
// and the status word.
#include "ffn_math.cuh"
#include "gemm_common.cuh"

#include <algorithm>
#include <mutex>
#include <type_traits>

namespace wstma {

namespace {

__device__ uint32_t ffn_status[32];  // one word is used; a sector of its own

constexpr int kSlopeWarps = 8;
constexpr int kSlopeColumns = 256;  // of a warp: 8 a lane
constexpr int kSlopeMaxSlices = 128;

// The five words from word W on of a lane's 16-byte group and the next one, two bytes further if
// `half`: four words.  The next group is the next lane's; the last lane's is `last`.
template <int W>
__device__ __forceinline__ uint4 turn(const uint4 q, const uint4 last, bool half)
{
    const uint32_t own[4] = {q.x, q.y, q.z, q.w}, behind[4] = {last.x, last.y, last.z, last.w};
    const bool end = (threadIdx.x & 31u) == 31u;
    uint32_t w[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        if (W + k < 4) {
            w[k] = own[W + k];
        } else {
            const uint32_t n = __shfl_down_sync(0xFFFFFFFFu, own[W + k - 4], 1);
            w[k] = end ? behind[W + k - 4] : n;
        }
    }
    const uint32_t by = half ? 16u : 0u;
    return make_uint4(__funnelshift_r(w[0], w[1], by), __funnelshift_r(w[1], w[2], by),
                      __funnelshift_r(w[2], w[3], by), __funnelshift_r(w[3], w[4], by));
}

// Eight columns c .. c+7 of a row, c = 8 lane + a multiple of 256: loaded by get(), which several calls
// of may precede value(), so that their loads are in flight together.  `live` and the row hold for
// all lanes.  A row that is only 2-byte aligned is read by whole 16-byte groups, each lane the one its
// vector starts in; the shift is one of four cases, the same for the warp.  Only groups that hold a
// byte of the row are read; past its end the values are zero.
template <bool kVec>
struct Vector8 {
    uint4 q, last;

    __device__ __forceinline__ void get(const uint16_t *row, int32_t c, int32_t C, bool live)
    {
        q = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (kVec) {
            if (live && c < C)
                q = load8_bf16(row, c, C, true);
        } else {
            last = q;
            const uint32_t mis = (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u;
            const int32_t first = c - (int32_t)(mis >> 1);  // of the group
            if (live && first < C)
                q = *reinterpret_cast<const uint4 *>(row + first);
            if (live && (threadIdx.x & 31u) == 31u && mis != 0u && first + 8 < C)
                last = *reinterpret_cast<const uint4 *>(row + first + 8);
        }
    }

    __device__ __forceinline__ uint4 value(const uint16_t *row, int32_t c, int32_t C) const
    {
        if constexpr (kVec)
            return q;
        const uint32_t mis = (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u;
        const bool half = (mis & 2u) != 0u;
        uint4 o;
        switch (__shfl_sync(0xFFFFFFFFu, mis >> 2, 0)) {
        case 0: o = turn<0>(q, last, half); break;
        case 1: o = turn<1>(q, last, half); break;
        case 2: o = turn<2>(q, last, half); break;
        default: o = turn<3>(q, last, half); break;
        }
        if (c + 8 > C) {
            const int32_t n = max(C - c, 0);
            uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = 2 * k + 1 < n ? w[k] : 2 * k < n ? w[k] & 0xFFFFu : 0u;
            o = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return o;
    }
};

// dz = dy act'(z), and its sums over a slice of the rows before it is rounded.  One pass over
// dy and z; a warp takes 256 columns of every eighth row of its slice, two rows at a time, so
// that a row's partial sums stay in registers until the end.  Sums of 8 warps meet in shared
// memory, those of the slices in ffn_column_sum_kernel: in a fixed order.
//
// Measured: 4096 x 4096 with gelu 21 us, with relu 15 (6.7 TB/s, HBM's rate); 6143 x 5999, no row aligned, 54
// with gelu (HBM's are 33; issue slots 59 % busy) and as long with relu: the shifted loads bound it.  With
// loads one iteration ahead of the work, 60, and aligned relu 43 for 32.
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
        Vector8<kVec> dy[kRows], z[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int32_t row = min(r + k * kSlopeWarps, r1 - 1);
            const bool live = r + k * kSlopeWarps < r1;
            dy[k].get(p.dy + (int64_t)row * p.lddy, c, p.C, live);
            if constexpr (A != kActNone)
                z[k].get(p.z + (int64_t)row * p.ldz, c, p.C, live);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int32_t row = r + k * kSlopeWarps, at = min(row, r1 - 1);
            const uint4 y = dy[k].value(p.dy + (int64_t)at * p.lddy, c, p.C);
            const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
            Pair f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = pair_of_bf16(yw[i]);
            if constexpr (A != kActNone) {
                const uint4 x = z[k].value(p.z + (int64_t)at * p.ldz, c, p.C);
                const uint32_t zw[4] = {x.x, x.y, x.z, x.w};
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
// four vectors a lane in flight: 6143 x 4104 and 5999 x 4104 take 28 us, 7 TB/s.
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
        uint16_t *const to = j.dst + r * j.ldd;
        auto copy = [&](auto vec) {
            Vector8<decltype(vec)::value> v[kPackVectors];
#pragma unroll
            for (int k = 0; k < kPackVectors; ++k)
                v[k].get(from, c + k * kSlopeColumns, j.C, true);
#pragma unroll
            for (int k = 0; k < kPackVectors; ++k) {
                const int32_t at = c + k * kSlopeColumns;
                const uint4 q = v[k].value(from, at, j.C);
                if (at < j.C)
                    *reinterpret_cast<uint4 *>(to + at) = q;
            }
        };
        if (j.vec)
            copy(std::true_type{});
        else
            copy(std::false_type{});
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
