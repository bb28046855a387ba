// CPU check of the plans that the feed-forward products choose for themselves (choose_tiling of
// ffn_api.cu, for a GPU of 152 SMs and 76 pairs): for sums of any length, empty ones too, every (tile,
// k-block) of a plan is one cluster's, and where the sum is empty every tile is still visited.
// The kernels' side is stubbed; nothing is launched.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../warp_specialized_tma_gb300/csrc/ffn_api.cu"
#include "ffn_gemm.cuh"

namespace wstma {
static const void *const nothing = nullptr;
const void *ffn_plain_fn(int, bool) { return nothing; }
const void *ffn_plain_segments_fn(int, bool) { return nothing; }
const void *ffn_gated_fn(int, bool) { return nothing; }
const void *ffn_gated_codes_fn(int) { return nothing; }
const void *ffn_grad_fn(int, bool) { return nothing; }
const void *ffn_together_fn(int) { return nothing; }
const void *ffn_together_segments_fn(int) { return nothing; }
uint32_t *ffn_status_word() { return nullptr; }
int64_t ffn_stream_rows(int) { return 0; }
int launch_ffn_stream(FfnStreamParams &, int, cudaStream_t) { return 1; }
int64_t ffn_stream_back_columns(int) { return 0; }
int launch_ffn_stream_back(FfnStreamBackParams &, int, int, cudaStream_t) { return 1; }
int launch_ffn_pack(FfnPackJobs &, int, cudaStream_t) { return 1; }
int ffn_slope_slices(int64_t, int64_t, int) { return 1; }
int launch_ffn_slope(const FfnSlopeParams &, int, cudaStream_t) { return 1; }
}  // namespace wstma

static Device gb300()
{
    Device d;
    d.index = 0;
    d.sms = 152;
    d.max_pairs = 76;
    d.max_smem = 232448;
    return d;
}

// Whether the clusters of plan `t` of x visit every k-block of every tile once: what they walk is added up.
static bool covers(const Product &x, const Tiling &t)
{
    const Sides s = sides_of(x, t);
    FfnParams p = {};
    p.num_tiles = (int32_t)(s.row_tiles * s.col_tiles);
    p.num_k_blocks = (int32_t)k_blocks_of(x);
    p.sk_tiles = (int32_t)t.sk_tiles;
    p.sk_units = t.sk_tiles * p.num_k_blocks;
    p.cluster = t.cluster;
    // pieces of a tile are contiguous, so that their lengths and ends tell: sums of kb1 - kb0 and of
    // kb1^2 - kb0^2 are the whole tile's only if nothing is left out, or twice there in place of another
    std::vector<int64_t> length(p.num_tiles), squares(p.num_tiles), visits(p.num_tiles);
    for (int64_t c = 0; c < t.clusters; ++c) {
        FfnWork w;
        w.init(p, (int32_t)c, (int32_t)t.clusters);
        FfnItem it;
        while (w.next(it)) {
            if (it.tile < 0 || it.tile >= p.num_tiles)
                return false;
            ++visits[it.tile];
            length[it.tile] += it.kb1 - it.kb0;
            squares[it.tile] += (int64_t)it.kb1 * it.kb1 - (int64_t)it.kb0 * it.kb0;
        }
    }
    const int64_t KB = p.num_k_blocks;
    for (int32_t i = 0; i < p.num_tiles; ++i)
        if (visits[i] < 1 || length[i] != KB || squares[i] != KB * KB || (KB == 0 && visits[i] != 1))
            return false;
    return true;
}

static int checked = 0, empty = 0, split = 0;

static bool check(const Product &x)
{
    const Device d = gb300();
    Tiling t;
    double cost = 0.0;
    if (!choose_tiling(d, x, t, cost))
        return true;  // the options allow no tiling
    ++checked;
    empty += x.K == 0;
    split += t.sk_tiles > 0;
    Plan pl;
    std::memset(&pl, 0, sizeof(pl));
    if (covers(x, t) && plan_tiles(x, t, pl) == FFN_OK)
        return true;
    std::printf("M %lld N %lld K %lld form %d epilogue %d save %d residual %d: %d x %d%s, %lld clusters, %lld tiles split\n",
                (long long)x.M, (long long)x.N, (long long)x.K, x.form, x.epilogue, x.p.save, x.p.aux[0].p != nullptr,
                t.cta_group, t.width, t.transposed ? " transposed" : "", (long long)t.clusters, (long long)t.sk_tiles);
    return false;
}

static Product product(int64_t M, int64_t N, int64_t K, int kind)
{
    static const uint8_t there = 0;
    Product x;
    x.M = M, x.N = N, x.K = K;
    switch (kind) {
    case 0: break;
    case 1: x.p.save = 1, x.p.aux[0].p = &there; break;
    case 2: x.form = kDual, x.epilogue = kFfnGated; break;
    case 3: x.form = kDual, x.epilogue = kFfnGated, x.p.save = 1; break;
    case 4: x.form = kDual, x.epilogue = kFfnGated, x.p.save = 2, x.no_split = x.not_transposed = true; break;
    case 5: x.b_mn = true, x.epilogue = kFfnGrad, x.p.aux[0].p = x.p.aux[1].p = &there; break;
    case 6:
        x.b_mn = true, x.epilogue = kFfnGrad, x.p.aux[0].p = x.p.aux[1].p = &there;
        x.p.aux[0].scales = x.p.aux[1].scales = &there;
        break;
    case 7: x.form = kSum, x.b_mn = true; break;
    case 8: x.form = kStack, x.a_mn = x.b_mn = true; break;
    default: x.a_mn = x.b_mn = true, x.fp32 = true; break;
    }
    return x;
}

int main()
{
    bool ok = true;
    // plans of empty sums that shared out tiles which nobody then visited
    const int64_t known[][3] = {{300, 8192, 0}, {8192, 300, 0}, {4096, 520, 0}, {281, 12248, 0}, {1675, 1886, 0}};
    for (const auto &k : known)
        for (int kind = 0; kind < 10; ++kind)
            ok = check(product(k[0], k[1], k[2], kind)) && ok;
    ffn_set_option(FFN_OPT_TRANSPOSED, 2);
    ok = check(product(1935, 13017, 0, 1)) && ok;
    std::mt19937 rng(1);
    auto size = [&](double top) { return (int64_t)std::exp(std::uniform_real_distribution<double>(0.0, std::log(top))(rng)); };
    auto pick = [&](int n) { return (int64_t)(rng() % (unsigned)n); };
    for (int i = 0; i < 4000; ++i) {
        const bool plain = pick(3) > 0;
        ffn_set_option(FFN_OPT_CTA_GROUP, plain ? 0 : pick(3));
        ffn_set_option(FFN_OPT_TRANSPOSED, plain ? 0 : pick(3));
        ffn_set_option(FFN_OPT_WIDTH, plain ? 0 : 32 * pick(9));
        ffn_set_option(FFN_OPT_SPLIT, plain ? 1 : pick(3));
        const int64_t M = size(16384), N = size(16384), K = pick(3) ? size(20000) : 0;
        ok = check(product(M, N, K, (int)pick(10))) && ok;
    }
    // and no plan leaves a tile to pieces of an empty sum, whoever made it
    Product x = product(300, 8192, 0, 3);
    Tiling t;
    t.cta_group = 1, t.width = 128, t.sk_tiles = 40, t.clusters = 152;
    Plan pl;
    std::memset(&pl, 0, sizeof(pl));
    if (plan_tiles(x, t, pl) == FFN_OK)
        ok = false, std::printf("a plan splits an empty sum\n");
    if (!ok)
        return 1;
    std::printf("%d plans, %d of empty sums, %d with split tiles: covered\n", checked, empty, split);
    return 0;
}
