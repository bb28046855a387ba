// CPU check of the feed-forward products' work split and tile order (host functions of
// ffn_gemm.cuh): every (tile, k-block) is one cluster's, a cluster leaves at most one partial and
// before it waits for any, an owner's list of pieces is exactly the ranges that start inside its
// tile, those ranges are of clusters with lower indices (in the cluster form: of the owner's own cluster),
// and every tile has a place of its own.
#include <cstdio>
#include <map>
#include <set>
#include <utility>

#include "ffn_gemm.cuh"

using namespace wstma;

static int check(int32_t tiles, int32_t KB, int32_t C, int32_t sk, int32_t cluster = 1)
{
    FfnParams p = {};
    p.cluster = cluster;
    p.num_k_blocks = KB;
    p.num_tiles = tiles;
    p.sk_tiles = sk;
    p.sk_units = (int64_t)sk * KB;
    std::map<std::pair<int, int>, int> seen;
    std::map<int, std::set<int>> pieces;  // tile -> ranges that leave a partial of it
    std::map<int, int> owner;             // tile -> its owner's range
    for (int c = 0; c < C; ++c) {
        FfnWork w;
        w.init(p, c, C);
        const int32_t range = ffn_range_at(p, C, c);
        if (ffn_range_at(p, C, range) != c)
            return 8;
        FfnItem it;
        int partials = 0, owned = 0;
        while (w.next(it)) {
            if (it.kb0 < 0 || it.kb1 > KB || (it.kb0 >= it.kb1 && KB > 0) || it.tile < 0 || it.tile >= tiles)
                return 1;
            if (KB == 0 && seen[{it.tile, 0}]++)
                return 2;
            for (int k = it.kb0; k < it.kb1; ++k)
                if (seen[{it.tile, k}]++)
                    return 2;
            if (it.kb0 > 0) {
                if (++partials > 1 || owned)
                    return 3;
                pieces[it.tile].insert(range);
            } else if (it.kb1 < KB) {
                if (owner.count(it.tile))
                    return 4;
                owner[it.tile] = range;
                ++owned;
            }
        }
    }
    if ((int64_t)seen.size() != (int64_t)tiles * (KB ? KB : 1))
        return 5;
    for (auto &o : owner) {
        const int last = ffn_range_of(p.sk_units, C, (int64_t)(o.first + 1) * KB - 1);
        std::set<int> listed;
        for (int j = o.second + 1; j <= last; ++j)
            if (ffn_range_holds(p.sk_units, C, j))
                listed.insert(j);
        if (listed != pieces[o.first])
            return 6;
        const int own = ffn_range_at(p, C, o.second);
        for (int j : listed) {
            const int other = ffn_range_at(p, C, j);
            if (cluster > 1 ? own % cluster != 0 || other / cluster != own / cluster : other >= own)
                return 9;
        }
        pieces.erase(o.first);
    }
    return pieces.empty() ? 0 : 7;
}

static int check_order(int32_t rows, int32_t cols, int32_t band)
{
    FfnParams p = {};
    p.num_row_tiles = rows;
    p.num_col_tiles = cols;
    p.raster_group = band < rows ? band : rows;
    p.band_tiles = ffn_band_tiles(p.raster_group, cols);
    std::set<std::pair<int, int>> seen;
    for (int32_t t = 0; t < rows * cols; ++t) {
        const FfnTile c = ffn_tile_coord(t, p);
        if (c.row < 0 || c.row >= rows || c.col < 0 || c.col >= cols || !seen.insert({c.row, c.col}).second)
            return 1;
    }
    return 0;
}

int main()
{
    int n = 0;
    for (int C : {1, 2, 3, 20, 76, 152})
        for (int KB : {0, 1, 2, 7, 94})
            for (int tiles : {1, 2, 19, 76, 77, 152, 153, 400}) {
                std::set<int> splits = {0};
                const int sk = tiles % C;
                if (sk && KB)
                    splits.insert(sk);
                if (tiles < C && KB)
                    splits.insert(tiles);
                if (tiles * 4 <= C && KB >= 4)  // a tile per cluster of four CTAs
                    if (const int e = check(tiles, KB, tiles * 4, tiles, 4)) {
                        std::printf("cluster form: tiles %d KB %d: %d\n", tiles, KB, e);
                        return 1;
                    }
                for (int s : splits) {
                    if (const int e = check(tiles, KB, C, s)) {
                        std::printf("tiles %d KB %d C %d sk %d: %d\n", tiles, KB, C, s, e);
                        return 1;
                    }
                    ++n;
                }
            }
    for (int rows : {1, 2, 7, 8, 9, 64})
        for (int cols : {1, 3, 31})
            for (int band : {1, 8, 1024})
                if (check_order(rows, cols, band)) {
                    std::printf("order: %d x %d in bands of %d\n", rows, cols, band);
                    return 1;
                }
    if (ffn_band_tiles(1024, 1 << 27) != 0x7FFFFFFFu || ffn_band_tiles(8, 31) != 248u)
        return 1;
    std::printf("%d splits\n", n);
    return 0;
}
