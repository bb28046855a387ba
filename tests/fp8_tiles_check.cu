// CPU check of the 8-bit product's tile order (host functions of fp8_gemm.cuh): every tile
// index is one tile inside the grid of tiles, whatever the band's height asks for, up to
// the largest numbers of tiles.
#include <cstdio>
#include <set>
#include <utility>

#include "fp8_gemm.cuh"

using namespace wstma;

static int bad(const char *what, int64_t rows, int64_t cols, int64_t group, int64_t t)
{
    std::printf("%s: %lld x %lld tiles, bands of %lld, tile %lld\n", what, (long long)rows, (long long)cols,
                (long long)group, (long long)t);
    return 1;
}

int main()
{
    int n = 0;
    for (int64_t asked : {0, 1, 2, 7, 8, 64, 1024})
        for (int64_t rows : {1, 2, 3, 9, 16, 100, 1 << 20, 1 << 26})
            for (int64_t cols : {1, 2, 5, 31, 1 << 16, 1 << 22, 1 << 26}) {
                if (rows * cols > 0x7FFFFFFFLL)
                    continue;
                Fp8GemmParams p = {};
                p.num_row_tiles = (int32_t)rows;
                p.num_col_tiles = (int32_t)cols;
                p.num_tiles = (int32_t)(rows * cols);
                p.raster_group = fp8_raster_group(asked, rows);
                const int64_t tiles = rows * cols, step = tiles < 4096 ? 1 : tiles / 1000;
                std::set<std::pair<int, int>> seen;
                for (int64_t t = 0; t < tiles; t += step) {
                    const TileCoord c = fp8_tile_coord((int32_t)t, p);
                    if (c.mb < 0 || c.mb >= rows || c.nb < 0 || c.nb >= cols)
                        return bad("outside", rows, cols, asked, t);
                    if (!seen.insert({c.mb, c.nb}).second)
                        return bad("twice", rows, cols, asked, t);
                }
                ++n;
            }
    std::printf("%d orders\n", n);
    return 0;
}
