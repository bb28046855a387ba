// CPU check of the 8-bit product's work split (host functions of fp8_gemm.cuh): every
// (tile, k-block) is one cluster's, a cluster leaves at most one partial and before
// it waits for any, and an owner's list of pieces is exactly the ranges that
// start inside its tile.
#include <cstdio>
#include <map>
#include <set>
#include <utility>
#include <vector>

#include "fp8_gemm.cuh"

using namespace wstma;

static int check(int32_t tiles, int32_t KB, int32_t C, int32_t sk)
{
    Fp8GemmParams p = {};
    p.num_k_blocks = KB;
    p.num_tiles = tiles;
    p.sk_tiles = sk;
    p.sk_units = (int64_t)sk * KB;
    std::map<std::pair<int, int>, int> seen;
    std::map<int, std::set<int>> pieces;  // tile -> clusters that leave a partial of it
    std::map<int, int> owner;
    for (int c = 0; c < C; ++c) {
        Fp8Work w;
        w.init(p, c, C);
        Fp8Item it;
        int partials = 0, owned = 0;
        while (w.next(it)) {
            if (it.kb0 < 0 || it.kb1 > KB || it.kb0 >= it.kb1 || it.tile < 0 || it.tile >= tiles)
                return 1;
            for (int k = it.kb0; k < it.kb1; ++k)
                if (seen[{it.tile, k}]++)
                    return 2;
            if (it.kb0 > 0) {
                if (++partials > 1 || owned)
                    return 3;
                pieces[it.tile].insert(c);
            } else if (it.kb1 < KB) {
                if (owner.count(it.tile))
                    return 4;
                owner[it.tile] = c;
                ++owned;
            }
        }
    }
    if ((int64_t)seen.size() != (int64_t)tiles * KB)
        return 5;
    for (auto &o : owner) {
        const int last = fp8_range_of(p.sk_units, C, (int64_t)(o.first + 1) * KB - 1);
        std::set<int> listed;
        for (int j = o.second + 1; j <= last; ++j)
            if (fp8_range_holds(p.sk_units, C, j))
                listed.insert(j);
        if (listed != pieces[o.first])
            return 6;
        pieces.erase(o.first);
    }
    return pieces.empty() ? 0 : 7;
}

int main()
{
    int n = 0;
    for (int32_t C : {1, 2, 3, 8, 19, 76, 152})
        for (int32_t KB : {1, 2, 3, 5, 32, 33, 64})
            for (int32_t tiles = 1; tiles < 3 * C + 3; tiles += tiles < 12 ? 1 : 7) {
                // the last partial wave, or every tile where they do not fill one
                std::vector<std::pair<int32_t, int32_t>> splits = {{C, tiles % C}};
                if (tiles < C)
                    for (int32_t c = tiles + 1; c <= C; c += c < 12 ? 1 : 13)
                        splits.push_back({c, tiles});
                splits.push_back({tiles < C ? tiles : C, 0});
                for (auto [clusters, sk] : splits) {
                    const int rc = check(tiles, KB, clusters, sk);
                    if (rc) {
                        std::printf("tiles %d KB %d clusters %d sk %d: %d\n", tiles, KB, clusters, sk, rc);
                        return 1;
                    }
                    ++n;
                }
                // clusters of c CTAs to a tile
                for (int32_t c = 2; c <= 8 && c <= KB; ++c) {
                    const int rc = check(tiles, KB, tiles * c, tiles);
                    if (rc) {
                        std::printf("tiles %d KB %d cluster %d: %d\n", tiles, KB, c, rc);
                        return 1;
                    }
                    ++n;
                }
            }
    std::printf("%d splits\n", n);
    return 0;
}
