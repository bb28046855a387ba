// CPU check of csrc/fp8_overlap.h against a count of every byte.
#include <cstdio>
#include <set>
#include <vector>

#include "fp8_overlap.h"

int main()
{
    int n = 0, clashes = 0;
    char *const base = reinterpret_cast<char *>(0x10000);
    for (int64_t R : {1, 2, 3, 5})
        for (int64_t width : {1, 2, 4, 7})
            for (int64_t lda = width; lda < width + 9; ++lda)
                for (int64_t ldb = width; ldb < width + 9; ++ldb)
                    for (int64_t d = -60; d <= 60; ++d) {
                        std::set<int64_t> bytes;
                        for (int64_t r = 0; r < R; ++r)
                            for (int64_t k = 0; k < width; ++k)
                                bytes.insert(r * lda + k);
                        bool want = false;
                        for (int64_t r = 0; r < R; ++r)
                            for (int64_t k = 0; k < width; ++k)
                                want = want || bytes.count(d + r * ldb + k);
                        if (d == 0 && (lda == ldb || R == 1))
                            want = false;
                        if (wstma::rows_clash(base, lda, base + d, ldb, R, width) != want) {
                            std::printf("R %d width %d lda %d ldb %d d %d: not %d\n", (int)R, (int)width, (int)lda,
                                        (int)ldb, (int)d, (int)want);
                            return 1;
                        }
                        ++n;
                        clashes += want;
                    }
    // pitches and rows whose products pass 64 bits
    const int64_t far = int64_t(1) << 39, many = int64_t(1) << 31;
    if (!wstma::rows_clash(base, far, base + 2, far, many, 8) || wstma::rows_clash(base, far, base + 8, far, many, 8))
        return 2;
    std::printf("%d layouts, %d of them clash\n", n, clashes);
    return 0;
}
