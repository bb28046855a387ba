// Whether the rows that a kernel writes lie partly over rows that it reads.
#pragma once

#include <stdint.h>

namespace wstma {

// Two matrices of R rows of `width` bytes, at pitches of lda and ldb bytes (at least `width`):
// true if a byte belongs to both and they are not the same rows, one for one.  A kernel that
// reads a row before it writes that row may have them the same; a row over part of
// another is read after or before it was written, as it happens.
inline bool rows_clash(const void *a, int64_t lda, const void *b, int64_t ldb, int64_t R, int64_t width)
{
    using Wide = __int128;  // a pitch times a number of rows
    const Wide at_a = (Wide) reinterpret_cast<uintptr_t>(a), at_b = (Wide) reinterpret_cast<uintptr_t>(b);
    if (R < 1 || width < 1 || (at_a == at_b && (lda == ldb || R == 1)))
        return false;
    const Wide end_a = at_a + (Wide)(R - 1) * lda + width, end_b = at_b + (Wide)(R - 1) * ldb + width;
    if (end_a <= at_b || end_b <= at_a)
        return false;
    // row j of b lies over row i of a or the next, i the last that starts at or before it
    const auto over = [&](Wide j) {
        const Wide from = at_b + j * ldb - at_a;
        const Wide i = from >= 0 ? from / lda : -1;
        return (i >= 0 && i < R && from - i * lda < width) || (i + 1 < R && (i + 1) * lda - from < width);
    };
    if (lda != ldb) {
        for (int64_t j = 0; j < R; ++j)
            if (over(j))
                return true;
        return false;
    }
    // one pitch: every row of b lies alike, but for a's first row and last
    const Wide d = at_b - at_a;
    const Wide k = d >= 0 ? d / lda : -((-d + lda - 1) / lda), m = d - k * lda;  // floor and rest
    return (m < width && k < R && -k < R) || (m + width > lda && k + 1 < R && -(k + 1) < R);
}

}  // namespace wstma
