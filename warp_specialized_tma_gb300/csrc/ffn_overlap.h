// Whether what a call writes lies over what it reads, for matrices of different shapes.
#pragma once

#include <stdint.h>

namespace wstma {

// Bytes that a call reads or writes: rows of `width` bytes, `ld` bytes apart.
struct Span {
    const void *p;
    int64_t ld, width, rows;
    bool same_allowed = false;  // with the first result
};

// Whether two spans share a byte; spans of different pitches that reach over each other count as sharing.
inline bool touch(const Span &a, const Span &b)
{
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1)
        return false;
    using Wide = __int128;
    const Wide at_a = (Wide) reinterpret_cast<uintptr_t>(a.p), at_b = (Wide) reinterpret_cast<uintptr_t>(b.p);
    if (at_a + (Wide)(a.rows - 1) * a.ld + a.width <= at_b || at_b + (Wide)(b.rows - 1) * b.ld + b.width <= at_a)
        return false;
    if (a.rows == 1 || b.rows == 1 || a.ld != b.ld)
        return true;
    // one pitch: b's rows start d bytes behind a's, or behind the row before
    Wide d = (at_b - at_a) % a.ld;
    if (d < 0)
        d += a.ld;
    return d < a.width || d + b.width > a.ld;
}

}  // namespace wstma
