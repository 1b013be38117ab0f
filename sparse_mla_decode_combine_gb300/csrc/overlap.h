// overlap.h -- whether arrays that a call reads and writes share bytes.  Host code of the argument checks.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cstdlib>
#include <initializer_list>

namespace dsv4 {

// `rows` rows of `width` bytes, `stride` bytes apart (none behind a null pointer)
struct Rows {
    const void *at;
    int64_t rows, stride, width;
};
inline Rows bytes(const void *at, int64_t n) { return Rows{at, 1, n, n}; }
inline Rows joined(const Rows &a) { return a.rows > 1 && a.stride == a.width ? bytes(a.at, a.rows * a.width) : a; }

// Rows that lie between the other array's, as in a buffer that holds both side by side, do not share a byte with it; where the
// strides of both differ that is not looked for, and what reaches into the other array's span counts as shared.
inline bool share(const Rows &x, const Rows &y)
{
    const Rows a = joined(x), b = joined(y);
    if (a.at == nullptr || b.at == nullptr || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0)
        return false;
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));
    const int64_t na = (a.rows - 1) * a.stride + a.width, nb = (b.rows - 1) * b.stride + b.width;
    if (d >= na || -d >= nb)
        return false;
    const int64_t s = a.rows > 1 ? a.stride : b.stride;
    if ((a.rows > 1 && b.rows > 1 && a.stride != b.stride) || a.width >= s || b.width >= s)
        return true;
    const int64_t k = d / s - (d % s < 0 ? 1 : 0), r = d - k * s;   // row j of b begins r bytes into row j + k of a
    return (r < a.width && k < a.rows && -k < b.rows) || (r + b.width > s && k + 1 < a.rows && -(k + 1) < b.rows);
}

inline bool share(const Rows &a, std::initializer_list<Rows> others)
{
    for (const Rows &o : others)
        if (share(a, o))
            return true;
    return false;
}

}  // namespace dsv4
