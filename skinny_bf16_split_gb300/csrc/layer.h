// layer.h -- argument checks shared by the operators around the projections.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace dep {

inline bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// `count` rows of `bytes` bytes each, `stride` bytes apart (count 0: nothing).
struct Rows {
    const void *base;
    int64_t bytes, stride, count;
    bool aligned(int64_t to) const
    {
        return count == 0 || (dep::aligned(base, (uintptr_t)to) && (count == 1 || stride % to == 0));
    }
};

// Whether two sets of rows share a byte.  Rows of one stride may interleave (column
// slices of one packed matrix); of sets with different strides only the spans are compared.
inline bool overlap(const Rows &a, const Rows &b)
{
    if (a.count == 0 || b.count == 0)
        return false;
    const int64_t a0 = (int64_t)reinterpret_cast<uintptr_t>(a.base), b0 = (int64_t)reinterpret_cast<uintptr_t>(b.base);
    const int64_t a1 = a0 + (a.count - 1) * a.stride + a.bytes, b1 = b0 + (b.count - 1) * b.stride + b.bytes;
    if (a1 <= b0 || b1 <= a0)
        return false;
    if (a.stride != b.stride || a.count == 1 || b.count == 1)
        return true;
    const int64_t d = ((b0 - a0) % a.stride + a.stride) % a.stride;
    return d < a.bytes || d + b.bytes > a.stride;
}

}  // namespace dep
