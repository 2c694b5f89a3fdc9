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

// Rows of `bytes` bytes at every combination of three strides (bytes): a paged cache's pages, slots and heads.
struct CacheRows {
    const void *base;
    int64_t bytes;
    struct Dim {
        int64_t stride, count;
    } dim[3];
    bool empty() const { return !base || dim[0].count * dim[1].count * dim[2].count == 0; }
    bool sound() const
    {
        for (const Dim &d : dim)
            if (d.count > 1 && d.stride < 0)
                return false;
        return true;
    }
    // Whether a dimension of more than one has no stride (rows that are all the same).
    bool flat() const
    {
        for (const Dim &d : dim)
            if (d.count > 1 && d.stride == 0)
                return true;
        return false;
    }
    bool aligned(int64_t to) const
    {
        if (empty())
            return true;
        for (const Dim &d : dim)
            if (d.count > 1 && d.stride % to != 0)
                return false;
        return dep::aligned(base, (uintptr_t)to);
    }
    // All of it, as one row.
    Rows span() const
    {
        int64_t n = bytes;
        for (const Dim &d : dim)
            n += (d.count - 1) * d.stride;
        return empty() ? Rows{base, 0, 0, 0} : Rows{base, n, n, 1};
    }
    // The dimensions of more than one by falling stride; the number of them.
    int sorted(Dim (&out)[3]) const
    {
        int n = 0;
        for (const Dim &d : dim)
            if (d.count > 1) {
                int i = n++;
                for (; i > 0 && out[i - 1].stride < d.stride; --i)
                    out[i] = out[i - 1];
                out[i] = d;
            }
        return n;
    }
    // Whether no two rows share a byte, told by each stride being as long as all that lies within it.
    bool distinct() const
    {
        if (empty())
            return true;
        Dim d[3];
        int64_t inner = bytes;
        for (int i = sorted(d) - 1; i >= 0; --i) {
            if (d[i].stride < inner)
                return false;
            inner += (d[i].count - 1) * d[i].stride;
        }
        return true;
    }
};

namespace detail {
// Whether rows of `bytes` bytes, `delta` apart but for whole steps of the nested strides d[i..n), can meet.
inline bool meet(int64_t delta, int64_t bytes, const CacheRows::Dim *d, int n)
{
    if (n == 0)
        return delta < bytes && -delta < bytes;
    const int64_t k = delta / d->stride;
    for (int64_t j = k - 1; j <= k + 1; ++j)
        if (j > -d->count && j < d->count && meet(delta - j * d->stride, bytes, d + 1, n - 1))
            return true;
    return false;
}
}  // namespace detail

// Whether two caches, each of distinct rows, share a byte.  Of the same strides and counts they may interleave
// (keys and values of one tensor); otherwise only the spans are compared.
inline bool overlap(const CacheRows &a, const CacheRows &b)
{
    if (a.empty() || b.empty() || !overlap(a.span(), b.span()))
        return false;
    CacheRows::Dim d[3], e[3];
    const int n = a.sorted(d);
    if (a.bytes != b.bytes || b.sorted(e) != n)
        return true;
    for (int i = 0; i < n; ++i)
        if (d[i].stride != e[i].stride || d[i].count != e[i].count)
            return true;
    return detail::meet((int64_t)(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base)), a.bytes, d, n);
}

}  // namespace dep
