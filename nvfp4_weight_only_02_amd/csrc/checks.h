// Argument checks of the fused operators' C entries: alignment, element types
// and whether what a call writes overlaps what it reads.
#ifndef NVFP4_CHECKS_H
#define NVFP4_CHECKS_H

#include <stddef.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace {

inline bool is_aligned(const void *p, size_t a)
{
    return ((uintptr_t)p % a) == 0;
}

// Memory an argument covers, in bytes: an array, or a matrix whose rows of
// `width` bytes lie `ld` apart.
struct Region {
    const void *p;
    size_t rows, ld, width;
    size_t span() const { return rows ? (rows - 1) * ld + width : 0; }
};

inline Region array(const void *p, size_t bytes)
{
    return {p, p && bytes ? 1u : 0u, 0, bytes};
}

inline Region matrix(const void *p, int n, int64_t ld, int64_t cols, int size)
{
    return {p, p && n > 0 ? (size_t)n : 0u, (size_t)ld * size, (size_t)cols * size};
}

// Rows that take turns in memory with one stride (neighbouring columns of one
// buffer) lie apart although their spans do not.
inline bool overlap(const Region &a, const Region &b)
{
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (!a.rows || !b.rows || x >= y + b.span() || y >= x + a.span())
        return false;
    const size_t ld = a.rows > 1 ? a.ld : b.ld;   // one row fits any stride
    if ((a.rows == 1 && b.rows == 1) || (a.rows > 1 && b.rows > 1 && a.ld != b.ld) || a.width > ld || b.width > ld)
        return true;
    const size_t from = (y % ld + ld - x % ld) % ld;   // b's first column, in a's rows
    return from < a.width || from + b.width > ld;
}

inline bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    return overlap(array(a, an), array(b, bn));
}

// Whether an output overlaps an argument.
template <int I>
bool any_overlap(const Region &out, const Region (&args)[I])
{
    for (const Region &a : args)
        if (overlap(out, a))
            return true;
    return false;
}

inline bool valid_dtype(int d)
{
    return d == NVFP4_DTYPE_F32 || d == NVFP4_DTYPE_BF16;
}

inline int dtype_size(int d)
{
    return d == NVFP4_DTYPE_F32 ? 4 : 2;
}

}  // namespace

#endif  // NVFP4_CHECKS_H
