// arrays.h -- checks of the arrays that an entry point is given.
#pragma once

#include <cstdint>

#include "internal.h"

namespace osr {

inline bool known_dtype(int32_t d)
{
    return d == ADAMW_DTYPE_F32 || d == ADAMW_DTYPE_BF16 || d == ADAMW_DTYPE_F16;
}
inline size_t size_of(int32_t d) { return d == ADAMW_DTYPE_F32 ? 4 : 2; }

inline int check_array(const void* p, size_t size, bool optional, const char* name)
{
    if (!p && !optional)
        return fail(ADAMW_EINVAL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % size)
        return fail(ADAMW_EINVAL, "%s is not %d-byte aligned", name, int(size));
    return ADAMW_OK;
}

inline int check_rows(const void* p, int64_t stride, int64_t rows, int32_t cols, size_t size,
                      const char* name)
{
    if (const int rc = check_array(p, size, rows == 0, name))
        return rc;
    if (stride < cols && rows > 1)
        return fail(ADAMW_EINVAL, "%s: rows %lld apart, of %d elements", name, (long long)stride,
                    cols);
    return ADAMW_OK;
}

// `rows` pieces of `bytes` each, `stride` bytes apart (0 for a single one); a
// vector is one piece.
struct Pieces {
    uintptr_t begin;
    int64_t stride, rows, bytes;
    const char* name;
};
inline Pieces rows_of(const void* p, int64_t stride, int64_t rows, int64_t cols, size_t size,
                      const char* name)
{
    return Pieces{reinterpret_cast<uintptr_t>(p), rows > 1 ? stride * int64_t(size) : 0, rows,
                  cols * int64_t(size), name};
}
inline Pieces vector_of(const void* p, int64_t n, size_t size, const char* name)
{
    return Pieces{reinterpret_cast<uintptr_t>(p), 0, p && n ? 1 : 0, n * int64_t(size), name};
}

// Whether a piece of `bytes` at `begin` shares a byte with some row of b.
inline bool touches(uintptr_t begin, int64_t bytes, const Pieces& b)
{
    // the last row that starts before the piece's end
    const int64_t before = int64_t(begin - b.begin) + bytes - 1;
    if (before < 0)
        return false;
    int64_t j = b.rows > 1 ? before / b.stride : 0;
    j = j < b.rows ? j : b.rows - 1;
    return j * b.stride + b.bytes > int64_t(begin - b.begin);
}
// Whether any byte belongs to both.  Rows of two arrays may lie between one
// another (columns of one matrix), so the ranges alone do not say.
inline bool overlap(const Pieces& a, const Pieces& b)
{
    if (a.rows == 0 || b.rows == 0)
        return false;
    const uintptr_t a_end = a.begin + uintptr_t((a.rows - 1) * a.stride + a.bytes);
    const uintptr_t b_end = b.begin + uintptr_t((b.rows - 1) * b.stride + b.bytes);
    if (a.begin >= b_end || b.begin >= a_end)
        return false;
    const Pieces &few = a.rows < b.rows ? a : b, &many = a.rows < b.rows ? b : a;
    // rows as far apart as the other's lie alike to it: the first that is
    // within the other's range, and the one before it, stand for all
    const bool alike = few.rows > 1 && few.stride == many.stride;
    int64_t i = 0, end = few.rows;
    if (alike) {
        const int64_t ahead = int64_t(many.begin - few.begin);
        i = ahead > 0 ? ahead / few.stride : 0;
        end = i + 2 < end ? i + 2 : end;
    }
    for (; i < end; ++i)
        if (touches(few.begin + uintptr_t(i * few.stride), few.bytes, many))
            return true;
    return false;
}
// Outputs share no byte with an input or with one another.
template <int kOut, int kIn>
int check_apart(const Pieces (&out)[kOut], const Pieces (&in)[kIn])
{
    for (int i = 0; i < kOut; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return fail(ADAMW_EINVAL, "%s overlaps %s", out[i].name, out[j].name);
        for (int j = 0; j < kIn; ++j)
            if (overlap(out[i], in[j]))
                return fail(ADAMW_EINVAL, "%s overlaps %s", out[i].name, in[j].name);
    }
    return ADAMW_OK;
}

}  // namespace osr
