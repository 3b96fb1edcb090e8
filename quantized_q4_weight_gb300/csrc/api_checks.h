// api_checks.h -- argument checks that the C ABI of the operators between the
// GEMVs shares (decode_api.cu, kv8_api.cu): alignment, extents, overlap.  Host
// code only.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "../../include/qgemv.h"

namespace qg {

constexpr long long kCounterArea = 16384;  // the workspace's zero-kept head (include/qgemv.h)

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

struct Span {
    uintptr_t lo, hi;
};
inline Span span(const void *p, long long bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + static_cast<uintptr_t>(bytes)};
}
inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

inline bool type_ok(int t) { return t == QGEMV_F32 || t == QGEMV_F16 || t == QGEMV_BF16; }
inline int type_bytes(qgemv_dtype t) { return t == QGEMV_F32 ? 4 : 2; }

// From an address to the end of the last of `n` pieces of `last` elements,
// `stride` elements apart.
inline Span strided(const void *p, long long n, long long stride, long long last, int bytes)
{
    return span(p, ((n - 1) * stride + last) * bytes);
}

// n rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void *p;
    long long n, stride, width;
};

// Whether two sets of rows share bytes.  Parts of one row buffer interleave.
inline bool rows_overlap(const Rows &a, const Rows &b)
{
    const auto all = [](const Rows &r) { return span(r.p, (r.n - 1) * r.stride + r.width); };
    if (!overlap(all(a), all(b))) return false;
    // row u of b begins b0 + u * b.stride after row 0 of a
    const long long b0 = static_cast<long long>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
    // whether a row at `at` meets one of the rows first + i * stride, 0 <= i < n: the first that ends behind its begin
    const auto meets = [&](long long at, long long first, long long stride, long long n) {
        const long long i = at < first + b.width || !stride ? 0 : (at - first - b.width) / stride + 1;
        return i < n && first + i * stride < at + a.width && first + i * stride + b.width > at;
    };
    // of one stride: only the difference of the row numbers matters
    if (a.stride == b.stride) return meets(0, b0 - (a.n - 1) * b.stride, b.stride, a.n + b.n - 1);
    if (a.n > 65536) return true;  // not looked through
    for (long long t = 0; t < a.n; ++t)
        if (meets(t * a.stride, b0, b.stride, b.n)) return true;
    return false;
}

// Whether n1 x n2 pieces of d elements at i * s1 + j * s2 lie apart from one another.
inline bool pieces_apart(long long n1, long long s1, long long n2, long long s2, long long d)
{
    if ((n1 == 1 || s1 >= (n2 - 1) * s2 + d) && (n2 == 1 || s2 >= d)) return true;  // the usual orders
    if ((n2 == 1 || s2 >= (n1 - 1) * s1 + d) && (n1 == 1 || s1 >= d)) return true;
    if (n1 > 1 && s1 < d) return false;
    for (long long j = 1; j < n2; ++j) {  // a piece j steps along, against those nearest to it
        const long long at = j * s2, i = s1 ? std::min(at / s1, n1 - 1) : 0;
        if (at - i * s1 < d || (i + 1 < n1 && (i + 1) * s1 - at < d)) return false;
    }
    return true;
}

constexpr long long kMaxExtent = 1ll << 46;  // elements of a tensor: products of strides and counts stay in 64 bits

// A product of non-negative counts and strides that stays below kMaxExtent.
inline bool extent_ok(long long n, long long stride)
{
    return n >= 0 && stride >= 0 && (n == 0 || stride == 0 || n <= kMaxExtent / stride);
}

inline qgemv_status check_cache(const qgemv_kv_cache *c)
{
    if (!c || !c->k || !c->v) return QGEMV_ERR_INVALID_ARG;
    if (c->type != QGEMV_F16 && c->type != QGEMV_BF16) return QGEMV_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX || c->page_size < 1 || (c->page_size & (c->page_size - 1)) ||
        c->n_heads < 1 || c->n_heads > 4096 || c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8)
        return QGEMV_ERR_INVALID_ARG;
    if (c->page_stride < 0 || c->row_stride < 0 || c->head_stride < 0) return QGEMV_ERR_INVALID_ARG;
    if (!extent_ok(c->n_pages, c->page_stride) || !extent_ok(c->page_size, c->row_stride) ||
        !extent_ok(c->n_heads, c->head_stride))
        return QGEMV_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % 8 || c->row_stride % 8 || c->head_stride % 8)
        return QGEMV_ERR_MISALIGNED;
    return QGEMV_OK;
}

inline Span cache_span(const qgemv_kv_cache *c, const void *base)
{
    return span(base, 2 * ((c->n_pages - 1) * c->page_stride + (c->page_size - 1) * c->row_stride +
                           (c->n_heads - 1) * c->head_stride + c->head_dim));
}

inline int log2_of(int v)
{
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

}  // namespace qg
