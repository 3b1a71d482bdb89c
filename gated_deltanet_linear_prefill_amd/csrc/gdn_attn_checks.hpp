// gdn_attn_checks.hpp -- host-side checks shared by the entry points of the cache and of attention
// (not part of the C ABI): types, strides, caches and their address ranges.
#pragma once

#include <math.h>

#include "gdn_checks.hpp"

namespace gdn {

inline bool attn_d(int32_t d)
{
    return d == 64 || d == 128 || d == 256;
}

inline bool attn_dtype(int32_t t)
{
    return t == GDN_F32 || t == GDN_BF16;
}

// Finite also in the units of exp2, which the kernels use.
inline bool attn_scale(float scale)
{
    return isfinite(scale * 1.4426950408889634f);
}

inline size_t elem(int32_t t)
{
    return t == GDN_F32 ? 4 : t == GDN_BF16 ? 2 : 1;
}

// A [rows][heads][d] tensor with strides: its extent in elements (0 for no rows), or false
// when the strides are not usable (not positive, not multiples of 16 bytes, too large for the
// kernels' 32-bit offsets within a tile) or tokens and heads would share elements.
inline bool strided(int64_t rows, int32_t heads, int32_t d, int64_t token, int64_t head, int32_t dtype,
             int64_t* extent)
{
    const int64_t step = 16 / (int64_t)elem(dtype);
    if (token <= 0 || head <= 0 || token % step || head % step) return false;
    if (token >= (INT64_C(1) << 22) || head >= (INT64_C(1) << 46)) return false;
    if (head < d || token < d) return false;
    int64_t a, b;
    if (!mul_ok(heads - 1, head, &b)) return false;
    *extent = 0;
    if (rows == 0) return true;
    if (!mul_ok(rows - 1, token, &a)) return false;
    // token-major (a token holds all its heads) or head-major (a head holds all its tokens)
    const bool token_major = rows == 1 || token >= b + d;
    const bool head_major = heads == 1 || head >= a + d;
    if (!token_major && !head_major) return false;
    if (a > (INT64_C(1) << 58) || b > (INT64_C(1) << 58)) return false;
    *extent = a + b + d;
    return true;
}

// Sizes and pools of a cache; *pool the elements of one pool.
inline gdn_status check_cache(const gdn_kv_cache* c, int32_t dtype, int64_t* pool)
{
    if (!c) return GDN_ERR_NULL;
    if (c->n < 0 || c->num_pages < 0 || c->max_pages < 0 || c->h_kv <= 0 || c->d <= 0 ||
        c->page_size <= 0)
        return GDN_ERR_SHAPE;
    if (c->n >= (INT64_C(1) << 31) || c->num_pages >= (INT64_C(1) << 31) ||
        c->max_pages >= (INT64_C(1) << 31))
        return GDN_ERR_SHAPE;
    if (!attn_d(c->d) || !attn_dtype(dtype)) return GDN_ERR_UNSUPPORTED;
    if (c->store != dtype && c->store != GDN_FP8) return GDN_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return GDN_ERR_UNSUPPORTED;
    int64_t rows, a;
    if (!mul_ok(c->num_pages, c->page_size, &a) || !mul_ok(a, c->h_kv, &rows) ||
        !mul_ok(rows, c->d, pool) || *pool > (INT64_C(1) << 58))
        return GDN_ERR_SHAPE;
    if (!mul_ok(c->max_pages, c->page_size, &a) || a >= (INT64_C(1) << 31)) return GDN_ERR_SHAPE;
    return GDN_OK;
}

inline gdn_status cache_pointers(const gdn_kv_cache* c)
{
    const bool fp8 = c->store == GDN_FP8;
    if (c->num_pages > 0 && (!c->k || !c->v || (fp8 && (!c->k_scale || !c->v_scale))))
        return GDN_ERR_NULL;
    if (c->max_pages > 0 && !c->page_table) return GDN_ERR_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4)) return GDN_ERR_ALIGN;
    if (fp8 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))) return GDN_ERR_ALIGN;
    return GDN_OK;
}

// The cache's device ranges: k, v, their scales, the page table.
struct CacheRanges {
    Range r[5];
    CacheRanges(const gdn_kv_cache* c, int64_t pool)
    {
        const int64_t rows = c->store == GDN_FP8 ? pool / c->d : 0;
        r[0] = range_of(c->k, pool, elem(c->store));
        r[1] = range_of(c->v, pool, elem(c->store));
        r[2] = range_of(rows ? c->k_scale : nullptr, rows, 1);
        r[3] = range_of(rows ? c->v_scale : nullptr, rows, 1);
        r[4] = range_of(c->page_table, c->n * c->max_pages, 4);
    }
};

inline bool any_overlap(Range x, const Range* r, int count)
{
    for (int i = 0; i < count; ++i)
        if (overlap(x, r[i])) return true;
    return false;
}

// Checks shared by gdn_kv_write and gdn_kv_read.
inline gdn_status check_rows(const gdn_kv_cache* c, int64_t total, int32_t dtype, const int32_t* start,
                      const int32_t* cu, int64_t* pool)
{
    const gdn_status st = check_cache(c, dtype, pool);
    if (st != GDN_OK) return st;
    if (total < 0 || total >= (INT64_C(1) << 31)) return GDN_ERR_SHAPE;
    if (!cu && total != c->n) return GDN_ERR_SHAPE;
    // one workgroup covers at least one (token, head) row
    int64_t rows;
    if (!mul_ok(total, c->h_kv, &rows) || rows >= (INT64_C(1) << 31)) return GDN_ERR_SHAPE;
    const gdn_status ps = cache_pointers(c);
    if (ps != GDN_OK) return ps;
    if (c->n > 0 && total > 0 && !start) return GDN_ERR_NULL;
    if (!aligned(start, 4) || !aligned(cu, 4)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

}  // namespace gdn
