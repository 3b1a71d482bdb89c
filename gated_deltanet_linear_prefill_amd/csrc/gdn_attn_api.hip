// gdn_attn_api.hip -- C entry points of the paged key-value cache and of attention (declared
// and documented in include/gdn.h): host-side validation and dispatch. Every check runs
// before the first HIP call, and on error nothing is enqueued.
#include "gdn_attn_checks.hpp"
#include "gdn_attn_internal.hpp"

namespace gdn {
namespace {

// What the sizes and strides of a prefill call have to be; *rows the query rows, *qe, *ke, *ve the
// tensors' extents.
gdn_status check_prefill(const gdn_attn_dims* d, int64_t* rows, int64_t* qe, int64_t* ke, int64_t* ve)
{
    if (!d) return GDN_ERR_NULL;
    if (d->n < 0 || d->total_q < 0 || d->total_k < 0 || d->h_q <= 0 || d->h_kv <= 0 || d->d <= 0)
        return GDN_ERR_SHAPE;
    if (d->h_q % d->h_kv != 0 || (d->causal != 0 && d->causal != 1) || !attn_scale(d->scale))
        return GDN_ERR_SHAPE;
    if (!attn_dtype(d->dtype) || !attn_d(d->d)) return GDN_ERR_UNSUPPORTED;
    const int64_t lim = INT64_C(1) << 31;
    const int64_t rows_lim = lim - (1 << 16);  // the kernels count rows and keys in 32 bits
    if (d->n >= lim || d->total_q >= rows_lim || d->total_k >= rows_lim) return GDN_ERR_SHAPE;
    if (!mul_ok(d->total_q, d->h_q, rows) || *rows / d->h_kv >= rows_lim) return GDN_ERR_SHAPE;
    // the grid: (tiles of query rows) x (KV heads), see the kernel
    if ((*rows / d->h_kv / attn_prefill_rows(d->d, d->dtype) + d->n) * d->h_kv >= lim) return GDN_ERR_SHAPE;
    if (!strided(d->total_q, d->h_q, d->d, d->q_token, d->q_head, d->dtype, qe) ||
        !strided(d->total_k, d->h_kv, d->d, d->k_token, d->k_head, d->dtype, ke) ||
        !strided(d->total_k, d->h_kv, d->d, d->v_token, d->v_head, d->dtype, ve))
        return GDN_ERR_SHAPE;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_kv_write(const gdn_kv_cache* c, int64_t total, int32_t dtype, const void* k,
                        int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                        int64_t v_head, const int32_t* start, const int32_t* cu, void* stream)
{
    int64_t pool, ke, ve;
    const gdn_status st = check_rows(c, total, dtype, start, cu, &pool);
    if (st != GDN_OK) return st;
    if (!strided(total, c->h_kv, c->d, k_token, k_head, dtype, &ke) ||
        !strided(total, c->h_kv, c->d, v_token, v_head, dtype, &ve))
        return GDN_ERR_SHAPE;
    const bool work = c->n > 0 && total > 0;
    if (work && (!k || !v)) return GDN_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16)) return GDN_ERR_ALIGN;
    const CacheRanges p(c, pool);
    const Range in[] = {range_of(k, ke, elem(dtype)), range_of(v, ve, elem(dtype)),
                        range_of(start, work ? c->n : 0, 4), range_of(cu, cu && work ? c->n + 1 : 0, 4)};
    for (int i = 0; i < 4; ++i)  // the pools and scales are outputs
        if (any_overlap(p.r[i], in, 4) || any_overlap(p.r[i], p.r + i + 1, 4 - i)) return GDN_ERR_ALIAS;
    if (!work || c->num_pages == 0 || c->max_pages == 0) return GDN_OK;
    KvCall call = {};
    call.c = *c;
    call.total = total;
    call.dtype = dtype;
    call.k = k;
    call.v = v;
    call.k_token = k_token;
    call.k_head = k_head;
    call.v_token = v_token;
    call.v_head = v_head;
    call.start = start;
    call.cu = cu;
    call.stream = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();  // report only errors raised by this call's launch
    return finish(launch_kv_write(call));
}

gdn_status gdn_kv_read(const gdn_kv_cache* c, int64_t total, int32_t dtype, void* k, void* v,
                       const int32_t* start, const int32_t* cu, void* stream)
{
    int64_t pool, elems;
    const gdn_status st = check_rows(c, total, dtype, start, cu, &pool);
    if (st != GDN_OK) return st;
    const bool work = c->n > 0 && total > 0;
    if (work && (!k || !v)) return GDN_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16)) return GDN_ERR_ALIGN;
    elems = total * c->h_kv * (int64_t)c->d;
    const CacheRanges p(c, pool);
    const Range out[] = {range_of(k, elems, elem(dtype)), range_of(v, elems, elem(dtype)),
                         range_of(start, work ? c->n : 0, 4), range_of(cu, cu && work ? c->n + 1 : 0, 4)};
    for (int i = 0; i < 2; ++i)
        if (any_overlap(out[i], p.r, 5) || any_overlap(out[i], out + i + 1, 3 - i)) return GDN_ERR_ALIAS;
    if (!work) return GDN_OK;
    KvCall call = {};
    call.c = *c;
    call.total = total;
    call.dtype = dtype;
    call.k_out = k;
    call.v_out = v;
    call.start = start;
    call.cu = cu;
    call.stream = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    return finish(launch_kv_read(call));
}

size_t gdn_attn_prefill_workspace_bytes(const gdn_attn_dims* d)
{
    int64_t rows, qe, ke, ve;
    return check_prefill(d, &rows, &qe, &ke, &ve) == GDN_OK ? attn_prefill_workspace(*d) : 0;
}

gdn_status gdn_attn_prefill(const gdn_attn_dims* d, const void* q, const void* k, const void* v,
                            const int32_t* cu_q, const int32_t* cu_k, void* out, float* lse, void* ws,
                            size_t ws_bytes, void* stream)
{
    int64_t rows, qe, ke, ve;
    const gdn_status st = check_prefill(d, &rows, &qe, &ke, &ve);
    if (st != GDN_OK) return st;
    if (!cu_k && d->total_k != d->total_q) return GDN_ERR_SHAPE;
    const bool work = d->n > 0 && d->total_q > 0;
    if (work && (!q || !out || !cu_q || (d->total_k > 0 && (!k || !v)))) return GDN_ERR_NULL;
    for (const void* p : {q, k, v, (const void*)out, (const void*)ws})
        if (!aligned(p, 16)) return GDN_ERR_ALIGN;
    if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4)) return GDN_ERR_ALIGN;
    const size_t es = elem(d->dtype);
    const size_t need = work ? attn_prefill_workspace(*d) : 0;
    if (need > 0 && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    const Range r[] = {range_of(out, rows * d->d, es), range_of(lse, lse ? rows : 0, 4),
                       range_of(need ? ws : nullptr, (int64_t)need, 1), range_of(q, qe, es), range_of(k, ke, es), range_of(v, ve, es),
                       range_of(cu_q, work ? d->n + 1 : 0, 4), range_of(cu_k, cu_k && work ? d->n + 1 : 0, 4)};
    for (int i = 0; i < 3; ++i)
        if (any_overlap(r[i], r + i + 1, 7 - i)) return GDN_ERR_ALIAS;
    if (!work) return GDN_OK;
    const AttnCall call = {*d, q, k, v, cu_q, cu_k ? cu_k : cu_q, out, lse, ws,
                           static_cast<hipStream_t>(stream), 0, 1, nullptr, nullptr};
    (void)hipGetLastError();
    return finish(launch_attn_prefill(call));
}

size_t gdn_attn_decode_workspace_bytes(const gdn_kv_cache* c, int32_t h_q, int64_t max_len)
{
    int64_t pool, rows;
    if (!c || h_q <= 0 || max_len < 0 || c->h_kv <= 0 || h_q % c->h_kv != 0) return 0;
    if (check_cache(c, c->store == GDN_FP8 ? GDN_BF16 : c->store, &pool) != GDN_OK) return 0;
    if (!mul_ok(c->n, h_q, &rows) || rows >= (INT64_C(1) << 31)) return 0;
    return attn_decode_workspace(c, h_q, max_len);
}

gdn_status gdn_attn_decode(const gdn_kv_cache* c, int32_t h_q, int32_t dtype, float scale,
                           int64_t max_len, const void* q, int64_t q_token, int64_t q_head,
                           const int32_t* lens, void* out, float* lse, void* ws, size_t ws_bytes,
                           void* stream)
{
    int64_t pool, qe, rows;
    gdn_status st = check_cache(c, dtype, &pool);
    if (st != GDN_OK) return st;
    if (h_q <= 0 || h_q % c->h_kv != 0 || max_len < 0 || !attn_scale(scale)) return GDN_ERR_SHAPE;
    if (!mul_ok(c->n, h_q, &rows) || rows >= (INT64_C(1) << 31)) return GDN_ERR_SHAPE;
    if (!strided(c->n, h_q, c->d, q_token, q_head, dtype, &qe)) return GDN_ERR_SHAPE;
    st = cache_pointers(c);
    if (st != GDN_OK) return st;
    if (c->n > 0 && (!q || !lens || !out)) return GDN_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 16) || !aligned(lens, 4) || !aligned(lse, 4))
        return GDN_ERR_ALIGN;
    const size_t need = attn_decode_workspace(c, h_q, max_len);
    if (need > 0 && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    const CacheRanges p(c, pool);
    const size_t es = elem(dtype);
    const Range r[] = {range_of(out, rows * c->d, es), range_of(lse, lse ? rows : 0, 4),
                       range_of(need ? ws : nullptr, (int64_t)need, 1), range_of(q, qe, es),
                       range_of(lens, c->n, 4)};
    for (int i = 0; i < 3; ++i)
        if (any_overlap(r[i], r + i + 1, 4 - i) || any_overlap(r[i], p.r, 5)) return GDN_ERR_ALIAS;
    if (c->n == 0) return GDN_OK;
    const AttnDecodeCall call = {*c, h_q, dtype, scale, max_len, q, q_token, q_head, lens,
                                 out, lse, ws, static_cast<hipStream_t>(stream)};
    (void)hipGetLastError();
    return finish(launch_attn_decode(call));
}

}  // extern "C"
