// gdn_extend_api.hip -- C entry points around the attention layers: norms and rotary positions,
// the cache written with them, attention of new tokens over the cache (declared and documented in
// include/gdn.h): host-side validation and dispatch. Every check runs before the first HIP call,
// and on error nothing is enqueued.
#include "gdn_attn_checks.hpp"
#include "gdn_attn_internal.hpp"

namespace gdn {
namespace {

// What a row goes through: sizes and values. `placed`: a token has a place to turn by.
gdn_status check_norm_rope(const gdn_norm_rope* f, int32_t d, bool placed)
{
    if (!f) return GDN_ERR_NULL;
    if (!isfinite(f->eps) || f->eps < 0.f || !isfinite(f->weight_bias)) return GDN_ERR_SHAPE;
    if (f->rot < 0 || f->rot > d || f->rot % 16) return GDN_ERR_SHAPE;
    if (f->interleaved != 0 && f->interleaved != 1) return GDN_ERR_SHAPE;
    if (f->rot > 0) {
        if (f->axes < 1 || f->axes > 4 || !isfinite(f->rope_scale)) return GDN_ERR_SHAPE;
        if (!f->pos && placed && f->axes != 1) return GDN_ERR_SHAPE;  // places are one position a token
    }
    return GDN_OK;
}

// Its pointers; `work`: there are rows.
gdn_status norm_rope_pointers(const gdn_norm_rope* f, bool placed, bool work)
{
    if (f->rot > 0 && work && (!f->freq || (!f->pos && !placed))) return GDN_ERR_NULL;
    if (!aligned(f->q_weight, 16) || !aligned(f->k_weight, 16) || !aligned(f->freq, 4) || !aligned(f->pos, 4))
        return GDN_ERR_ALIGN;
    return GDN_OK;
}

// Its device ranges: weights, frequencies, axes, positions.
struct NormRopeRanges {
    Range r[5];
    NormRopeRanges(const gdn_norm_rope* f, int64_t total, int32_t d, int32_t dtype)
    {
        const bool turns = f->rot > 0;
        r[0] = range_of(f->q_weight, d, elem(dtype));
        r[1] = range_of(f->k_weight, d, elem(dtype));
        r[2] = range_of(turns ? f->freq : nullptr, f->rot / 2, 4);
        r[3] = range_of(turns ? f->axis : nullptr, f->rot / 2, 1);
        r[4] = range_of(turns ? f->pos : nullptr, total * (turns ? f->axes : 0), 4);
    }
};

// Sizes of an extend call; *rows its query rows (of all heads), *qe the extent of q. `b` gets the call's
// sizes within what the kernels count in.
gdn_status check_extend(const gdn_kv_cache* c, const gdn_extend_dims* d, int64_t* pool, int64_t* rows, int64_t* qe,
                        gdn_extend_dims* b)
{
    if (!c || !d) return GDN_ERR_NULL;
    const gdn_status st = check_cache(c, d->dtype, pool);
    if (st != GDN_OK) return st;
    if (d->total_q < 0 || d->max_q < 0 || d->max_len < 0 || d->window < 0 || d->sinks < 0) return GDN_ERR_SHAPE;
    if (d->h_q <= 0 || d->h_q % c->h_kv != 0 || !attn_scale(d->scale)) return GDN_ERR_SHAPE;
    const int64_t lim = INT64_C(1) << 31, rows_lim = lim - (1 << 16);  // the kernels count in 32 bits
    if (d->total_q >= rows_lim || !mul_ok(d->total_q, d->h_q, rows) || *rows / c->h_kv >= rows_lim) return GDN_ERR_SHAPE;
    if (!strided(d->total_q, d->h_q, c->d, d->q_token, d->q_head, d->dtype, qe)) return GDN_ERR_SHAPE;
    *b = *d;
    const int64_t cap = c->num_pages > 0 ? c->max_pages * c->page_size : 0;
    b->max_len = d->max_len < cap ? d->max_len : cap;
    if (b->max_len >= rows_lim) return GDN_ERR_SHAPE;
    b->max_q = d->max_q < d->total_q ? d->max_q : d->total_q;
    if (d->window >= b->max_len || d->sinks >= b->max_len) b->window = 0;  // every position is in sight
    if (b->window == 0) b->sinks = 0;
    // the grid: (tiles of at least 16 query rows) x (KV heads)
    const int64_t g = d->h_q / c->h_kv;
    if ((*rows / c->h_kv / 16 + c->n) * c->h_kv >= lim || b->max_q * g >= rows_lim) return GDN_ERR_SHAPE;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_qk_norm_rope(const gdn_norm_rope* f, int64_t total, int32_t h_q, int32_t h_kv, int32_t d, int32_t dtype,
                            const void* q, int64_t q_token, int64_t q_head, const void* k, int64_t k_token,
                            int64_t k_head, void* q_out, void* k_out, void* stream)
{
    if (!f) return GDN_ERR_NULL;
    const int64_t lim = INT64_C(1) << 31;
    if (total < 0 || total >= lim || h_q < 0 || h_kv < 0 || d <= 0) return GDN_ERR_SHAPE;
    if (!attn_d(d) || !attn_dtype(dtype)) return GDN_ERR_UNSUPPORTED;
    int64_t rows, qe = 0, ke = 0;
    if (!mul_ok(total, (int64_t)h_q + h_kv, &rows) || rows >= lim) return GDN_ERR_SHAPE;
    gdn_status st = check_norm_rope(f, d, false);
    if (st != GDN_OK) return st;
    if (h_q > 0 && !strided(total, h_q, d, q_token, q_head, dtype, &qe)) return GDN_ERR_SHAPE;
    if (h_kv > 0 && !strided(total, h_kv, d, k_token, k_head, dtype, &ke)) return GDN_ERR_SHAPE;
    const bool wq = rows > 0 && h_q > 0, wk = rows > 0 && h_kv > 0;
    if ((wq && (!q || !q_out)) || (wk && (!k || !k_out))) return GDN_ERR_NULL;
    if ((wq && (!aligned(q, 16) || !aligned(q_out, 16))) || (wk && (!aligned(k, 16) || !aligned(k_out, 16))))
        return GDN_ERR_ALIGN;
    st = norm_rope_pointers(f, false, rows > 0);
    if (st != GDN_OK) return st;
    const size_t es = elem(dtype);
    const NormRopeRanges n(f, total, d, dtype);
    const Range r[] = {range_of(wq ? q_out : nullptr, total * h_q * (int64_t)d, es),
                       range_of(wk ? k_out : nullptr, total * h_kv * (int64_t)d, es),
                       range_of(wq ? q : nullptr, qe, es), range_of(wk ? k : nullptr, ke, es)};
    for (int i = 0; i < 2; ++i)
        if (any_overlap(r[i], r + i + 1, 3 - i) || any_overlap(r[i], n.r, 5)) return GDN_ERR_ALIAS;
    if (rows == 0) return GDN_OK;
    RopeCall call = {};
    call.f = *f;
    call.total = total;
    call.h_q = h_q;
    call.h_kv = h_kv;
    call.d = d;
    call.dtype = dtype;
    call.q = q;
    call.k = k;
    call.q_token = q_token;
    call.q_head = q_head;
    call.k_token = k_token;
    call.k_head = k_head;
    call.q_out = q_out;
    call.k_out = k_out;
    call.stream = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();  // report only errors raised by this call's launch
    return finish(launch_rope(call, false));
}

gdn_status gdn_kv_append(const gdn_kv_cache* c, const gdn_norm_rope* f, int64_t total, int32_t dtype, const void* k,
                         int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                         const int32_t* start, const int32_t* cu, int32_t h_q, const void* q, int64_t q_token,
                         int64_t q_head, void* q_out, void* stream)
{
    int64_t pool, ke, ve, qe = 0, rows;
    gdn_status st = check_rows(c, total, dtype, start, cu, &pool);
    if (st != GDN_OK) return st;
    if (h_q < 0 || !mul_ok(total, h_q + 2 * (int64_t)c->h_kv, &rows) || rows >= (INT64_C(1) << 31)) return GDN_ERR_SHAPE;
    st = check_norm_rope(f, c->d, true);
    if (st != GDN_OK) return st;
    if (!strided(total, c->h_kv, c->d, k_token, k_head, dtype, &ke) ||
        !strided(total, c->h_kv, c->d, v_token, v_head, dtype, &ve) ||
        (h_q > 0 && !strided(total, h_q, c->d, q_token, q_head, dtype, &qe)))
        return GDN_ERR_SHAPE;
    const bool work = c->n > 0 && total > 0, wq = work && h_q > 0;
    if (work && (!k || !v)) return GDN_ERR_NULL;
    if (wq && (!q || !q_out)) return GDN_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || (wq && (!aligned(q, 16) || !aligned(q_out, 16)))) return GDN_ERR_ALIGN;
    st = norm_rope_pointers(f, true, work);
    if (st != GDN_OK) return st;
    const size_t es = elem(dtype);
    const CacheRanges p(c, pool);
    const NormRopeRanges n(f, total, c->d, dtype);
    const Range out = range_of(wq ? q_out : nullptr, total * h_q * (int64_t)c->d, es);
    const Range in[] = {range_of(k, ke, es), range_of(v, ve, es), range_of(wq ? q : nullptr, qe, es),
                        range_of(start, work ? c->n : 0, 4), range_of(cu, cu && work ? c->n + 1 : 0, 4)};
    for (int i = 0; i < 4; ++i)  // the pools and scales are outputs
        if (any_overlap(p.r[i], in, 5) || any_overlap(p.r[i], n.r, 5) || any_overlap(p.r[i], p.r + i + 1, 4 - i))
            return GDN_ERR_ALIAS;
    if (any_overlap(out, in, 5) || any_overlap(out, n.r, 5) || any_overlap(out, p.r, 5)) return GDN_ERR_ALIAS;
    if (!work || (h_q == 0 && (c->num_pages == 0 || c->max_pages == 0))) return GDN_OK;
    RopeCall call = {};
    call.f = *f;
    call.c = *c;
    call.total = total;
    call.h_q = h_q;
    call.h_kv = c->h_kv;
    call.d = c->d;
    call.dtype = dtype;
    call.q = q;
    call.k = k;
    call.v = v;
    call.q_token = q_token;
    call.q_head = q_head;
    call.k_token = k_token;
    call.k_head = k_head;
    call.v_token = v_token;
    call.v_head = v_head;
    call.q_out = q_out;
    call.start = start;
    call.cu = cu;
    call.stream = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    return finish(launch_rope(call, true));
}

size_t gdn_attn_extend_workspace_bytes(const gdn_kv_cache* c, const gdn_extend_dims* d)
{
    int64_t pool, rows, qe;
    gdn_extend_dims b;
    if (check_extend(c, d, &pool, &rows, &qe, &b) != GDN_OK || c->n == 0 || b.max_q == 0) return 0;
    return attn_extend_workspace(*c, b);
}

gdn_status gdn_attn_extend(const gdn_kv_cache* c, const gdn_extend_dims* d, const void* q, const int32_t* cu_q,
                           const int32_t* lens, void* out, float* lse, void* ws, size_t ws_bytes, void* stream)
{
    int64_t pool, rows, qe;
    gdn_extend_dims b;
    gdn_status st = check_extend(c, d, &pool, &rows, &qe, &b);
    if (st != GDN_OK) return st;
    if (!cu_q && (d->total_q != c->n || b.max_q > 1)) return GDN_ERR_SHAPE;
    st = cache_pointers(c);
    if (st != GDN_OK) return st;
    const bool work = c->n > 0 && b.max_q > 0;
    if (work && (!q || !lens || !out)) return GDN_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 16) || !aligned(cu_q, 4) || !aligned(lens, 4) || !aligned(lse, 4))
        return GDN_ERR_ALIGN;
    const size_t need = work ? attn_extend_workspace(*c, b) : 0;
    if (need > 0 && (!ws || ws_bytes < need)) return GDN_ERR_WORKSPACE;
    const CacheRanges p(c, pool);
    const size_t es = elem(d->dtype);
    const Range r[] = {range_of(out, rows * c->d, es), range_of(lse, lse ? rows : 0, 4),
                       range_of(need ? ws : nullptr, (int64_t)need, 1), range_of(q, qe, es),
                       range_of(cu_q, cu_q && work ? c->n + 1 : 0, 4), range_of(lens, work ? c->n : 0, 4)};
    for (int i = 0; i < 3; ++i)
        if (any_overlap(r[i], r + i + 1, 5 - i) || any_overlap(r[i], p.r, 5)) return GDN_ERR_ALIAS;
    if (!work) return GDN_OK;
    const ExtendCall call = {*c, b, q, cu_q, lens, out, lse, ws, static_cast<hipStream_t>(stream)};
    (void)hipGetLastError();
    return finish(launch_attn_extend(call));
}

}  // extern "C"
