// Drives the refusals and the size computations of the entry points around the attention layers (fake
// device addresses, nothing launched) for a build of their host code with sanitizers.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <limits>

#include "gdn.h"

static void expect(const char* what, long got, long want)
{
    if (got != want) {
        std::printf("%s: got %ld, want %ld\n", what, got, want);
        std::exit(1);
    }
}

static char* at(int i)
{
    return reinterpret_cast<char*>(0x7f0000000000ull + ((unsigned long long)i << 32));
}

static const int32_t* i32(int i)
{
    return reinterpret_cast<const int32_t*>(at(i));
}

int main()
{
    const int64_t huge = std::numeric_limits<int64_t>::max();
    const int32_t wide = 0x7fffffff;
    gdn_norm_rope f = {1e-6f, 1.f, at(20), at(21), 32, 0, 1, 1.f, reinterpret_cast<float*>(at(22)), nullptr, i32(23)};
    expect("rope: null", gdn_qk_norm_rope(nullptr, 1, 1, 1, 64, GDN_BF16, at(1), 64, 64, at(2), 64, 64, at(3), at(4), nullptr), GDN_ERR_NULL);
    for (int64_t total : {huge, huge / 2, (int64_t)1 << 40, (int64_t)1 << 31})
        expect("rope: total", gdn_qk_norm_rope(&f, total, 1, 1, 64, GDN_BF16, at(1), 64, 64, at(2), 64, 64, at(3), at(4), nullptr), GDN_ERR_SHAPE);
    expect("rope: heads", gdn_qk_norm_rope(&f, 3, wide, wide, 64, GDN_BF16, at(1), 64, 64, at(2), 64, 64, at(3), at(4), nullptr), GDN_ERR_SHAPE);
    expect("rope: strides", gdn_qk_norm_rope(&f, 3, 2, 1, 64, GDN_BF16, at(1), huge - 7, huge - 7, at(2), 64, 64, at(3), at(4), nullptr), GDN_ERR_SHAPE);
    expect("rope: alias", gdn_qk_norm_rope(&f, 3, 2, 1, 64, GDN_BF16, at(1), 128, 64, at(2), 64, 64, at(1), at(4), nullptr), GDN_ERR_ALIAS);
    f.rot = wide - 15;
    expect("rope: rot", gdn_qk_norm_rope(&f, 3, 2, 1, 64, GDN_BF16, at(1), 128, 64, at(2), 64, 64, at(3), at(4), nullptr), GDN_ERR_SHAPE);
    f.rot = 32;
    gdn_kv_cache c = {2, 8, 4, 16, 2, 64, GDN_BF16, at(1), at(2), nullptr, nullptr, i32(3)};
    for (int64_t total : {huge, (int64_t)1 << 30})
        expect("append: total", gdn_kv_append(&c, &f, total, GDN_BF16, at(4), 128, 64, at(5), 128, 64, i32(6), i32(7), wide, at(8), 128, 64, at(9), nullptr), GDN_ERR_SHAPE);
    expect("append: alias", gdn_kv_append(&c, &f, 10, GDN_BF16, at(4), 128, 64, at(5), 128, 64, i32(6), i32(7), 2, at(8), 128, 64, at(1), nullptr), GDN_ERR_ALIAS);
    expect("append: null", gdn_kv_append(&c, nullptr, 10, GDN_BF16, at(4), 128, 64, at(5), 128, 64, i32(6), i32(7), 0, nullptr, 0, 0, nullptr, nullptr), GDN_ERR_NULL);

    gdn_extend_dims d = {10, 8, 64, 0, 0, 4, GDN_BF16, 0.125f, 256, 64};
    auto call = [&]() { return gdn_attn_extend(&c, &d, at(4), i32(5), i32(6), at(7), nullptr, nullptr, 0, nullptr); };
    const gdn_extend_dims keep = d;
    for (int64_t big : {huge, huge / 2, (int64_t)1 << 40}) {
        d.total_q = big;
        expect("extend: rows", call(), GDN_ERR_SHAPE);
        d = keep;
        gdn_kv_cache b = c;
        b.num_pages = big;
        expect("extend: pages", gdn_attn_extend(&b, &d, at(4), i32(5), i32(6), at(7), nullptr, nullptr, 0, nullptr), GDN_ERR_SHAPE);
    }
    d.scale = NAN;
    expect("extend: scale", call(), GDN_ERR_SHAPE);
    d = keep;
    d.h_q = wide - 1;
    expect("extend: heads", call(), GDN_ERR_SHAPE);
    // sizes over their whole ranges
    for (int64_t pages : {(int64_t)1, (int64_t)500, (int64_t)1 << 17, ((int64_t)1 << 27) - 4097})
        for (int64_t n : {(int64_t)1, (int64_t)40, (int64_t)77, (int64_t)1 << 20})
            for (int64_t total : {(int64_t)1, (int64_t)1000, (int64_t)1 << 24, ((int64_t)1 << 30)})
                for (int64_t max_q : {(int64_t)1, (int64_t)40, huge})
                    for (int64_t window : {(int64_t)0, (int64_t)1, (int64_t)5000, huge})
                        for (int32_t heads : {1, 8, 100})
                            for (int dim : {64, 128, 256})
                                for (int store : {GDN_BF16, GDN_F32, GDN_FP8}) {
                                    c.n = n;
                                    c.max_pages = pages;
                                    c.d = dim;
                                    c.store = store;
                                    d = keep;
                                    d.dtype = store == GDN_F32 ? GDN_F32 : GDN_BF16;
                                    d.total_q = total;
                                    d.max_q = max_q;
                                    d.max_len = huge;
                                    d.window = window;
                                    d.sinks = window / 2;
                                    d.h_q = 2 * heads;
                                    d.q_head = dim;
                                    d.q_token = 2 * heads * dim;
                                    (void)gdn_attn_extend_workspace_bytes(&c, &d);
                                }
    std::printf("extend driver ok\n");
    return 0;
}
