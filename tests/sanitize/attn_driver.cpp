// Drives the refusals of the attention entry points (fake device addresses, nothing launched) for a
// build of their host code with sanitizers.
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
    gdn_kv_cache c = {2, 8, 4, 16, 2, 64, GDN_BF16, at(1), at(2), nullptr, nullptr, i32(3)};
    expect("write: null cache", gdn_kv_write(nullptr, 1, GDN_BF16, at(4), 128, 64, at(5), 128, 64, i32(6), i32(7), nullptr), GDN_ERR_NULL);
    expect("write: alias", gdn_kv_write(&c, 10, GDN_BF16, at(1), 128, 64, at(5), 128, 64, i32(6), i32(7), nullptr), GDN_ERR_ALIAS);
    expect("write: strides", gdn_kv_write(&c, 10, GDN_BF16, at(4), huge - 7, huge - 7, at(5), 128, 64, i32(6), i32(7), nullptr), GDN_ERR_SHAPE);
    expect("write: total", gdn_kv_write(&c, huge, GDN_BF16, at(4), 128, 64, at(5), 128, 64, i32(6), i32(7), nullptr), GDN_ERR_SHAPE);
    expect("read: align", gdn_kv_read(&c, 10, GDN_BF16, at(4) + 2, at(5), i32(6), i32(7), nullptr), GDN_ERR_ALIGN);
    for (int64_t big : {huge, huge / 2, (int64_t)1 << 40}) {
        gdn_kv_cache b = c;
        b.num_pages = big;
        expect("write: pages", gdn_kv_write(&b, 1, GDN_BF16, at(4), 128, 64, at(5), 128, 64, i32(6), i32(7), nullptr), GDN_ERR_SHAPE);
        b = c;
        b.n = big;
        expect("decode: n", gdn_attn_decode(&b, 4, GDN_BF16, 0.1f, 64, at(4), 256, 64, i32(6), at(5), nullptr, nullptr, 0, nullptr), GDN_ERR_SHAPE);
    }
    gdn_kv_cache wide = c;
    wide.num_pages = (1ll << 31) - 1;
    wide.page_size = 1024;
    wide.h_kv = 0x7fffffff;
    expect("read: pool size", gdn_kv_read(&wide, 1, GDN_BF16, at(4), at(5), i32(6), i32(7), nullptr), GDN_ERR_SHAPE);
    expect("workspace: h_q", (long)gdn_attn_decode_workspace_bytes(&c, 3, huge), 0);
    gdn_kv_cache lng = c;
    lng.max_pages = 1 << 20;
    const size_t need = gdn_attn_decode_workspace_bytes(&lng, 4, huge);
    expect("workspace: bounded by the table", need > 0, 1);
    expect("decode: workspace", gdn_attn_decode(&lng, 4, GDN_BF16, 0.1f, huge, at(4), 256, 64, i32(6), at(5), nullptr, at(8), need - 1, nullptr), GDN_ERR_WORKSPACE);
    expect("decode: scale", gdn_attn_decode(&c, 4, GDN_BF16, NAN, 64, at(4), 256, 64, i32(6), at(5), nullptr, nullptr, 0, nullptr), GDN_ERR_SHAPE);
    gdn_attn_dims d = {2, 10, 20, 4, 2, 64, GDN_BF16, 1, 0.125f, 256, 64, 128, 64, 128, 64};
    expect("prefill: null", gdn_attn_prefill(&d, at(1), nullptr, at(3), i32(5), i32(6), at(4), nullptr, nullptr, 0, nullptr), GDN_ERR_NULL);
    d.total_q = huge;
    expect("prefill: total", gdn_attn_prefill(&d, at(1), at(2), at(3), i32(5), i32(6), at(4), nullptr, nullptr, 0, nullptr), GDN_ERR_SHAPE);
    d.total_q = 10;
    d.h_q = 0x7ffffffe;
    d.h_kv = 2;
    expect("prefill: heads", gdn_attn_prefill(&d, at(1), at(2), at(3), i32(5), i32(6), at(4), nullptr, nullptr, 0, nullptr), GDN_ERR_SHAPE);
    std::printf("attention driver ok\n");
    return 0;
}
