// Asks for the workspace of attention calls at the ends of what their checks let through, and beyond, for
// a build of the size computations with sanitizers.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <limits>

#include "gdn.h"

int main()
{
    const int64_t sizes[] = {0, 1, 3, 1000, 1 << 20, (1ll << 31) - 1, 1ll << 31, 1ll << 40, std::numeric_limits<int64_t>::max()};
    const int32_t heads[] = {1, 2, 1 << 10, 1 << 20, 0x7ffffffe, 0x7fffffff};
    long asked = 0;
    for (int64_t n : sizes)
        for (int64_t pages : {0ll, 1ll, 1ll << 14, (1ll << 27) - 1, 1ll << 40})
            for (int32_t h_kv : heads)
                for (int32_t h_q : heads)
                    for (int64_t max_len : sizes) {
                        const gdn_kv_cache c = {n, 0, pages, 16, h_kv, 64, GDN_BF16, nullptr, nullptr, nullptr, nullptr, nullptr};
                        const size_t need = gdn_attn_decode_workspace_bytes(&c, h_q, max_len);
                        ++asked;
                        // a call that gdn_attn_decode refuses for its sizes needs none
                        if (need > 0 && (h_q % h_kv || n <= 0 || (double)n * h_q >= 2147483648.0 || pages > 1ll << 27)) {
                            std::printf("decode: n %lld, heads %d / %d: %zu\n", (long long)n, h_q, h_kv, need);
                            return 1;
                        }
                    }
    for (int64_t n : sizes)
        for (int64_t q : sizes)
            for (int64_t k : sizes)
                for (int32_t h_kv : heads)
                    for (int32_t h_q : heads) {
                        const int64_t row = 64ll * h_q;
                        const gdn_attn_dims d = {n, q, k, h_q, h_kv, 64, GDN_F32, 1, 0.1f, row, 64, 64ll * h_kv, 64, 64ll * h_kv, 64};
                        asked += gdn_attn_prefill_workspace_bytes(&d) <= 64 * 1024 * (4 * 64 + 16) ? 1 : 1 << 30;
                    }
    if (asked >= 1 << 30) return 2;
    std::printf("sizes ok: %ld\n", asked);
    return 0;
}
