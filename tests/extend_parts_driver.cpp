// Replays, on the host, which part of the workspace each workgroup of a gdn_attn_extend call divided by lengths
// writes, and which ones the join reads: the plan, the order of the parts and their bounds are the kernels' own
// code, the sequences are counted here. Nothing is launched.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "gdn_attn_extend.hip"

using namespace gdn;

namespace {

int clamped(int64_t x, int64_t hi)
{
    return (int)(x < 0 ? 0 : x > hi ? hi : x);
}

void fail(const char* what, long a, long b)
{
    std::printf("%s: %ld, %ld\n", what, a, b);
    std::exit(1);
}

struct Seen {
    long divided = 0, past = 0;  // calls divided by lengths; of them, sequences past the end
};

void replay(const gdn_kv_cache& c, const gdn_extend_dims& d, const std::vector<int>& cu, const std::vector<int>& lens, bool overlap, Seen* seen)
{
    const ExtendPlan p = make_plans(c, d).stream;
    if (p.m == 0 || !p.share) return;
    ++seen->divided;
    const int n = (int)c.n, g = d.h_q / c.h_kv, h = c.h_kv, longest = (int)extend_longest(c, d, p.m);
    std::vector<int> tiles(n), steps(n), ranges(n), before(n);
    int64_t work = 0;
    for (int s = 0; s < n; ++s) {
        const int len_q = clamped(cu[s + 1], d.total_q) - clamped(cu[s], d.total_q), used = len_q < d.max_q ? len_q : (int)d.max_q;
        const int rows = len_q <= 0 ? 0 : used * g, len = clamped(lens[s], d.max_len);
        int sight = len - len_q + used;
        sight = sight < longest ? sight : longest;
        tiles[s] = rows <= 0 || rows < p.rows_from || rows > p.rows_to ? 0 : (rows + p.m - 1) / p.m;
        steps[s] = sight <= kStep ? 1 : (sight + kStep - 1) / kStep;
        work += (int64_t)tiles[s] * h * steps[s];
    }
    int per = (int)((work + p.share - 1) / p.share);
    per = per > p.least ? per : p.least;
    for (int x = 0;; ++x, per += (per + 15) / 16) {
        int64_t sum = 0;
        for (int s = 0; s < n; ++s) {
            ranges[s] = (steps[s] + per - 1) / per;
            before[s] = (int)sum;
            sum += (int64_t)tiles[s] * h * ranges[s];
        }
        if (x == 8 || sum <= p.share) break;
    }
    // the grid and the workspace have workgroups() parts
    const long parts = p.workgroups();
    if ((size_t)parts * p.m * (c.d * sizeof(float) + sizeof(float4)) != p.workspace(c)) fail("workspace", parts, p.m);
    std::vector<char> written(parts, 0);
    for (long index = 0; index < parts; ++index)
        for (int s = 0; s < n; ++s) {
            if (index < before[s] || index >= before[s] + (long)tiles[s] * ranges[s] * h) continue;
            SharePart w;
            if (!share_part((uint32_t)index, before[s], tiles[s], ranges[s], h, (uint32_t)parts, &w)) continue;
            if (w.at >= parts) fail("a part past the end", w.at, parts);
            if (w.tile >= (uint32_t)tiles[s] || w.rg >= (uint32_t)ranges[s] || w.head >= (uint32_t)h) fail("no such part", w.tile, w.rg);
            if (written[w.at]++) fail("a part of two workgroups", w.at, index);
        }
    for (int s = 0; s < n; ++s) {
        if (!tiles[s]) continue;
        if (!block_fits(before[s], tiles[s], ranges[s], h, (uint32_t)parts)) {
            if (!overlap) fail("a sequence without parts", s, parts);
            ++seen->past;
            continue;
        }
        for (long at = before[s]; at < before[s] + (long)tiles[s] * ranges[s] * h; ++at)
            if (!written[at]) fail("a part that nobody wrote", at, s);
    }
}

gdn_kv_cache cache_of(int n, int h, int d, int store, int64_t positions)
{
    gdn_kv_cache c = {};
    c.n = n;
    c.num_pages = 1;
    c.page_size = 16;
    c.max_pages = (positions + 15) / 16;
    c.h_kv = h;
    c.d = d;
    c.store = store;
    return c;
}

}  // namespace

int main()
{
    Seen fixed;
    {  // every other sequence has all the rows: four times what the plan counts on
        const gdn_kv_cache c = cache_of(8, 2, 256, GDN_F32, 7168);
        const gdn_extend_dims d = {128, 128, 7168, 0, 0, 16, GDN_F32, 0.0625f, 4096, 256};
        replay(c, d, {0, 128, 0, 128, 0, 128, 0, 128, 0}, {128, 1, 128, 1, 7168, 1, 128, 1}, true, &fixed);
        if (fixed.divided != 1 || fixed.past == 0) fail("the plan was not asked for more than it has", fixed.divided, fixed.past);
    }
    std::mt19937_64 rng(1);
    auto in = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
    Seen good, bad;
    for (int i = 0; i < 6000; ++i) {
        const bool overlap = i % 2;
        const int n = (int)in(2, 64), h = (int)in(1, 4), g = (int)in(1, 8), dim = 64 << in(0, 2);
        const int dtype = in(0, 1) ? GDN_BF16 : GDN_F32, store = in(0, 1) ? GDN_FP8 : dtype;
        const int64_t most = in(0, 3) ? in(256, 20000) : in(20000, 200000);
        std::vector<int> cu(n + 1, 0), lens(n);
        const int big = in(0, 1) ? 8 : 150;
        for (int s = 0; s < n; ++s) {
            cu[s + 1] = cu[s] + (int)in(0, big);
            lens[s] = (int)(in(0, 1) ? in(-3, most) : in(0, 200));
        }
        const int64_t total = cu[n] > 0 ? cu[n] : 1;
        if (overlap)
            for (int s = 0; s <= n; ++s) cu[s] = (int)(in(0, 2) ? (s % 2) * total : in(-5, total + 5));
        gdn_extend_dims d = {total, in(0, 2) ? total : in(1, total), most, in(0, 2) ? 0 : in(1, most), in(0, 64), h * g, dtype, 0.1f, h * g * dim, dim};
        gdn_kv_cache c = cache_of(n, h, dim, store, most);
        // within what the kernels count in, as the entry point brings it
        if (d.window >= d.max_len || d.sinks >= d.max_len) d.window = 0;
        if (d.window == 0) d.sinks = 0;
        replay(c, d, cu, lens, overlap, overlap ? &bad : &good);
    }
    if (good.divided < 500 || bad.divided < 500 || bad.past < 100) fail("too few cases", good.divided, bad.past);
    std::printf("extend parts ok: %ld and %ld calls divided, %ld sequences past the end\n", good.divided, bad.divided, bad.past);
    return 0;
}
