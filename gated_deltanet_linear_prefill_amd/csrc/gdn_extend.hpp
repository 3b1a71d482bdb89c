// gdn_extend.hpp -- what the kernels of gdn_attn_extend share: which rows a workgroup takes, what they
// see, and where divided sums go (not part of the C ABI).
#pragma once

#include "gdn_attn_tile.hpp"

namespace gdn {

// Where the keys of a call's tiles are divided into ranges, sums go to the workspace, a row at a time:
// o [D] fp32 and (m, l, exact l, -). Few rows: [workgroup][row of its tile]. Tiles of many rows:
// [range][KV head][row], the rows of the call as they are packed, for a batch may leave most of its slots for tiles empty
// (512 sequences of 732 tokens, fp8, d = 256: 21 GB by workgroups).
struct ExtendPlan {
    int m;          // rows of a tile (0: nothing is launched)
    int per_seq;    // tiles of every sequence, or 0: as many as its rows need, packed
    int64_t slots;  // tiles of one KV head that the grid has room for
    int64_t units;  // ... of all KV heads
    int64_t range;  // virtual positions of a range
    int64_t ranges;
    int64_t share;  // workgroups that the call's positions are divided over by their lengths, or 0: by range
    int least;      // ... with at least so many steps each
    int rows_from, rows_to;  // the sequences that are taken: by their rows (of a KV head)
    int64_t packed;          // rows of a KV head that the call has, where the workspace is by these; or 0
    int64_t workgroups() const { return share ? share + units : units * ranges; }
    int64_t part_rows(const gdn_kv_cache& c) const { return packed ? ranges * c.h_kv * packed : workgroups() * m; }
    size_t workspace(const gdn_kv_cache& c) const
    {
        return m == 0 || ranges == 1 ? 0 : (size_t)part_rows(c) * (c.d * sizeof(float) + sizeof(float4));
    }
};

struct ExtendArgs {
    ExtendCall c;
    int64_t range;
    int ranges, slots, per_seq, rows_from, rows_to, page_shift;
    int share, least, longest;  // longest: virtual positions that a tile may have
    int64_t packed;
    float* part_o;
    float4* part_ml;
};

// Virtual positions that a tile of m rows may have.
inline int64_t extend_longest(const gdn_kv_cache& c, const gdn_extend_dims& d, int m)
{
    if (d.window == 0) return d.max_len;
    const int64_t g = d.h_q / c.h_kv;
    const int64_t w = d.window + (m - 1) / g + 1 + 15 + (d.sinks + 15) / 16 * 16;
    return w < d.max_len ? w : d.max_len;
}

inline ExtendArgs extend_args(const ExtendCall& c, const ExtendPlan& p, void* ws)
{
    ExtendArgs a;
    a.c = c;
    a.range = p.range;
    a.ranges = (int)p.ranges;
    a.slots = (int)p.slots;
    a.per_seq = p.per_seq;
    a.rows_from = p.rows_from;
    a.rows_to = p.rows_to;
    a.page_shift = __builtin_ctz((unsigned)c.c.page_size);
    a.share = (int)p.share;
    a.least = p.least;
    a.longest = (int)extend_longest(c.c, c.d, p.m);
    a.packed = p.packed;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float4*>(a.part_o + p.part_rows(c.c) * c.c.d);
    return a;
}

hipError_t launch_extend_join(const ExtendArgs& a, int m);
ExtendPlan extend_tile_plan(const gdn_kv_cache& c, const gdn_extend_dims& d);
hipError_t launch_extend_tiles(const ExtendCall& c, const ExtendPlan& p, void* ws);

namespace {

// A tile: rows row0 .. of the `rows` that its sequence has, and the positions that they see. These are
// [0, sinks) and the stretch from the first row's window to the last row, in whole 16-position
// blocks and numbered through: virtual position v is position v below `sink` and v + skip from there on.
// Where something is skipped, all of the tile's rows lie behind it, so that a row at position p sees
//     v < p + 1 - skip  with  v >= p + 1 - window - skip  or  v < sinks.
struct Span {
    int64_t q0;
    int seq, head, rows, row0, g;
    int first, last;      // positions of its first and last row
    int shift;            // position of the sequence's row 0
    int sink, skip, len;  // len: virtual positions
    __device__ __forceinline__ int pos(int v) const { return v < sink ? v : v + skip; }
};

// Sequences up to which a workgroup counts the tiles before its own (64 at a time); of more it looks its
// sequence up in slots that are spread enough to need no counting.
constexpr int kExactSeqs = 256;

// Rows of a KV head that a sequence of len_q tokens has.
__device__ __forceinline__ int rows_of(const ExtendCall& p, int len_q, int g)
{
    return len_q <= 0 ? 0 : (len_q < p.d.max_q ? len_q : (int)p.d.max_q) * g;
}

// A sequence's length as the call takes it.
__device__ __forceinline__ int length_of(const ExtendCall& p, int s)
{
    const int len = p.lens[s] < p.d.max_len ? p.lens[s] : (int)p.d.max_len;
    return len < 0 ? 0 : len;
}

// Tile `local` of sequence s, which has the rows from qa to qb - 1 and the length len, or false if there is none.
template <int M>
__device__ __forceinline__ bool span_at(const ExtendArgs& a, int s, int qa, int qb, int len, int local, Span* t)
{
    const ExtendCall& p = a.c;
    const int g = p.d.h_q / p.c.h_kv;
    const int len_q = qb - qa;
    if (len_q <= 0 || local < 0) return false;
    t->seq = s;
    t->q0 = qa;
    t->g = g;
    t->rows = rows_of(p, len_q, g);
    if (t->rows < a.rows_from || t->rows > a.rows_to) return false;
    const int tiles = (t->rows + M - 1) / M;
    if (local >= tiles) return false;
    t->row0 = (tiles - 1 - local) * M;  // the last, which see most, first
    t->shift = len - len_q;
    t->first = t->shift + t->row0 / g;
    t->last = t->shift + ((t->row0 + M < t->rows ? t->row0 + M : t->rows) - 1) / g;
    const int w = (int)p.d.window, lo = w && t->first >= w ? (t->first - w + 1) & ~15 : 0;
    const int sinks = (int)((p.d.sinks + 15) & ~15);
    t->sink = sinks < lo ? sinks : lo;
    t->skip = lo - t->sink;
    t->len = t->last < 0 ? 0 : t->last + 1 - t->skip;
    return true;
}

// Workgroup i of a sequence's takes tile *tile of its `pairs` (range, head): the tiles of a pair, which read the
// same keys, at the same time and on one XCD, whose L2 they share (workgroups i and i + 8).
// 8 tokens after 32760, d = 256, 16/2 heads (two tiles) 37 us without and 33 with it; tiles of many rows, which read
// slower, are as fast either way.
__host__ __device__ __forceinline__ uint32_t pair_of(uint32_t i, uint32_t pairs, uint32_t tiles, uint32_t* tile)
{
    const uint32_t eight = i / (8 * tiles), rest = i - eight * 8 * tiles, left = pairs - 8 * eight;
    const uint32_t row = left < 8 ? left : 8;
    *tile = rest / row;
    return 8 * eight + rest - *tile * row;
}

// The part that workgroup `index` of a call divided by lengths takes. A sequence's parts are a block from `before` on, one for
// each range of its tiles of h heads. The grid and the workspace hold it as a whole or not at all: sequences that
// overlap (offsets that go back) may ask for more than the `parts` that there are, and that order would send
// workgroups at the grid's end past it.
struct SharePart {
    uint32_t tile, rg, head, at;  // at: its place in the workspace
};

__host__ __device__ __forceinline__ bool block_fits(uint32_t before, uint32_t tiles, uint32_t ranges, uint32_t h, uint32_t parts)
{
    return before + (uint64_t)tiles * ranges * h <= parts;
}

__host__ __device__ __forceinline__ bool share_part(uint32_t index, uint32_t before, uint32_t tiles, uint32_t ranges, uint32_t h,
                                                    uint32_t parts, SharePart* x)
{
    if (!block_fits(before, tiles, ranges, h, parts)) return false;
    const uint32_t pair = pair_of(index - before, h * ranges, tiles, &x->tile);
    x->rg = pair / h;
    x->head = pair - x->rg * h;
    x->at = before + (x->rg * tiles + x->tile) * h + x->head;
    return true;
}

// One sequence's workgroups in that order: the number [range][tile][head] of workgroup `index`.
__device__ __forceinline__ uint32_t together(const ExtendArgs& a, uint32_t index)
{
    const uint32_t h = (uint32_t)a.c.c.h_kv;
    if (a.c.c.n > 1 || a.slots == 1 || a.ranges == 1) return index;
    uint32_t tile;
    const uint32_t pair = pair_of(index, h * (uint32_t)a.ranges, (uint32_t)a.slots, &tile), rg = pair / h;
    return (rg * (uint32_t)a.slots + tile) * h + (pair - rg * h);
}

// A workgroup's tile, or false where there is none. Workgroups without one come last, where the tiles are
// counted: in between they cost more than they seem to (one in nine of them made a call of 256
// others, one a CU, take two rounds: 260 us instead of 155).
template <int M>
__device__ __forceinline__ bool find_span(const ExtendArgs& a, uint32_t unit, Span* t)
{
    const ExtendCall& p = a.c;
    const int g = p.d.h_q / p.c.h_kv, n = (int)p.c.n, total = (int)p.d.total_q;
    const int slot = (int)(unit / (uint32_t)p.c.h_kv);
    t->head = (int)(unit - (uint32_t)slot * (uint32_t)p.c.h_kv);
    int s = 0, qa, qb, local;
    if (a.per_seq) {
        s = slot / a.per_seq;
        if (s >= n) return false;
        qa = p.cu_q ? clamp_to(p.cu_q[s], total) : s;
        qb = p.cu_q ? clamp_to(p.cu_q[s + 1], total) : s + 1;
        local = slot - s * a.per_seq;
    } else if (n <= 64) {
        // A lane a sequence, the longest first: their tiles take longest, and what ends last then is short.
        const int lane = threadIdx.x & 63;
        int tiles = 0, len = -1;
        if (lane < n) {
            const int rows = rows_of(p, clamp_to(p.cu_q ? p.cu_q[lane + 1] : lane + 1, total) - clamp_to(p.cu_q ? p.cu_q[lane] : lane, total), g);
            tiles = rows < a.rows_from || rows > a.rows_to ? 0 : (rows + M - 1) / M;
            len = max(p.lens[lane], -1);
        }
        int before = 0;  // tiles of the sequences that come before the lane's
        for (int x = 0; x < n; ++x) {
            const int other = __builtin_amdgcn_readlane(len, x);
            before += other > len || (other == len && x < lane) ? __builtin_amdgcn_readlane(tiles, x) : 0;
        }
        const uint64_t here = __ballot(slot >= before && slot < before + tiles);
        if (!here) return false;
        s = __builtin_ctzll(here);
        qa = clamp_to(p.cu_q ? p.cu_q[s] : s, total);
        qb = clamp_to(p.cu_q ? p.cu_q[s + 1] : s + 1, total);
        local = slot - __builtin_amdgcn_readlane(before, s);
    } else if (n <= kExactSeqs) {
        // the tiles of the sequences that are taken, one after another: a lane counts a sequence's
        const int lane = threadIdx.x & 63;
        int before = 0;
        for (; s < n; s += 64) {
            const int x = s + lane;
            int tiles = 0;
            if (x < n) {
                const int rows = rows_of(p, clamp_to(p.cu_q ? p.cu_q[x + 1] : x + 1, total) - clamp_to(p.cu_q ? p.cu_q[x] : x, total), g);
                tiles = rows < a.rows_from || rows > a.rows_to ? 0 : (rows + M - 1) / M;
            }
            int upto = tiles;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int y = __shfl_up(upto, off, 64);
                upto += lane >= off ? y : 0;
            }
            const uint64_t past = __ballot(before + upto > slot);
            if (past) {
                const int l = __builtin_ctzll(past);
                before += __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l);
                s += l;
                break;
            }
            before += __builtin_amdgcn_readlane(upto, 63);
        }
        if (s >= n) return false;
        qa = clamp_to(p.cu_q ? p.cu_q[s] : s, total);
        qb = clamp_to(p.cu_q ? p.cu_q[s + 1] : s + 1, total);
        local = slot - before;
    } else {
        // sequence s has the slots [floor(cu[s] g / M) + s, floor(cu[s + 1] g / M) + s + 1): disjoint, in order
        // and enough; it is looked for 64 sequences at a time, one a lane
        const int lane = threadIdx.x & 63;
        auto base = [&](int x) { return (int)((int64_t)clamp_to(p.cu_q ? p.cu_q[x] : x, total) * g / M) + x; };
        for (int span = n; span > 1;) {  // the sequence is in [s, s + span)
            const int step = (span + 63) / 64, at = s + lane * step;
            const bool before = lane * step < span && (lane == 0 || base(at) <= slot);
            const int x = 63 - __builtin_clzll(__ballot(before) | 1);  // the last lane not past the slot
            s += x * step;
            span = span - x * step < step ? span - x * step : step;
        }
        s = __builtin_amdgcn_readfirstlane(s);
        qa = p.cu_q ? clamp_to(p.cu_q[s], total) : s;
        qb = p.cu_q ? clamp_to(p.cu_q[s + 1], total) : s + 1;
        local = slot - ((int)((int64_t)qa * g / M) + s);
    }
    return span_at<M>(a, s, qa, qb, length_of(p, s), local, t);
}

// What a workgroup takes of a tile: virtual positions [rg * range, rg * range + range). Its sums, where the
// tile has others, go to the workspace's rows from `at` on; for the join, at is that of range 0, the next lie
// `step` after one another.
struct Part {
    Span t;
    int64_t range, at, step;
    int rg;
};

// A share's least unit: the positions that a workgroup's four waves take in a step.
constexpr int kStep = 128;

// The call's positions divided over about a.share workgroups by the lengths that the sequences have, one a
// lane: its tiles, the ranges of each, and the workgroups before its own. Lengths are only known here; ranges
// of a bound on them are too long for what is shorter, and fill the chip badly (16 sequences of 4 tokens, of up
// to 8192 positions, 82 us against 72). The last range of a tile is the shortest; in whole steps of the workgroup it would be
// shorter still, and the same for one XCD in eight (64 us against 59 for 32 sequences behind a window).
template <int M>
struct Shares {
    int qa, qb, len, tiles, steps, ranges, before;  // of the lane's sequence

    // Sums of the lanes up to each.
    __device__ __forceinline__ static int upto(int x)
    {
        x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // row_shr:1
        x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
        x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
        x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
        x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast:15, :31
        x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
        return x;
    }

    __device__ __forceinline__ explicit Shares(const ExtendArgs& a)
    {
        const ExtendCall& p = a.c;
        const int lane = threadIdx.x & 63, g = p.d.h_q / p.c.h_kv, total = (int)p.d.total_q;
        qa = qb = len = tiles = steps = 0;
        if (lane < (int)p.c.n) {
            qa = clamp_to(p.cu_q ? p.cu_q[lane] : lane, total);
            qb = clamp_to(p.cu_q ? p.cu_q[lane + 1] : lane + 1, total);
            len = length_of(p, lane);
            const int rows = rows_of(p, qb - qa, g);
            int sight = len - (qb - qa) + (qb - qa < p.d.max_q ? qb - qa : (int)p.d.max_q);  // to the last row's
            sight = sight < a.longest ? sight : a.longest;
            tiles = rows <= 0 || rows < a.rows_from || rows > a.rows_to ? 0 : (rows + M - 1) / M;
            steps = sight <= kStep ? 1 : (sight + kStep - 1) / kStep;
        }
        // the share of one: as short as keeps all of them running at once, for what comes late costs a round
        const int mine = tiles * p.c.h_kv;
        int per = max((__builtin_amdgcn_readlane(upto(mine * steps), 63) + a.share - 1) / a.share, a.least), sums;
        for (int x = 0;; ++x, per += (per + 15) / 16) {
            ranges = (int)((uint32_t)(steps + per - 1) / (uint32_t)per);
            sums = upto(mine * ranges);
            if (x == 8 || __builtin_amdgcn_readlane(sums, 63) <= a.share) break;
        }
        before = sums - mine * ranges;
    }

    // Positions of a range of sequence s, whole steps of a wave.
    __device__ __forceinline__ int64_t range(int s) const
    {
        const int n = __builtin_amdgcn_readlane(ranges, s);
        return (int64_t)(((uint32_t)__builtin_amdgcn_readlane(steps, s) * (kStep / 32) + n - 1) / (uint32_t)n) * 32;
    }

    __device__ __forceinline__ bool span(const ExtendArgs& a, int s, int local, Span* t) const
    {
        return span_at<M>(a, s, __builtin_amdgcn_readlane(qa, s), __builtin_amdgcn_readlane(qb, s),
                          __builtin_amdgcn_readlane(len, s), local, t);
    }
};

// A workgroup's part, or false where there is none.
template <int M>
__device__ __forceinline__ bool find_part(const ExtendArgs& a, uint32_t index, Part* x)
{
    const ExtendCall& p = a.c;
    if (!a.share) {
        // ranges of one index lie together in the grid: late ones, which few tiles have, spread over all XCDs
        const uint32_t units = (uint32_t)a.slots * (uint32_t)p.c.h_kv;
        if (index >= units * (uint64_t)a.ranges) return false;  // past the grid's end
        index = together(a, index);
        x->at = (int64_t)index * M;
        const uint32_t unit = index % units;
        x->rg = (int)(index / units);
        x->range = a.range;
        return find_span<M>(a, unit, &x->t);
    }
    const uint32_t h = (uint32_t)p.c.h_kv, parts = (uint32_t)a.share + (uint32_t)a.slots * h;
    if (index >= parts) return false;  // past the grid's end
    const Shares<M> sh(a);
    const int slot = (int)index;
    const uint64_t here = __ballot(slot >= sh.before && slot < sh.before + sh.tiles * sh.ranges * p.c.h_kv);
    if (!here) return false;
    const int s = __builtin_ctzll(here);
    SharePart w;
    if (!share_part(index, (uint32_t)__builtin_amdgcn_readlane(sh.before, s), (uint32_t)__builtin_amdgcn_readlane(sh.tiles, s),
                    (uint32_t)__builtin_amdgcn_readlane(sh.ranges, s), h, parts, &w))
        return false;
    x->rg = (int)w.rg;
    x->t.head = (int)w.head;
    x->at = (int64_t)w.at * M;
    x->range = sh.range(s);
    return sh.span(a, s, (int)w.tile, &x->t);
}

// The first row of a tile in a workspace by rows, of range 0.
__device__ __forceinline__ int64_t packed_row(const ExtendArgs& a, const Span& t)
{
    return t.head * a.packed + t.q0 * t.g + t.row0;
}

// The parts of a unit, a tile of a KV head, or false where it has one or none; rg is their number.
template <int M>
__device__ __forceinline__ bool find_parts(const ExtendArgs& a, uint32_t unit, Part* x)
{
    const ExtendCall& p = a.c;
    if (!a.share) {
        if (!find_span<M>(a, unit, &x->t)) return false;
        x->at = a.packed ? packed_row(a, x->t) : (int64_t)unit * M;
        x->step = a.packed ? a.packed * p.c.h_kv : (int64_t)a.slots * p.c.h_kv * M;
        x->range = a.range;
    } else {
        const Shares<M> sh(a);
        const int slot = (int)(unit / (uint32_t)p.c.h_kv), upto = sh.upto(sh.tiles);
        const uint64_t here = __ballot(slot >= upto - sh.tiles && slot < upto);
        if (!here) return false;
        const int s = __builtin_ctzll(here), tiles = __builtin_amdgcn_readlane(sh.tiles, s);
        const int local = slot - (__builtin_amdgcn_readlane(upto, s) - tiles);
        x->t.head = (int)(unit - (uint32_t)slot * (uint32_t)p.c.h_kv);
        if (!sh.span(a, s, local, &x->t)) return false;
        const int before = __builtin_amdgcn_readlane(sh.before, s);
        if (!block_fits((uint32_t)before, (uint32_t)tiles, (uint32_t)__builtin_amdgcn_readlane(sh.ranges, s), (uint32_t)p.c.h_kv,
                        (uint32_t)a.share + (uint32_t)a.slots * (uint32_t)p.c.h_kv))
            return false;  // nobody wrote its sums
        x->step = (int64_t)tiles * p.c.h_kv * M;
        x->at = ((int64_t)before + (int64_t)local * p.c.h_kv + x->t.head) * M;
        x->range = sh.range(s);
    }
    if (x->t.len <= x->range) return false;  // written by its only workgroup
    x->rg = (int)((x->t.len + x->range - 1) / x->range);
    return true;
}

}  // namespace
}  // namespace gdn
