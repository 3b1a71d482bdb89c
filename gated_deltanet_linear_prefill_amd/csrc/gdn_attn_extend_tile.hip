// gdn_attn_extend_tile.hip -- attention of new tokens over the paged cache: sequences with many rows.
//
// The matrix form, the padded LDS groups and the step are those of gdn_attn_prefill.hip
// (gdn_attn_tile.hpp); what differs is where keys come from and which of them a row sees. A staged
// group is 1 KiB of consecutive keys and never crosses a page (pages are 16 keys or more, virtual
// positions skip whole blocks of 16): each wave holds a unit's page ids, one 16-position block a
// lane, loaded a unit ahead, and takes a group's from there into the scalar unit, where its address
// and how many of its bytes exist are formed; the rest of a group reads as zeros.
//
// Bound by the matrix units and the softmax between them, which a wave does one after the other and two waves
// of a SIMD overlap in part: 8192 tokens behind a window of 4096, d = 128, 16/2 heads, 286 us (0.97 PFLOP/s, 48% of the
// cycles in matrix instructions, with 145 vector instructions to 32 of them in a step); 4096 tokens after
// 28672, d = 256, 16/2 heads 1.84 ms (1.13 PFLOP/s; 1.81 from a packed copy); 24 sequences of 1 to 700 tokens
// after up to 4096, 32/8 heads, d = 128, 335 us. Two groups of waves of which one multiplies while the other
// takes its softmax were slower (406 us of the first): their registers did not fit.
//
// fp8 pages are staged as codes, 8 KiB of LDS, and converted to bf16 beside the step that uses the unit
// before: 512 tokens after 32256, d = 256, 16/2 heads 285 us with 16 of join (converted on their way from
// global memory by the threads that wait for them: 1067).
//
// Ranges. A tile's keys are divided into ranges of a fixed length where the tiles alone would not fill
// the chip, and joined by the second kernel of gdn_attn_extend.hip.
#include "gdn_extend.hpp"

namespace gdn {
namespace {

// 128 rows, two workgroups a CU: one starts and ends while the other computes.
using Twin = Shape<4, 1, 1, 2>;
// 128 rows; half the waves take the first of two steps and half the second, and are joined at the end:
// half the sums that ranges write.
using Split = Shape<8, 2, 2, 2>;
// 256 rows share every staged key: the least traffic.
using Wide = Shape<8, 2, 1, 2>;
// The same for an fp8 store, whose codes take LDS of their own beside the bf16 keys.
using Codes8 = Shape<8, 1, 1, 2>;
// fp32 with d = 256, where a wave's O and Q take all of 256 registers.
using Lone = Shape<4, 1, 1, 1>;

// Every wave's loads to LDS have landed, and every wave is past its reads of LDS. The wait is one that the
// compiler sees (vmcnt 0, lgkmcnt 0): it would otherwise wait, before a buffer is read, for loads that
// were issued to the other one since, where it cannot count them.
__device__ __forceinline__ void landed_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What a row sees of a step: `span` keys from the window's first on; in steps with sinks or with absent pages
// (blocks of 16, a bit each) more and less.
struct SeesWindow {
    static constexpr bool RARE = true;
    int lo;
    uint32_t span;
    int sink;
    uint32_t gone;
    bool other;
    __device__ __forceinline__ bool operator()(int key) const { return (uint32_t)(lo + key) < span; }
    __device__ __forceinline__ bool rare() const { return other; }
    __device__ __forceinline__ bool rarely(int key) const
    {
        return ((uint32_t)(lo + key) < span || key < sink) && !(gone >> ((uint32_t)key / 16) & 1);
    }
};

// What is the same in all lanes, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x)
{
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)x));
}

template <typename T, bool FP8, int D, bool LSE, typename S>
__global__ void __launch_bounds__(64 * S::WAVES, S::PER_SIMD) extend_tile_kernel(ExtendArgs a)
{
    using C = Tile<T, D>;
    static_assert(!FP8 || (sizeof(T) == 2 && S::WAVES == 8 && S::STEPS == 1 && S::SPLIT == 1), "what codes are staged for");
    constexpr int N = C::N, UNIT = S::STEPS * N, M = S::ROWS, ND = D / 32, SPLIT = S::SPLIT, ES = C::ES;
    constexpr int BLOCKS = UNIT / 16;  // 16-position blocks of a unit
    static_assert(BLOCKS <= 64, "a lane each");
    // separate arrays: the compiler then knows that reading one need not wait for the loads that
    // are filling another
    __shared__ __align__(16) char s_k0[S::STEPS * C::GROUPS * C::KG], s_k1[S::STEPS * C::GROUPS * C::KG];
    __shared__ __align__(16) char s_v0[S::STEPS * C::GROUPS * C::VG], s_v1[S::STEPS * C::GROUPS * C::VG];
    // fp8: the codes of a unit's K and V, 8 KiB each, and their scales
    __shared__ __align__(16) char s_r0[FP8 ? 2 * UNIT * D : 16], s_r1[FP8 ? 2 * UNIT * D : 16];
    __shared__ __align__(16) char s_c0[FP8 ? 2 * UNIT : 16], s_c1[FP8 ? 2 * UNIT : 16];
    const ExtendCall& p = a.c;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5;
    const int rw = wave % (S::WAVES / SPLIT), turn = wave / (S::WAVES / SPLIT);  // 32 rows, steps
    const uint32_t units = (uint32_t)a.slots * (uint32_t)p.c.h_kv;
    const uint32_t unit = block_index() % units;
    const int rg = (int)(block_index() / units);
    if (rg >= a.ranges) return;  // past the grid's end
    Span w;
    if (!find_span<M>(a, unit, &w)) return;
    const int64_t begin64 = rg * a.range;
    if (rg > 0 && begin64 >= w.len) return;  // the join does not read this range
    const bool whole = w.len <= a.range;     // nothing to join
    // from here on a key's number is its virtual position's distance from `begin`
    const int begin = (int)begin64, valid = w.len - begin;
    const int keys = valid < a.range ? valid : (int)a.range;

    // K: row lane & 31 of a product is place (lane & 31) / GROUPS of group (lane & 31) % GROUPS. V,
    // bf16: the reads of 16 lanes cover groups 4 half + 0..3, 16 elements of each, the next 16
    // lanes the next 16; fp32: a half reads 32 elements of one group, 4 half on
    const int klane = lane % C::GROUPS * C::KG + lane % 32 / C::GROUPS * C::ROWB + half * 16;
    const int vlane = ES == 2 ? (4 * half + ((lane >> 2) & 3)) * C::VG + ((lane >> 4) & 1) * 32 + (lane & 3) * 8
                              : 4 * half * C::VG + lane % 32 * 4;

    // Page ids of the unit from key v0 on, a block a lane. Blocks past the end are as its last.
    const int32_t* table = p.c.page_table + w.seq * p.c.max_pages;
    auto pages_of = [&](int v0) __attribute__((always_inline)) {
        const int v = begin + v0 + 16 * (lane < BLOCKS ? lane : BLOCKS - 1);
        return table[w.pos(v < w.len ? v : w.len - 1) >> a.page_shift];
    };
    auto absent = [&](int id) __attribute__((always_inline)) { return id < 0 || id >= p.c.num_pages; };
    // Stages the unit from key v0 on, whose pages are `ids`, and loads those of the unit after it (before
    // the keys: loads are waited for in their order, and these are not to wait for the keys'). Returns the
    // unit's blocks that are not there, a bit each.
    const char* kpool = static_cast<const char*>(p.c.k);
    const char* vpool = static_cast<const char*>(p.c.v);
    int ids = 0;
    auto fetch = [&](int v0, char* sk, char* sv) __attribute__((always_inline)) {
        asm volatile("" : "+v"(ids));  // not looked at before the barrier that this follows
        const int now = absent(ids) ? -1 : ids;
        ids = pages_of(v0 + UNIT);
        // A wave stages consecutive keys, at most 16 of which lie in one block and need one address. It starts
        // at another group than its neighbours, whose runs are a multiple of the memory channels' stride away.
        constexpr int MINE = UNIT / S::WAVES, RUN = MINE < 16 ? MINE : 16, GR = RUN / C::ROWS;
#pragma unroll
        for (int y = 0; y < MINE / RUN; ++y) {
            const int first = wave * MINE + y * RUN, v = v0 + first;
            const int id = __builtin_amdgcn_readlane(now, first / 16), left = id < 0 ? 0 : valid - v;
            const int64_t row = uniform((((int64_t)(id < 0 ? 0 : id) * p.c.h_kv + w.head) << a.page_shift) +
                                        (w.pos(begin + v) & (p.c.page_size - 1)));
            const int bytes = __builtin_amdgcn_readfirstlane((left >= RUN ? RUN : left <= 0 ? 0 : left) * C::ROWB);
            const __amdgpu_buffer_rsrc_t rk = make_rsrc(kpool + row * C::ROWB, bytes), rv = make_rsrc(vpool + row * C::ROWB, bytes);
#pragma unroll
            for (int i = 0; i < GR; ++i) {
                const int gi = (i + wave) % GR, at = first / C::ROWS + gi;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (__attribute__((address_space(3))) void*)(sk + at * C::KG), 16, lane * 16, gi * 1024, 0, 0);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (__attribute__((address_space(3))) void*)(sv + at * C::VG), 16, lane * 16, gi * 1024, 0, 0);
            }
        }
        return (uint32_t)__ballot(lane < BLOCKS && now < 0);
    };
    // The same for codes: 1 KiB of K and of V a wave, and the scales by the first two waves.
    auto fetch_codes = [&](int v0, char* raw, char* scales) __attribute__((always_inline)) {
        asm volatile("" : "+v"(ids));
        const int now = absent(ids) ? -1 : ids;
        ids = pages_of(v0 + UNIT);
        constexpr int RUN = UNIT / 8;
        const int first = wave * RUN, v = v0 + first;
        const int id = __builtin_amdgcn_readlane(now, first / 16), left = id < 0 ? 0 : valid - v;
        const int64_t row = uniform((((int64_t)(id < 0 ? 0 : id) * p.c.h_kv + w.head) << a.page_shift) +
                                    (w.pos(begin + v) & (p.c.page_size - 1)));
        const int bytes = __builtin_amdgcn_readfirstlane((left >= RUN ? RUN : left <= 0 ? 0 : left) * D);
        load_to_lds(make_rsrc(kpool + row * D, bytes), raw + wave * 1024, lane * 16);
        load_to_lds(make_rsrc(vpool + row * D, bytes), raw + UNIT * D + wave * 1024, lane * 16);
        if (wave < 2 && lane < UNIT / 4) {  // four keys a lane; of absent pages and past the end any, not used
            const int at = __shfl(now, lane / 4), vb = begin + v0 + lane / 4 * 16;
            const int pos = w.pos(vb < w.len ? vb : (w.len - 1) & ~15);
            const uint8_t* from = (wave == 0 ? p.c.k_scale : p.c.v_scale) +
                                  ((((int64_t)(at < 0 ? 0 : at) * p.c.h_kv + w.head) << a.page_shift) + (pos & (p.c.page_size - 1)) + lane % 4 * 4);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                             (__attribute__((address_space(3))) void*)(scales + wave * UNIT), 4, 0, 0);
        }
        return (uint32_t)__ballot(lane < BLOCKS && now < 0);
    };
    // Codes that have arrived to bf16 in the places where keys are staged: 16 of K and of V a thread. A value is
    // its code times a power of two, which bf16 holds exactly (but below its normal range).
    auto convert = [&](int v0, uint32_t gone, const char* raw, const char* scales, char* sk, char* sv) __attribute__((always_inline)) {
        const int row = threadIdx.x / (D / 16), at = row / C::ROWS, to = row % C::ROWS * C::ROWB + threadIdx.x % (D / 16) * 32;
        const bool there = v0 + row < valid && !(gone >> (row / 16) & 1);  // elsewhere codes are 0, scales anything
        auto write = [&](const char* codes, int scale, char* dst) __attribute__((always_inline)) {
            const u32x4_t x = *reinterpret_cast<const u32x4_t*>(codes + threadIdx.x * 16);
            const float f = __uint_as_float((uint32_t)(there ? scale : 127) << 23);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4_t y;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    y[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * h + i], f, false));
                    y[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * h + i], f, true));
                }
                *reinterpret_cast<u32x4_t*>(dst + to + 16 * h) = y;
            }
        };
        const uint8_t* sc = reinterpret_cast<const uint8_t*>(scales);
        write(raw, sc[row], sk + at * C::KG);
        write(raw + UNIT * D, sc[UNIT + row], sv + at * C::VG);
    };
    uint32_t gone0 = 0, gone1 = 0;
    auto start = [&]() __attribute__((always_inline)) {
        if (keys <= 0) return;
        ids = pages_of(0);
        if constexpr (FP8) {
            gone0 = fetch_codes(0, s_r0, s_c0);
            if (UNIT < keys) gone1 = fetch_codes(UNIT, s_r1, s_c1);
            landed_barrier();
            convert(0, gone0, s_r0, s_c0, s_k0, s_v0);
        } else {
            gone0 = fetch(0, s_k0, s_v0);
        }
    };
    start();

    // What rows see: keys below upto that are at or past from, or sinks. Of the wave's first row, its last,
    // and this lane's.
    const int window = (int)p.d.window, sinks = (int)p.d.sinks - begin;
    auto end_of = [&](int row) {
        const int pos = w.shift + (int)((uint32_t)(row < w.rows ? row : w.rows - 1) / (uint32_t)w.g);
        return pos < w.skip ? 0 : pos + 1 - w.skip;
    };
    auto from_of = [&](int end) { return (window && end > window ? end - window : 0) - begin; };
    const int wfirst = w.row0 + 32 * rw, wlast = end_of(wfirst + 31);
    const int wall = end_of(wfirst) - begin, wkeys = (wfirst < w.rows ? wlast : 0) - begin, wfrom = from_of(wlast);
    const int r = wfirst + (lane & 31), rc = r < w.rows ? r : w.rows - 1, pos = (int)((uint32_t)rc / (uint32_t)w.g);
    const int upto = end_of(r) - begin, from = from_of(end_of(r));

    const char* qp = static_cast<const char*>(p.q) +
                     ES * ((w.q0 + pos) * p.d.q_token + (w.head * w.g + (rc - pos * w.g)) * p.d.q_head) + 16 * half;
    // A negative scale becomes a positive one of the negated query, zero the smallest positive number: see
    // gdn_attn_prefill.hip.
    const uint32_t flip = p.d.scale < 0.f ? (ES == 2 ? 0x80008000u : 0x80000000u) : 0u;
    const float c = fmaxf(fabsf(p.d.scale) * kLog2e, 0x1p-149f);
    u32x4_t q[D / (2 * C::PER)];  // piece kk: elements 2 PER kk + PER half ..
#pragma unroll
    for (int kk = 0; kk < D / (2 * C::PER); ++kk) q[kk] = *reinterpret_cast<const u32x4_t*>(qp + 32 * kk) ^ flip;

    f32x16_t o[ND];
    Stats st;
    bool odd = false;
    auto step = [&](auto mode, const char* sk, const char* sv, int j0, uint32_t gone) __attribute__((always_inline)) {
        constexpr int MODE = decltype(mode)::value;
        if (MODE != kPlain && j0 >= wkeys) return;  // nothing there for this wave's rows
        gone &= (1u << (N / 16)) - 1;
        const bool masked = j0 + N > wall || (j0 < wfrom && j0 + N > sinks) || gone != 0;
        const SeesWindow sees = {j0 - from, (uint32_t)max(upto - from, 0), min(sinks, upto) - j0, gone, gone != 0 || j0 < sinks};
        attn_step<T, D, LSE, MODE>(sk, sv, klane, vlane, q, o, st, c, masked, sees, lane, odd);
    };
    auto use = [&](auto mode, const char* sk, const char* sv, int j0, uint32_t gone) __attribute__((always_inline)) {
        if constexpr (SPLIT == 2) {
            step(mode, sk + turn * C::GROUPS * C::KG, sv + turn * C::GROUPS * C::VG, j0 + turn * N, gone >> (turn * (N / 16)));
        } else {
#pragma unroll 1
            for (int t = 0; t < S::STEPS; ++t)
                step(mode, sk + t * C::GROUPS * C::KG, sv + t * C::GROUPS * C::VG, j0 + t * N, gone >> (t * (N / 16)));
        }
    };
    // Two buffers: while the steps in one are used those in the other arrive. The barrier before
    // a use has every wave's loads of it landed, and every wave past the buffer refilled next. Codes arrive a
    // unit earlier, in buffers of their own, and are converted while the unit before them is used.
    auto pair = [&](auto mode, int j0) __attribute__((always_inline)) {
        landed_barrier();
        if constexpr (FP8) {
            uint32_t gone = 0;
            if (j0 + 2 * UNIT < keys) gone = fetch_codes(j0 + 2 * UNIT, s_r0, s_c0);
            if (j0 + UNIT < keys) convert(j0 + UNIT, gone1, s_r1, s_c1, s_k1, s_v1);
            use(mode, s_k0, s_v0, j0, gone0);
            gone0 = gone;
            if (j0 + UNIT >= keys) return;
            landed_barrier();
            gone = 0;
            if (j0 + 3 * UNIT < keys) gone = fetch_codes(j0 + 3 * UNIT, s_r1, s_c1);
            if (j0 + 2 * UNIT < keys) convert(j0 + 2 * UNIT, gone0, s_r0, s_c0, s_k0, s_v0);
            use(mode, s_k1, s_v1, j0 + UNIT, gone1);
            gone1 = gone;
        } else {
            if (j0 + UNIT < keys) gone1 = fetch(j0 + UNIT, s_k1, s_v1);
            use(mode, s_k0, s_v0, j0, gone0);
            if (j0 + UNIT >= keys) return;
            landed_barrier();
            if (j0 + 2 * UNIT < keys) gone0 = fetch(j0 + 2 * UNIT, s_k0, s_v0);
            use(mode, s_k1, s_v1, j0 + UNIT, gone1);
        }
    };
    // Whether all rows see all of two units: the second's pages are in `ids` when it is asked, or in gone1.
    const int tend = end_of(w.row0) - begin, tfrom = from_of(end_of(w.row0 + M - 1));
    auto plain = [&](int j0) __attribute__((always_inline)) {
        return j0 >= tfrom && j0 + 2 * UNIT <= tend && j0 + 2 * UNIT <= keys && gone0 == 0 &&
               (FP8 ? gone1 == 0 : !__any(lane < BLOCKS && absent(ids)));
    };
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[db][i] = 0.f;
        st = Stats{-INFINITY, 0.f, 0.f};
    };
    clear();
    // In order: the window's edge, what all rows see, the causal edge (or all from the first absent page on).
    // O stays in place from loop to loop: without the pins d = 128 kept two copies of it, one in scratch memory
    // (2.4 times the time).
    auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int db = 0; db < ND; ++db) asm volatile("" : "+v"(o[db]));
    };
    int j0 = 0;
    for (; j0 < keys && !plain(j0); j0 += 2 * UNIT) pair(std::integral_constant<int, kMasks>{}, j0);
    pin();
    for (; j0 < keys && plain(j0); j0 += 2 * UNIT) pair(std::integral_constant<int, kPlain>{}, j0);
    pin();
    for (; j0 < keys; j0 += 2 * UNIT) pair(std::integral_constant<int, kMasks>{}, j0);
    if (__syncthreads_or(odd)) {  // rare: the whole tile again
        clear();
        start();
        for (j0 = 0; j0 < keys; j0 += 2 * UNIT) pair(std::integral_constant<int, kOdd>{}, j0);
        __syncthreads();  // the buffers are written to below
    }

    if constexpr (SPLIT == 2) {
        // O of the second steps' waves through LDS: D / 2 registers of 64 lanes a wave, in the
        // buffers of K and V, a row group in each
        static_assert(D / 2 * 256 <= S::STEPS * C::GROUPS * C::KG, "a wave's O fits a buffer");
        float* so = reinterpret_cast<float*>(rw == 0 ? s_k0 : rw == 1 ? s_k1 : rw == 2 ? s_v0 : s_v1);
        __shared__ float s_st[4][3][64];
        if (turn == 1) {
#pragma unroll
            for (int db = 0; db < ND; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) so[(16 * db + i) * 64 + lane] = o[db][i];
            s_st[rw][0][lane] = st.m;
            s_st[rw][1][lane] = st.l;
            s_st[rw][2][lane] = st.exact;
        }
        __syncthreads();
        if (turn == 1) return;
        const float m1 = s_st[rw][0][lane], mm = fmaxf(st.m, m1);
        const float a0 = st.m == -INFINITY ? 0.f : rescaled(st.m, mm, c);
        const float a1 = m1 == -INFINITY ? 0.f : rescaled(m1, mm, c);
        st.m = mm;
        st.l = a0 * st.l + a1 * s_st[rw][1][lane];
        st.exact = a0 * st.exact + a1 * s_st[rw][2][lane];
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[db][i] = a0 * o[db][i] + a1 * so[(16 * db + i) * 64 + lane];
    }
    if (!whole) {  // this range's sums, for the join
        const float l = other_half_sum(st.l), e = ES == 2 && LSE ? other_half_sum(st.exact) : l;
        const int64_t at = rg * a.packed * p.c.h_kv + packed_row(a, w) + 32 * rw + (lane & 31);
        if (r < w.rows) {
            float* to = a.part_o + at * D + 4 * half;
#pragma unroll
            for (int db = 0; db < ND; ++db)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<f32x4_t*>(to + 32 * db + 8 * i) =
                        f32x4_t{o[db][4 * i], o[db][4 * i + 1], o[db][4 * i + 2], o[db][4 * i + 3]};
            if (half == 0) a.part_ml[at] = make_float4(st.m * c, l, e, 0.f);
        }
        return;
    }
    // All waves have met since the last use of K and V: each has a part of the buffers to itself (with
    // SPLIT 2 in the one where it read the other half's O).
    constexpr int PART = 32 * ((C::ROWB < 256 ? C::ROWB : 256) + 16), PER_BUFFER = (M / 32 + 3) / 4;
    char* part;
    if constexpr (FP8) {
        static_assert(PART <= (int)sizeof(s_k0) && 2 * PART <= (int)sizeof(s_v0) && PART <= (int)sizeof(s_r0), "eight parts");
        part = rw == 0 ? s_k0 : rw == 1 ? s_k1 : rw < 4 ? s_v0 : rw < 6 ? s_v1 : rw == 6 ? s_r0 : s_r1;
        if (rw == 3 || rw == 5) part += PART;
    } else {
        static_assert(PER_BUFFER * PART <= (int)sizeof(s_k0), "the waves' parts fit the buffers");
        const int buffer = rw / PER_BUFFER;
        part = (buffer == 0 ? s_k0 : buffer == 1 ? s_k1 : buffer == 2 ? s_v0 : s_v1) + rw % PER_BUFFER * PART;
    }
    st.m *= c;
    write_rows<T, D>(p, w, wfirst, lane, o, st, part);
}

enum { kTwin, kSplit, kWide, kLone, kCodes };

// Measured (us of a call, bf16, Twin / Split / Wide; tiles of 128 rows, all KV heads; Split's and Wide's keys in
// ranges where tiles are few). Few tiles: d = 256, 16/2 heads, 128 new tokens after 8192 (16) 51 / 46 / 63, 512 (64)
// 102 / 95 / 99, 1024 (128) 170 / 165 / 165, 2048 (256) 336 / 312 / 313; d = 128, 32/8 heads 512 (128)
// 95 / 92, 1024 (256) 173 / 158; d = 64, 16/16 heads 1024 (128) 77 / 71. 512 tiles: d = 256 4096 from the start 187 /
// 158 / 205, after 8192 650 / 645 / 660, after 30000 1960 / 1965 / 1890; d = 128 2048 after 8192 317 / 324. More: d = 256
// 8192 from the start (1024) 539 / 546 / 500, 8 sequences of 100 to 2000 after 4000 376 / 380 / 397; d = 128 4096
// after 8192 (1024) 671 / 695, 16 prompts of 1 to 2500 307 / 393; d = 64 8192 (1024) 209 / 227.
int shape_of(const gdn_kv_cache& c, const gdn_extend_dims& d)
{
    if (c.store == GDN_FP8) return kCodes;
    if (d.dtype == GDN_F32 && c.d == 256) return kLone;
    const int64_t tiles = d.total_q * d.h_q / 128;
    if (tiles <= 256) return kSplit;
    if (c.d == 256 && d.dtype == GDN_BF16) {
        if (c.n == 1 && tiles >= 512 && (tiles > 512 || d.max_len >= 16384)) return kWide;
        if (tiles <= 512) return kSplit;
    }
    return kTwin;
}

template <typename T, bool FP8, int D, bool LSE, typename S>
hipError_t launch_kernel(const ExtendCall& c, const ExtendPlan& pl, void* ws)
{
    const ExtendArgs a = extend_args(c, pl, ws);
    hipLaunchKernelGGL((extend_tile_kernel<T, FP8, D, LSE, S>), grid_of(pl.units * pl.ranges), dim3(64 * S::WAVES), 0, c.stream, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || pl.ranges == 1 ? e : launch_extend_join(a, pl.m);
}

template <typename T, int D, bool LSE>
hipError_t launch_shape(const ExtendCall& c, const ExtendPlan& pl, void* ws)
{
    if constexpr (Tile<T, D>::ROWS == 1) {
        return launch_kernel<T, false, D, LSE, Lone>(c, pl, ws);
    } else {
        switch (shape_of(c.c, c.d)) {
            case kSplit: return launch_kernel<T, false, D, LSE, Split>(c, pl, ws);
            case kWide:
                if constexpr (D == 256) return launch_kernel<T, false, D, LSE, Wide>(c, pl, ws);
                else return hipErrorInvalidValue;
            case kCodes:
                if constexpr (sizeof(T) == 2) return launch_kernel<T, true, D, LSE, Codes8>(c, pl, ws);
                else return hipErrorInvalidValue;
            default: return launch_kernel<T, false, D, LSE, Twin>(c, pl, ws);
        }
    }
}

template <int D>
hipError_t launch_d(const ExtendCall& c, const ExtendPlan& pl, void* ws)
{
    if (c.d.dtype == GDN_F32) return launch_shape<float, D, false>(c, pl, ws);
    return c.lse ? launch_shape<uint16_t, D, true>(c, pl, ws) : launch_shape<uint16_t, D, false>(c, pl, ws);
}

}  // namespace

ExtendPlan extend_tile_plan(const gdn_kv_cache& c, const gdn_extend_dims& d)
{
    ExtendPlan p;
    p.share = p.least = 0;
    const int shape = shape_of(c, d);
    p.m = shape == kWide || shape == kCodes ? 256 : 128;
    const int64_t g = d.h_q / c.h_kv;
    p.per_seq = c.n == 1 ? (int)((d.max_q * g + p.m - 1) / p.m) : 0;
    p.slots = c.n == 1 ? p.per_seq : d.total_q * g / p.m + c.n;
    p.units = p.slots * c.h_kv;
    p.packed = d.total_q * g;
    // 256 workgroups of eight waves run at a time. Each costs its keys and what starting, masking, ending and
    // joining take, 15 to 20 us: as long as 280 keys (d = 256; a key takes 75 ns with 128 rows), 700 (128)
    // or 1200 (64). Ranges are those that make this estimate least, as long as the join's grid, which has slots for tiles
    // of all sequences, holds less than 2^31 workgroups.
    const int64_t tiles = (d.total_q * g + p.m - 1) / p.m * c.h_kv, len = extend_longest(c, d, p.m);
    const int64_t over = c.d == 256 ? 280 : c.d == 128 ? 700 : 1200;
    int64_t ranges = 1, least = (tiles + 255) / 256 * (len + over);
    if (shape != kTwin && p.units < (INT64_C(1) << 31) / (p.m * (c.d / 64)))
        for (int64_t r = 2; r <= 64 && len >= 512 * r && tiles * r <= 1024; ++r) {
            const int64_t cost = (tiles * r + 255) / 256 * (len / r + over) + over / 2;
            if (cost < least) {
                least = cost;
                ranges = r;
            }
        }
    const int64_t per = ((len + ranges - 1) / ranges + 255) / 256 * 256;  // whole units of every shape
    p.range = per > 0 ? per : 256;
    p.ranges = len > 0 ? (len + p.range - 1) / p.range : 1;
    return p;
}

hipError_t launch_extend_tiles(const ExtendCall& c, const ExtendPlan& p, void* ws)
{
    switch (c.c.d) {
        case 64: return launch_d<64>(c, p, ws);
        case 128: return launch_d<128>(c, p, ws);
        case 256: return launch_d<256>(c, p, ws);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
