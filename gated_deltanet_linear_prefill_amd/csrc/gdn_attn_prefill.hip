// gdn_attn_prefill.hip -- attention over packed prompts: causal or full, grouped heads.
//
// Rows. The G = h_q / h_kv heads of a KV head read the same keys, so a workgroup's tile is M
// packed query rows of one (sequence, KV head): row r is position r / G, head r % G of the
// group. A tile then reads each key once for all its heads, and its causal edge is M / G
// positions wide.
//
// Grid. The host does not know the sequences' lengths. Sequence s gets the tiles
// [floor(cu_q[s] G / M) + s, floor(cu_q[s + 1] G / M) + s + 1), which are disjoint, in order
// and enough for its ceil(len G / M); a workgroup looks its sequence up in them and leaves
// if its tile is past the end. Tiles are taken last first within a sequence: under a causal
// mask the last are the longest.
//
// Matrix form (32x32 MFMA, one query per lane). S^T = K Q^T puts one query in a column: lane l
// holds query l & 31, and of a 32-key block the keys 8 (i / 4) + 4 (l >> 5) + i % 4, so the
// softmax over keys is in-lane but for one exchange with lane l ^ 32, and O^T = V^T P^T takes
// those registers as its B operand as they are: A and B only have to agree on which key a
// k slot means, so the V^T operand is read with the same permutation (transposing LDS reads).
// Every statistic of a row (maximum, sum, rescaling) is one register in the row's lanes.
//
// Steps. K and V of a step arrive in LDS by direct loads while the step before is used. The
// reference maximum of a row moves only when a score passes it by 2^8 (weights then stay below
// 2^8 and sums far from overflow), so O is rarely rescaled.
//
// Bound by the matrix rate together with the softmax's vector instructions, which the matrix
// instructions of the other wave of a SIMD hide only in part: by the counters 4.6 of them a score
// and lane for a long d = 256 segment, 6.1 for packed d = 128 prompts (masked steps, each tile's
// start and end). Measured, bf16: 4096 tokens after 28672, 16/2 heads, d = 256 1765 us (1705 to
// 1960 by machine), 1.17 PFLOP/s (the library's large product 1.2 to 1.4; matrix units 66% busy); a
// 4096-token prompt 144 us, 0.95 PFLOP/s; 16 packed prompts of up to 2500, 32/8 heads, d = 128
// 275 us, 0.80 PFLOP/s (44% busy). fp32: 4096 tokens, 16/2 heads, d = 256 1140 us, d = 128 530 us,
// 79 and 85% of the fp32 library product's 153 TFLOP/s. 8192 tokens without a mask, bf16,
// d = 256, 128 and 64: without the softmax 7, 12 and 20% less time, with each operand read once
// 10, 9 and 5%, without loads 7, 6 and 4%: no single part is in the way. Few rows: see ranges_of.
//
// Masked keys get weight exactly 0. A matrix product would still turn 0 x NaN into NaN, so
// rows past the end of a sequence are read as zeros, and in steps that hold masked keys a V that
// is not finite is left out of the product and added only to the rows that see its key.
#include <type_traits>

#include "gdn_attn_internal.hpp"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 32 query rows per wave. Of a staged key, a row of D elements; ROWS of them fill the 1 KiB that
// a wave's load to LDS writes, and GROUPS such groups, each padded, are a step of N keys. The key
// of group x, place y is ROWS x + y: the keys of a group lie next to each other in memory, and a
// wave reads one place of all groups together, in banks that the padding keeps apart (K: 16
// bytes a group, for reads of 16 bytes a lane; V: 64 for the transposing reads of 64-byte pieces
// of four groups, 32 for reads of 128 bytes of groups x and x + 4). A reading lane has one
// address; everything else is an instruction offset.
template <typename T, int D>
struct Tile {
    static constexpr int ES = sizeof(T), ROWB = ES * D, ROWS = 1024 / ROWB;
    static constexpr int GROUPS = ROWS == 1 ? 32 : 16, N = GROUPS * ROWS, BLOCKS = N / 32;
    static constexpr int PLACES = 32 / GROUPS;  // places that a 32-key block takes of every group
    static constexpr int KG = 1024 + 16, VG = 1024 + (ES == 2 ? 64 : 32);  // bytes of a padded group
    static constexpr int PER = 16 / ES;  // elements of a 16-byte operand piece
};

// How a workgroup is made up: its waves, the steps that are staged at a time, and over how many
// groups of waves the steps are divided.
template <int WAVES_, int STEPS_, int SPLIT_, int PER_SIMD_, bool RANGES_ = false>
struct Shape {
    static constexpr int WAVES = WAVES_, STEPS = STEPS_, SPLIT = SPLIT_, ROWS = 32 * WAVES / SPLIT;
    static constexpr int PER_SIMD = PER_SIMD_;  // waves that a SIMD should hold
    static constexpr bool RANGES = RANGES_;     // a tile's keys may be divided over workgroups
};
// 256 rows share every staged key: the least traffic, for long work.
using Wide = Shape<8, 2, 1, 2>;
// 128 rows; half the waves take the first of two steps and half the second, and are joined at the
// end: half the time per workgroup, for calls that have too few tiles to keep all CUs busy evenly.
using Split = Shape<8, 2, 2, 2>;
// 64 rows in the same way, one wave a SIMD, and the keys of a tile over several workgroups whose
// sums are joined by a second kernel: for calls whose few tiles leave most CUs idle.
using Few = Shape<4, 2, 2, 1, true>;
// 128 rows, two workgroups a CU: one starts and ends while the other computes, for many short tiles.
using Twin = Shape<4, 1, 1, 2>;
// fp32 with d = 256, where a wave's O and Q take all of 256 registers.
using Lone = Shape<4, 1, 1, 1, true>;

// A workgroup's tile: its sequence's rows and keys, and its own first row. The host keeps
// rows and keys below 2^31 - 2^16.
struct Work {
    int64_t q0, k0;    // first packed rows of the sequence
    int len_q, len_k;
    int row0, rows;    // first (position, head) row of the tile; how many the sequence has
    int g, head;       // heads of the group; KV head
};

__device__ __forceinline__ int clamp_to(int x, int hi)
{
    return x < 0 ? 0 : (x > hi ? hi : x);
}

// The workgroup's work, or false if there is none. floor(cu[s] G / M) + s, the first tile of
// sequence s, is looked for 64 sequences at a time, one a lane.
template <int M>
__device__ __forceinline__ bool find_work(const AttnCall& p, int tile, int head, int lane, Work* w)
{
    const gdn_attn_dims& d = p.d;
    const int g = d.h_q / d.h_kv, n = (int)d.n, total_q = (int)d.total_q, total_k = (int)d.total_k;
    auto base = [&](int s) { return (int)((int64_t)clamp_to(p.cu_q[s], total_q) * g / M) + s; };
    int s = 0;
    for (int span = n; span > 1;) {  // the sequence is in [s, s + span)
        const int step = (span + 63) / 64, at = s + lane * step;
        const bool before = lane * step < span && (lane == 0 || base(at) <= tile);
        const int x = 63 - __builtin_clzll(__ballot(before) | 1);  // the last lane not past the tile
        s += x * step;
        span = span - x * step < step ? span - x * step : step;
    }
    s = __builtin_amdgcn_readfirstlane(s);
    const int qa = clamp_to(p.cu_q[s], total_q), qb = clamp_to(p.cu_q[s + 1], total_q);
    const int ka = clamp_to(p.cu_k[s], total_k), kb = clamp_to(p.cu_k[s + 1], total_k);
    w->q0 = qa;
    w->k0 = ka;
    w->len_q = qb - qa;
    w->len_k = kb > ka ? kb - ka : 0;
    w->rows = w->len_q * g;
    w->g = g;
    w->head = head;
    if (w->len_q <= 0) return false;
    const int tiles = (w->rows + M - 1) / M, local = tile - ((int)((int64_t)qa * g / M) + s);
    if (local < 0 || local >= tiles) return false;
    w->row0 = (tiles - 1 - local) * M;
    return true;
}

// Keys that a query row at position pos sees: [0, limit).
__device__ __forceinline__ int key_limit(const Work& w, int pos, int causal)
{
    return causal ? clamp_to(pos + 1 + w.len_k - w.len_q, w.len_k) : w.len_k;
}

// Keys of one of `ranges` ranges of a tile's keys: whole units, not below 256. ranges is at most 64,
// so that the end of the last stays below 2^31.
__device__ __forceinline__ int range_keys(int keys, int ranges, int unit)
{
    const int per = (keys + ranges - 1) / ranges;
    return ((per < 256 ? 256 : per) + unit - 1) / unit * unit;
}

__device__ __forceinline__ float other_half_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float other_half_sum(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The keys [row, row + STEPS N) of a strided tensor into LDS, in padded groups of GROUP bytes;
// zeros from `valid` rows on. `off` is this lane's byte offset within a group's rows in memory.
template <typename T, int D, typename S, int GROUP>
__device__ __forceinline__ void stage(const char* base, int row, int valid, int64_t stride,
                                      char* lds, int wave, int off)
{
    using C = Tile<T, D>;
#pragma unroll
    for (int i = 0; i < S::STEPS * C::GROUPS / S::WAVES; ++i) {
        const int x = i * S::WAVES + wave;
        const int first = row + x * C::ROWS;
        const int left = valid - first, have = left < C::ROWS ? left : C::ROWS;
        const __amdgpu_buffer_rsrc_t r =
            make_rsrc(base + first * stride, have <= 0 ? 0 : (have - 1) * stride + C::ROWB);
        load_to_lds(r, lds + x * GROUP, off);
    }
}

// The same where all of the keys exist: `base` is this wave's first group's memory, `ahead` the
// bytes from a group of the wave to its next.
template <typename T, int D, typename S, int GROUP>
__device__ __forceinline__ void stage_whole(const char* base, int ahead, char* lds, int wave, int off)
{
    using C = Tile<T, D>;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(base, 0x7fffffff);
#pragma unroll
    for (int i = 0; i < S::STEPS * C::GROUPS / S::WAVES; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            r, (__attribute__((address_space(3))) void*)(lds + (i * S::WAVES + wave) * GROUP), 16, off, i * ahead, 0, 0);
}

// Every wave's loads to LDS have landed, and every wave is past its reads of LDS. A plain barrier
// does not wait for loads to LDS: each wave has to wait for its own before it.
__device__ __forceinline__ void staged_barrier()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ bf16x4_t read_tr(const char* p)
{
    typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 v4;
    const v4 r = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) v4*)(p));
    return __builtin_bit_cast(bf16x4_t, r);
}

__device__ __forceinline__ f32x16_t mfma32(bf16x8_t a, bf16x8_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ bool is_finite(float x)
{
    return fabsf(x) <= 3.4028234e38f;  // false for NaN
}

// Whether any lane holds a NaN or infinity in its 16 bytes of T. bf16: adding one to an all-ones
// exponent carries into the sign's place.
template <typename T>
__device__ __forceinline__ bool any_not_finite(u32x4_t u)
{
    bool odd = false;
    if constexpr (sizeof(T) == 2) {
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) c |= (u[i] & 0x7f807f80u) + 0x00800080u;
        odd = (c & 0x80008000u) != 0;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) odd |= !is_finite(__uint_as_float(u[i]));
    }
    return __any(odd);
}

// The same operand with 0 in the place of NaN and infinities.
__device__ __forceinline__ bf16x8_t only_finite(bf16x8_t x)
{
    u32x4_t u = __builtin_bit_cast(u32x4_t, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t odd = (((u[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 15;
        u[i] &= ~(odd * 0xffffu);
    }
    return __builtin_bit_cast(bf16x8_t, u);
}

__device__ __forceinline__ float only_finite(float x)
{
    return is_finite(x) ? x : 0.f;
}

// Softmax state of a wave's 32 rows: each lane's own query.
struct Stats {
    float m;      // reference maximum (-inf: nothing seen)
    float l;      // sum of the weights of this lane's keys, as they multiply V
    float exact;  // the same before rounding, if lse is wanted and weights are rounded
};

// Writes a wave's 32 rows, divided by their sums. A lane holds 4-element pieces of its own row: they
// go through the wave's part of LDS (256 bytes a row at a time, padded), so that 16 bytes of each
// of 16 lanes are one stretch of memory. `first` is the first of the rows.
template <typename T, int D>
__device__ __forceinline__ void write_rows(const AttnCall& p, const Work& w, int first, int lane,
                                           const f32x16_t* o, const Stats& st, char* lds)
{
    constexpr int ROWB = sizeof(T) * D, PASS = ROWB < 256 ? ROWB : 256, STRIDE = PASS + 16, LPR = PASS / 16;
    constexpr int BLOCKS = PASS / (32 * (int)sizeof(T));  // 32-element blocks of O^T in a pass
    const float l = other_half_sum(st.l), e = sizeof(T) == 2 ? other_half_sum(st.exact) : l;
    const int half = lane >> 5, r = first + (lane & 31), rc = r < w.rows ? r : w.rows - 1;
    const int pos = (int)((uint32_t)rc / (uint32_t)w.g);
    const int64_t row = (w.q0 + pos) * p.d.h_q + w.head * w.g + (rc - pos * w.g);
    if (p.lse && lane < 32 && r < w.rows)
        p.lse[row] = e > 0.f ? (st.m + __builtin_amdgcn_logf(e)) * kLn2 : (e == e ? -INFINITY : e);
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
#pragma unroll
    for (int pass = 0; pass < ROWB / PASS; ++pass) {
#pragma unroll
        for (int x = 0; x < BLOCKS; ++x) {
            const f32x16_t v = o[pass * BLOCKS + x] * inv;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                char* at = lds + (lane & 31) * STRIDE + (32 * x + 8 * i + 4 * half) * (int)sizeof(T);
                if constexpr (sizeof(T) == 2)
                    *reinterpret_cast<u32x2_t*>(at) = u32x2_t{pack_bf16(v[4 * i], v[4 * i + 1]), pack_bf16(v[4 * i + 2], v[4 * i + 3])};
                else
                    *reinterpret_cast<f32x4_t*>(at) = f32x4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            }
        }
        // the wave's own writes, read by its other lanes
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int i = 0; i < 32 * LPR / 64; ++i) {
            const int at = i * (64 / LPR) + lane / LPR;  // of the 32 rows
            const u32x4_t x = *reinterpret_cast<const u32x4_t*>(lds + at * STRIDE + lane % LPR * 16);
            const int64_t to = __shfl(row, at, 64);
            if (first + at < w.rows)
                *reinterpret_cast<u32x4_t*>(static_cast<char*>(p.out) + to * ROWB + pass * PASS + lane % LPR * 16) = x;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// kPlain: every row sees every key. kMasks: where `masked`, some rows may not see some keys, and
// `odd` is set if V holds a NaN or an infinity there. kOdd: for tiles where that was found.
enum { kPlain, kMasks, kOdd };

// The factor of weights relative to maximum `from` when they become relative to `to`. Raw scores may be
// up to the largest float, and their difference twice that: it is halved, which is exact.
__device__ __forceinline__ float rescaled(float from, float to, float c)
{
    return __builtin_amdgcn_exp2f((0.5f * from - 0.5f * to) * (2.f * c));
}

// One step of a wave's 32 rows over N staged keys at sk, sv (klane, vlane: this lane's offsets).
// This lane's row sees the keys below lim (which may be negative, or above N).
template <typename T, int D, bool LSE, int MODE>
__device__ __forceinline__ void attn_step(const char* sk, const char* sv, int klane, int vlane,
                                          const u32x4_t (&q)[D / (32 / sizeof(T))], f32x16_t (&o)[D / 32],
                                          Stats& st, float c, bool masked, int lim, int lane, bool& odd)
{
    using C = Tile<T, D>;
    constexpr bool BF = sizeof(T) == 2;
    constexpr int N = C::N, NB = C::BLOCKS, ND = D / 32, KK = D / (2 * C::PER), PF = 4;
    const int half = lane >> 5;
    // row m of block b of the product is place PLACES b + m / GROUPS of group m % GROUPS; register
    // i of this lane is row 8 (i / 4) + 4 half + i % 4
    auto group_of = [&](int i) { return (8 * (i / 4) + i % 4) % C::GROUPS; };  // and 4 half more
    auto place_of = [&](int b, int i) { return C::PLACES * b + 8 * (i / 4) / C::GROUPS; };

    f32x16_t s[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
    auto k_at = [&](int x) {  // piece x: block x % NB, elements 2 PER (x / NB) + PER half ..
        return *reinterpret_cast<const u32x4_t*>(sk + klane + x % NB * C::PLACES * C::ROWB + x / NB * 32);
    };
    u32x4_t kf[PF];
#pragma unroll
    for (int x = 0; x < PF; ++x) kf[x] = k_at(x);
#pragma unroll
    for (int x = 0; x < KK * NB; ++x) {
        const u32x4_t a = kf[x % PF], b = q[x / NB];
        if constexpr (BF) {
            s[x % NB] = mfma32(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), s[x % NB]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[x % NB] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(b[e]), s[x % NB], 0, 0, 0);
        }
        if (x + PF < KK * NB) kf[x % PF] = k_at(x + PF);
    }

    if (MODE != kPlain && masked) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s[b][i] = C::ROWS * (group_of(i) + 4 * half) + place_of(b, i) < lim ? s[b][i] : -INFINITY;
        if (MODE == kMasks)
#pragma unroll 1
            for (int x = 0; x < C::GROUPS; ++x)
                odd |= any_not_finite<T>(*reinterpret_cast<const u32x4_t*>(sv + x * C::VG + lane * 16));
    }
    float mx = -INFINITY;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
    mx = other_half_max(mx);
    // the reference maximum moves only when weights would pass 2^8: O is then rescaled
    const bool rise = mx > st.m && (st.m == -INFINITY || (mx - st.m) * c > 8.f);
    if (__any(rise)) {
        const float a = !rise ? 1.f : st.m == -INFINITY ? 0.f : rescaled(st.m, mx, c);
        st.m = rise ? mx : st.m;
        st.l *= a;
        if (BF && LSE) st.exact *= a;
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[db][i] *= a;
    }
    const float ref = st.m == -INFINITY ? 0.f : st.m * c;

    // V^T operand x, rows 32 (x % ND) .. of V^T: bf16, keys at place x / ND of every group, in the
    // order of the weights' registers; fp32, the two keys of the register that halves share
    constexpr int NV = (BF ? 2 : 16) * NB * ND;
    auto v_at = [&](int x) {
        if constexpr (BF) {
            const char* at = sv + vlane + x / ND * C::ROWB + x % ND * 64;
            return __builtin_shufflevector(read_tr(at), read_tr(at + 8 * C::VG), 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const int b = x / ND / 16, i = x / ND % 16;
            return *reinterpret_cast<const float*>(sv + vlane + group_of(i) * C::VG + place_of(b, i) * C::ROWB + x % ND * 128);
        }
    };
    using VF = decltype(v_at(0));
    VF vf[PF];
#pragma unroll
    for (int x = 0; x < 2; ++x) vf[x] = v_at(x);
    u32x4_t pw[BF ? 2 * NB : 1];  // bf16 weights as B operands: place y of every group
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], c, -ref));
            s[b][i] = p;
            if constexpr (BF) {
                if (LSE) st.exact += p;
                if (i & 1) {
                    const uint32_t w = pack_bf16(s[b][i - 1], s[b][i]);
                    pw[2 * b + i / 8][i % 8 / 2] = w;
                    // the output is divided by the sum of the rounded weights, which is what V is
                    // multiplied by; lse is of the unrounded ones
                    st.l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w),
                                                           __builtin_bit_cast(bf16x2_t, 0x3f803f80u), st.l, false);
                }
            } else {
                st.l += p;
            }
        }
    auto add = [&](int x, VF a) {
        if constexpr (BF)
            o[x % ND] = mfma32(a, __builtin_bit_cast(bf16x8_t, pw[x / ND]), o[x % ND]);
        else
            o[x % ND] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, s[x / ND / 16][x / ND % 16], o[x % ND], 0, 0, 0);
    };
    if constexpr (MODE == kOdd) {
        // The product with what is finite, then, key by key, what is not: in a row that sees the
        // key, any positive weight of an infinity is that infinity, and NaN is NaN.
#pragma unroll
        for (int x = 0; x < NV; ++x) add(x, only_finite(v_at(x)));
#pragma unroll 1
        for (int key = 0; key < N; ++key) {
            const char* at = sv + key / C::ROWS * C::VG + key % C::ROWS * C::ROWB + 4 * half * C::ES;
            const bool sees = key < lim;
#pragma unroll
            for (int db = 0; db < ND; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = load1_f32(reinterpret_cast<const T*>(at) + 32 * db + 8 * (i / 4) + i % 4);
                    o[db][i] += sees && !is_finite(x) ? x : 0.f;
                }
        }
    } else {
#pragma unroll
        for (int x = 2; x < PF; ++x) vf[x] = v_at(x);
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            add(x, vf[x % PF]);
            if (x + PF < NV) vf[x % PF] = v_at(x + PF);
        }
    }
}

template <typename T, int D, bool LSE, typename S>
__global__ void __launch_bounds__(64 * S::WAVES, S::PER_SIMD) prefill_kernel(AttnCall p)
{
    using C = Tile<T, D>;
    constexpr int N = C::N, UNIT = S::STEPS * N, M = S::ROWS, ND = D / 32, SPLIT = S::SPLIT;
    constexpr int ES = C::ES;
    // separate arrays: the compiler then knows that reading one need not wait for the loads that
    // are filling another
    __shared__ __align__(16) char s_k0[S::STEPS * C::GROUPS * C::KG], s_k1[S::STEPS * C::GROUPS * C::KG];
    __shared__ __align__(16) char s_v0[S::STEPS * C::GROUPS * C::VG], s_v1[S::STEPS * C::GROUPS * C::VG];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5;
    const int rw = wave % (S::WAVES / SPLIT), turn = wave / (S::WAVES / SPLIT);  // 32 rows, steps
    Work w;
    const uint32_t block = block_index();
    if (block >= (uint32_t)p.units * (uint32_t)(S::RANGES ? p.ranges : 1)) return;  // past the grid's end
    const int unit = S::RANGES ? block % (uint32_t)p.units : block, rg = S::RANGES ? block / (uint32_t)p.units : 0;
    if (!find_work<M>(p, unit / p.d.h_kv, unit % p.d.h_kv, lane, &w)) return;

    const int64_t ks = ES * p.d.k_token, vs = ES * p.d.v_token;
    const char* kb = static_cast<const char*>(p.k) + w.k0 * ks + ES * w.head * p.d.k_head;
    const char* vb = static_cast<const char*>(p.v) + w.k0 * vs + ES * w.head * p.d.v_head;
    constexpr int LPR = 64 / C::ROWS;  // lanes that load a row
    const int koff = (int)(lane / LPR * ks) + lane % LPR * 16, voff = (int)(lane / LPR * vs) + lane % LPR * 16;
    // K: row lane & 31 of a product is place (lane & 31) / GROUPS of group (lane & 31) % GROUPS. V,
    // bf16: the reads of 16 lanes cover groups 4 half + 0..3, 16 elements of each, the next 16
    // lanes the next 16; fp32: a half reads 32 elements of one group, 4 half on
    const int klane = lane % C::GROUPS * C::KG + lane % 32 / C::GROUPS * C::ROWB + half * 16;
    const int vlane = ES == 2 ? (4 * half + ((lane >> 2) & 3)) * C::VG + ((lane >> 4) & 1) * 32 + (lane & 3) * 8
                              : 4 * half * C::VG + lane % 32 * 4;
    int valid = w.len_k;
    auto fetch = [&](int row, char* sk, char* sv) __attribute__((always_inline)) {
        stage<T, D, S, C::KG>(kb, row, valid, ks, sk, wave, koff);
        stage<T, D, S, C::VG>(vb, row, valid, vs, sv, wave, voff);
    };

    // keys that a row sees: the workgroup's last row and all of its rows; the last of the wave's
    // and all of the wave's; this lane's
    auto limit_of = [&](int row) {
        return key_limit(w, (int)((uint32_t)(row < w.rows ? row : w.rows - 1) / (uint32_t)w.g), p.d.causal);
    };
    const int wfirst = w.row0 + 32 * rw;
    int keys = limit_of(w.row0 + M - 1), all = limit_of(w.row0);
    // With ranges: from here on a key's number is its distance from `begin`, the range's first.
    int begin = 0;
    bool whole = true;
    if constexpr (S::RANGES) {
        const int per = range_keys(keys, p.ranges, UNIT);
        begin = rg * per;
        if (rg > 0 && begin >= keys) return;  // the join does not read this range
        whole = keys <= per;
        keys = keys - begin < per ? keys - begin : per;
        all = all - begin < keys ? all - begin : keys;
        valid -= begin;
        kb += begin * ks;
        vb += begin * vs;
    }
    if (keys > 0) fetch(0, s_k0, s_v0);
    const int wkeys = (wfirst < w.rows ? limit_of(wfirst + 31) : 0) - begin, wall = limit_of(wfirst) - begin;

    // this lane's query: row r of the sequence's packed rows
    const int r = wfirst + (lane & 31), rc = r < w.rows ? r : w.rows - 1, pos = (int)((uint32_t)rc / (uint32_t)w.g);
    const int limit = key_limit(w, pos, p.d.causal) - begin;
    const char* qp = static_cast<const char*>(p.q) +
                     ES * ((w.q0 + pos) * p.d.q_token + (w.head * w.g + (rc - pos * w.g)) * p.d.q_head) + 16 * half;
    // A negative scale becomes a positive one of the negated query: the maximum of the raw scores
    // is then that of the scaled ones. Zero becomes the smallest positive number, which takes any
    // finite score to less than 2^-20 and leaves a masked score, -infinity, as it is.
    const uint32_t flip = p.d.scale < 0.f ? (ES == 2 ? 0x80008000u : 0x80000000u) : 0u;
    const float c = fmaxf(fabsf(p.d.scale) * kLog2e, 0x1p-149f);
    u32x4_t q[D / (2 * C::PER)];  // piece kk: elements 2 PER kk + PER half ..
#pragma unroll
    for (int kk = 0; kk < D / (2 * C::PER); ++kk) q[kk] = *reinterpret_cast<const u32x4_t*>(qp + 32 * kk) ^ flip;

    f32x16_t o[ND];
    Stats st;
    bool odd = false;
    auto step = [&](auto mode, const char* sk, const char* sv, int j0) __attribute__((always_inline)) {
        constexpr int MODE = decltype(mode)::value;
        if (MODE != kPlain && j0 >= wkeys) return;  // nothing there for this wave's rows
        attn_step<T, D, LSE, MODE>(sk, sv, klane, vlane, q, o, st, c, j0 + N > wall, limit - j0, lane, odd);
    };
    auto use = [&](auto mode, const char* sk, const char* sv, int j0) __attribute__((always_inline)) {
        if constexpr (SPLIT == 2) {
            step(mode, sk + turn * C::GROUPS * C::KG, sv + turn * C::GROUPS * C::VG, j0 + turn * N);
        } else {
#pragma unroll 1
            for (int t = 0; t < S::STEPS; ++t) step(mode, sk + t * C::GROUPS * C::KG, sv + t * C::GROUPS * C::VG, j0 + t * N);
        }
    };
    // Two buffers: while the steps in one are used those in the other arrive. The barrier before
    // a use has every wave's loads of it landed, and every wave past the buffer refilled next.
    auto run = [&](auto mode, int j0) __attribute__((always_inline)) {
        for (; j0 < keys; j0 += 2 * UNIT) {
            staged_barrier();
            if (j0 + UNIT < keys) fetch(j0 + UNIT, s_k1, s_v1);
            use(mode, s_k0, s_v0, j0);
            if (j0 + UNIT >= keys) break;
            staged_barrier();
            if (j0 + 2 * UNIT < keys) fetch(j0 + 2 * UNIT, s_k0, s_v0);
            use(mode, s_k1, s_v1, j0 + UNIT);
        }
    };
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[db][i] = 0.f;
        st = Stats{-INFINITY, 0.f, 0.f};
    };
    clear();
    // keys that all rows see; here the next keys to fetch always exist
    const int kahead = (int)(S::WAVES * C::ROWS * ks), vahead = (int)(S::WAVES * C::ROWS * vs);
    const char* kw = kb + (UNIT + wave * C::ROWS) * ks;
    const char* vw = vb + (UNIT + wave * C::ROWS) * vs;
    auto fetch_whole = [&](char* sk, char* sv) __attribute__((always_inline)) {
        stage_whole<T, D, S, C::KG>(kw, kahead, sk, wave, koff);
        stage_whole<T, D, S, C::VG>(vw, vahead, sv, wave, voff);
        kw += UNIT * ks;
        vw += UNIT * vs;
    };
    int j0 = 0;
    for (; j0 + 3 * UNIT <= all; j0 += 2 * UNIT) {
        staged_barrier();
        fetch_whole(s_k1, s_v1);
        use(std::integral_constant<int, kPlain>{}, s_k0, s_v0, j0);
        staged_barrier();
        fetch_whole(s_k0, s_v0);
        use(std::integral_constant<int, kPlain>{}, s_k1, s_v1, j0 + UNIT);
    }
    run(std::integral_constant<int, kMasks>{}, j0);
    if (__syncthreads_or(odd)) {  // rare: the whole tile again
        clear();
        fetch(0, s_k0, s_v0);
        run(std::integral_constant<int, kOdd>{}, 0);
        __syncthreads();  // the buffers are written to below
    }

    if constexpr (SPLIT == 2) {
        // O of the second steps' waves through LDS: D / 2 registers of 64 lanes a wave, in the
        // buffers of K and V, a row group in each
        static_assert(D / 2 * 256 <= S::STEPS * C::GROUPS * C::KG, "a wave's O fits a buffer");
        float* so = reinterpret_cast<float*>(rw == 0 ? s_k0 : rw == 1 ? s_k1 : rw == 2 ? s_v0 : s_v1);
        __syncthreads();
        if (turn == 1) {
#pragma unroll
            for (int db = 0; db < ND; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) so[(16 * db + i) * 64 + lane] = o[db][i];
        }
        __syncthreads();
        __shared__ float s_st[4][3][64];
        if (turn == 1) {
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
    if constexpr (S::RANGES) {
        if (!whole) {  // this range's sums, for the join
            const float l = other_half_sum(st.l), e = ES == 2 && LSE ? other_half_sum(st.exact) : l;
            const int64_t at = ((int64_t)unit * p.ranges + rg) * M + 32 * rw + (lane & 31);
            if (r < w.rows) {
                float* to = p.part_o + at * D + 4 * half;
#pragma unroll
                for (int db = 0; db < ND; ++db)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<f32x4_t*>(to + 32 * db + 8 * i) =
                            f32x4_t{o[db][4 * i], o[db][4 * i + 1], o[db][4 * i + 2], o[db][4 * i + 3]};
                if (half == 0) p.part_ml[at] = make_float4(st.m * c, l, e, 0.f);
            }
            return;
        }
    }
    // All waves have met since the last use of K and V: each has a part of the buffers to itself (with
    // SPLIT 2 in the one where it read the other half's O).
    constexpr int PART = 32 * ((C::ROWB < 256 ? C::ROWB : 256) + 16), PER_BUFFER = (M / 32 + 3) / 4;
    static_assert(PER_BUFFER * PART <= S::STEPS * C::GROUPS * C::KG, "the waves' parts fit the buffers");
    const int buffer = rw / PER_BUFFER;
    char* part = buffer == 0 ? s_k0 : buffer == 1 ? s_k1 : buffer == 2 ? s_v0 : s_v1;
    st.m *= c;
    write_rows<T, D>(p, w, wfirst, lane, o, st, part + rw % PER_BUFFER * PART);
}

constexpr int kMaxRanges = 64;

// Joins the ranges of a tile: D / 4 lanes hold a row, first one range each for the weights
// exp2(m - max m), then four elements each of the weighted sum, in the order of the ranges.
template <typename T, int D, typename S>
__global__ void __launch_bounds__(256) join_kernel(AttnCall p)
{
    constexpr int M = S::ROWS, LANES = D / 4, ROWS = 256 / LANES;
    __shared__ float s_w[ROWS][kMaxRanges];
    const int unit = blockIdx.x / (M / ROWS), mine = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int row = blockIdx.x % (M / ROWS) * ROWS + mine;
    Work w;
    if (!find_work<M>(p, unit / p.d.h_kv, unit % p.d.h_kv, threadIdx.x & 63, &w)) return;
    const int last = w.row0 + M - 1, keys = key_limit(w, (last < w.rows ? last : w.rows - 1) / w.g, p.d.causal);
    const int per = range_keys(keys, p.ranges, S::STEPS * Tile<T, D>::N), r = w.row0 + row;
    if (keys <= per || r - mine >= w.rows) return;
    const int used = (keys + per - 1) / per;
    const int64_t at = (int64_t)unit * p.ranges * M + row;
    float top = -INFINITY, l = 0.f, e = 0.f;
    if (r < w.rows) {
        constexpr int EACH = kMaxRanges / LANES;
        float4 ml[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int x = i * LANES + lane;
            ml[i] = x < used ? p.part_ml[at + x * M] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
            top = fmaxf(top, ml[i].x);
        }
#pragma unroll
        for (int off = LANES / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const float f = ml[i].x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[i].x - top);
            s_w[mine][i * LANES + lane] = f;
            l += ml[i].y * f;
            e += ml[i].z * f;
        }
#pragma unroll
        for (int off = LANES / 2; off >= 1; off >>= 1) {
            l += __shfl_xor(l, off, 64);
            e += __shfl_xor(e, off, 64);
        }
    }
    __syncthreads();
    if (r >= w.rows) return;
    const float* from = p.part_o + at * D + lane * 4;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 16
    for (int x = 0; x < used; ++x) o += *reinterpret_cast<const f32x4_t*>(from + (int64_t)x * M * D) * s_w[mine][x];
    o *= l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    const int pos = r / w.g;
    const int64_t to = (w.q0 + pos) * p.d.h_q + w.head * w.g + (r - pos * w.g);
    T* out = static_cast<T*>(p.out) + to * D + lane * 4;
    if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2_t*>(out) = u32x2_t{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    else *reinterpret_cast<f32x4_t*>(out) = o;
    if (p.lse && lane == 0) p.lse[to] = e > 0.f ? (top + __builtin_amdgcn_logf(e)) * kLn2 : (e == e ? -INFINITY : e);
}

int64_t units_of(const gdn_attn_dims& d, int rows)
{
    return (d.total_q * (d.h_q / d.h_kv) / rows + d.n) * d.h_kv;
}

int range_rows(const gdn_attn_dims& d)  // of the shape with ranges
{
    return d.dtype == GDN_F32 && d.d == 256 ? Lone::ROWS : Few::ROWS;
}

// Ranges that every tile's keys are divided into: what makes the estimate of the call's time least.
// 256 workgroups run at a time; each costs its keys and about 128 more, and a join about 256 (a key
// takes some 20 ns, d = 256 bf16). Undivided, a workgroup takes 128 rows. Measured (us of a call,
// undivided / divided): d = 256, 16/2 heads, 16 tokens after 32752 684 / 56, 128 after 32640 686 / 104,
// 512 after 8192 195 / 108; d = 128, 32/8 heads, 8 sequences of 8 tokens after 8192 134 / 85.
int ranges_of(const gdn_attn_dims& d)
{
    if (d.n == 0 || d.total_q == 0) return 1;
    const int rows = range_rows(d);
    const int64_t all = d.total_q * (d.h_q / d.h_kv), keys = d.total_k / d.n;
    auto units = [&](int m) { return ((all + m - 1) / m > d.n ? (all + m - 1) / m : d.n) * d.h_kv; };
    const int64_t u = units(rows), most = units_of(d, rows);
    int best = 1;
    int64_t least = (units(128) + 255) / 256 * (keys + 128);
    for (int64_t r = 2; r <= kMaxRanges && most * r <= 1024 && keys >= 256 * r; ++r) {
        const int64_t cost = (u * r + 255) / 256 * (keys / r + 128) + 256 + 4 * r;
        if (cost < least) {
            least = cost;
            best = (int)r;
        }
    }
    return best;
}

template <typename T, int D, bool LSE, typename S>
hipError_t launch_kernel(const AttnCall& c, int ranges = 1)
{
    const int64_t units = units_of(c.d, S::ROWS);
    AttnCall a = c;
    a.units = (int)units;
    a.ranges = ranges;
    a.part_o = static_cast<float*>(c.ws);
    a.part_ml = reinterpret_cast<float4*>(a.part_o + units * ranges * S::ROWS * D);
    hipLaunchKernelGGL((prefill_kernel<T, D, LSE, S>), grid_of(units * ranges), dim3(64 * S::WAVES), 0, c.stream, a);
    const hipError_t e = hipGetLastError();
    if constexpr (S::RANGES)
        if (e == hipSuccess && ranges > 1) {
            hipLaunchKernelGGL((join_kernel<T, D, S>), dim3((unsigned)(units * (S::ROWS * D / 1024))), dim3(256), 0,
                               c.stream, a);
            return hipGetLastError();
        }
    return e;
}

template <typename T, int D, bool LSE>
hipError_t launch_shape(const AttnCall& c)
{
    const int ranges = ranges_of(c.d);
    if constexpr (Tile<T, D>::ROWS == 1) {
        return launch_kernel<T, D, LSE, Lone>(c, ranges);
    } else {
        if (ranges > 1) return launch_kernel<T, D, LSE, Few>(c, ranges);
        // Measured (us, bf16, Wide / Split / Twin; tiles of 256 rows). Few tiles of many keys, where
        // one workgroup's time is the call's: d = 256, 16/2 heads, 2048-token prompt (128 tiles)
        // 98 / 63 / 68, 4096 (256) 190 / 150 / 163, 4112 (257) 193 / 161 / 163, 4352 206 / 180 / 177,
        // 5120 253 / 241 / 224, 6144 (384) 321 / 323 / 300, 7168 (448) 390 / 414 / 413; Split / Twin,
        // d = 128, 16/16 heads, 4096 (256) 82 / 94, 4112 93 / 95, 5120 133 / 126; d = 64, 32/8 heads,
        // 2048 (256) 35 / 32, 2064 42 / 34. A 257th tile makes the busiest CU's list longer in every
        // shape. (Wide would also save 6% from 448 tiles of fewer keys.)
        // Few keys: 32 prompts of 64, 32/8 heads (256) 21 / 30 / 18; many tiles: 16 of 1024 (2048)
        // 205 / 270 / 193, 8192 (1024) 513 / 542 / 504. Long rows and many keys, where the traffic
        // of staging counts: d = 256, 8192 (512) 472 / 508 / 512, 16 of 1024 197 / 270 / 191.
        const int64_t tiles = c.d.total_q * c.d.h_q / 256, keys = c.d.total_k / c.d.n;
        // fp32, Twin / Few: three prompts of up to 200, d = 64 22.3 / 17.9, 1024 tokens, 16/2 heads, d = 128
        // (64) 131 / 79. bf16 gains 5% at 512 tokens and loses as much at eight of 64.
        if (sizeof(T) == 4 && tiles <= 64) return launch_kernel<T, D, LSE, Few>(c);
        if (tiles <= 256 && keys >= 1024) return launch_kernel<T, D, LSE, Split>(c);
        if constexpr (Tile<T, D>::ROWS == 2 && sizeof(T) == 2)
            if (keys >= 8192) return launch_kernel<T, D, LSE, Wide>(c);
        return launch_kernel<T, D, LSE, Twin>(c);
    }
}

template <int D>
hipError_t launch_d(const AttnCall& c)
{
    if (c.d.dtype == GDN_F32) return launch_shape<float, D, false>(c);
    return c.lse ? launch_shape<uint16_t, D, true>(c) : launch_shape<uint16_t, D, false>(c);
}

}  // namespace

size_t attn_prefill_workspace(const gdn_attn_dims& d)
{
    const int ranges = ranges_of(d), rows = range_rows(d);
    return ranges == 1 ? 0 : (size_t)(units_of(d, rows) * ranges * rows) * (d.d * sizeof(float) + sizeof(float4));
}

int attn_prefill_rows(int32_t, int32_t)
{
    return 64;  // the smallest of the kernels' tiles
}

hipError_t launch_attn_prefill(const AttnCall& c)
{
    switch (c.d.d) {
        case 64: return launch_d<64>(c);
        case 128: return launch_d<128>(c);
        case 256: return launch_d<256>(c);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
