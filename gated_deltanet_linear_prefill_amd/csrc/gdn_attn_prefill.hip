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
// Masked keys get weight exactly 0. A matrix product would still turn 0 x NaN into NaN, so
// rows past the end of a sequence are read as zeros, and in steps that hold masked keys a V that
// is not finite is left out of the product and added only to the rows that see its key.
#include <type_traits>
#include <utility>

#include "gdn_attn_internal.hpp"

namespace gdn {
namespace {

constexpr int kWaves = 4;      // of the fp32 kernel
constexpr int kBf16Waves = 8;  // of the bf16 kernel
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T, int D>
struct Tile;

// bf16: 32 query rows per wave. A staged row of D elements; ROWS of them fill the 1 KiB that a
// wave's load to LDS writes, and 16 such groups, each padded, are a step of N keys. The key of
// group x, place y is ROWS x + y: the keys of group x lie next to each other in memory, and a
// wave reads place y of all 16 groups together, in banks that the padding keeps apart (16 bytes
// a group for K, read 16 bytes a lane; 64 for V, read in 64-byte pieces of four groups). A
// reading lane has one address; everything else is an instruction offset.
template <int D>
struct Tile<uint16_t, D> {
    static constexpr int ROWS = 512 / D, N = 16 * ROWS, BLOCKS = N / 32, WAVES = kBf16Waves;
    static constexpr int ROWB = 2 * D, KG = 1024 + 16, VG = 1024 + 64;  // bytes: row, padded groups
};

// fp32: 32 query rows per wave, 32 keys per step
template <int D>
struct Tile<float, D> {
    static constexpr int N = 32, M = 32 * kWaves;
};

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

// fp32 rows: the 16-byte chunk at which logical chunk c is kept, so that the rows that a read
// touches together lie in different banks. The loads to LDS apply it by choosing which chunk
// each lane fetches.
template <int CHUNKS>
__device__ __forceinline__ int swz(int row)
{
    return row & (CHUNKS < 16 ? CHUNKS - 1 : 15);
}

// Rows [row, row + N) of a strided fp32 [..][D] tensor into LDS, zeros from `valid` rows on.
// CHUNKS 16-byte chunks a row; swizzled.
template <int N, int CHUNKS>
__device__ __forceinline__ void stage_f32(const char* base, int64_t row, int64_t valid, int64_t stride,
                                          char* lds, int wave, int lane)
{
    const int64_t left = valid - row;
    const int64_t have = left < N ? left : N;
    const __amdgpu_buffer_rsrc_t r =
        make_rsrc(base + row * stride, have <= 0 ? 0 : (have - 1) * stride + CHUNKS * 16);
#pragma unroll
    for (int i = 0; i < N * CHUNKS / (64 * kWaves); ++i) {
        const int at = (i * kWaves + wave) * 64;  // first chunk of this wave's 1 KiB
        const int c = at + lane, rr = c / CHUNKS, cc = c % CHUNKS;
        load_to_lds(r, lds + at * 16, (int)(rr * stride) + (cc ^ swz<CHUNKS>(rr)) * 16);
    }
}

// Two steps' keys [row, row + 2 N) of a strided bf16 tensor into LDS, in padded groups of GROUP
// bytes; zeros from `valid` rows on. `off` is this lane's byte offset within a group's rows in
// memory.
template <int D, int GROUP>
__device__ __forceinline__ void stage(const char* base, int row, int valid, int64_t stride,
                                      char* lds, int wave, int off)
{
    using C = Tile<uint16_t, D>;
#pragma unroll
    for (int i = 0; i < 32 / C::WAVES; ++i) {
        const int x = i * C::WAVES + wave;
        const int first = row + x * C::ROWS;
        const int left = valid - first, have = left < C::ROWS ? left : C::ROWS;
        const __amdgpu_buffer_rsrc_t r =
            make_rsrc(base + first * stride, have <= 0 ? 0 : (have - 1) * stride + C::ROWB);
        load_to_lds(r, lds + x * GROUP, off);
    }
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

// Whether any lane holds a NaN or infinity among its eight bf16 values: adding one to an
// all-ones exponent carries into the sign's place.
__device__ __forceinline__ bool any_not_finite(bf16x8_t x)
{
    const u32x4_t u = __builtin_bit_cast(u32x4_t, x);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c |= (u[i] & 0x7f807f80u) + 0x00800080u;
    return __any((c & 0x80008000u) != 0);
}

// Softmax state of a wave's 32 rows: each lane's own query. Scores are in units of log 2.
struct Stats {
    float m;      // reference maximum (-inf: nothing seen)
    float l;      // sum of the weights of this lane's keys, as they multiply V
    float exact;  // the same before rounding, if lse is wanted
};

// New weights from scores: p = exp2(s - m), with O and l rescaled if the maximum rose.
template <int R, int ND>
__device__ __forceinline__ void softmax_step(float* s, f32x16_t (&o)[ND], Stats* st)
{
    float mx = s[0];
#pragma unroll
    for (int i = 1; i < R; ++i) mx = fmaxf(mx, s[i]);
    mx = other_half_max(mx);
    const float m_new = fmaxf(st->m, mx);
    if (__any(m_new > st->m)) {
        const float a = m_new == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(st->m - m_new);
        st->m = m_new;
        st->l *= a;
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[db][i] *= a;
    }
    const float ref = st->m == -INFINITY ? 0.f : st->m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        s[i] = __builtin_amdgcn_exp2f(s[i] - ref);
        sum += s[i];
    }
    st->l += sum;
}

// Writes a row's output: this lane's 4-element pieces of O^T, divided by the sum.
template <typename T, int D>
__device__ __forceinline__ void write_row(const AttnCall& p, const Work& w, int r, int lane,
                                          const f32x16_t* o, const Stats& st)
{
    const float l = other_half_sum(st.l), e = other_half_sum(st.exact);
    if (r >= w.rows) return;
    const int pos = (int)((uint32_t)r / (uint32_t)w.g);
    const int64_t row = (w.q0 + pos) * p.d.h_q + w.head * w.g + (r - pos * w.g);
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    T* out = static_cast<T*>(p.out) + row * D + 4 * (lane >> 5);
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = o[db][4 * i] * inv, b = o[db][4 * i + 1] * inv;
            const float c = o[db][4 * i + 2] * inv, f = o[db][4 * i + 3] * inv;
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<u32x2_t*>(out + 32 * db + 8 * i) = u32x2_t{pack_bf16(a, b), pack_bf16(c, f)};
            else
                *reinterpret_cast<f32x4_t*>(out + 32 * db + 8 * i) = f32x4_t{a, b, c, f};
        }
    if (p.lse && lane < 32) p.lse[row] = e > 0.f ? (st.m + __builtin_amdgcn_logf(e)) * kLn2 : (e == e ? -INFINITY : e);
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

// kPlain: every row sees every key. kMasks: where `masked`, some rows may not see some keys, and
// `odd` is set if V holds a NaN or an infinity there. kOdd: for tiles where that was found.
enum { kPlain, kMasks, kOdd };

// One step of a wave's 32 rows over N staged keys at sk, sv (klane, vlane: this lane's offsets).
// This lane's row sees the keys below lim (which may be negative, or above N).
template <int D, bool LSE, int MODE>
__device__ __forceinline__ void bf16_step(const char* sk, const char* sv, int klane, int vlane,
                                          const bf16x8_t (&q)[D / 16], f32x16_t (&o)[D / 32], Stats& st,
                                          float c, bool masked, int lim, int lane, bool& odd)
{
    using C = Tile<uint16_t, D>;
    constexpr int N = C::N, NB = C::BLOCKS, ND = D / 32, KK = D / 16, PF = 4;
    const int half = lane >> 5;
    f32x16_t s[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
    auto k_at = [&](int x) {  // product x: block x % NB, elements 16 (x / NB) ..
        return *reinterpret_cast<const bf16x8_t*>(sk + klane + x % NB * 2 * C::ROWB + x / NB * 32);
    };
    bf16x8_t kf[PF];
#pragma unroll
    for (int x = 0; x < PF; ++x) kf[x] = k_at(x);
#pragma unroll
    for (int x = 0; x < KK * NB; ++x) {
        s[x % NB] = mfma32(kf[x % PF], q[x / NB], s[x % NB]);
        if (x + PF < KK * NB) kf[x % PF] = k_at(x + PF);
    }

    // V^T operand x: rows 32 (x % ND) .. of V^T, keys at place x / ND of every group
    auto v_at = [&](int x) {
        const char* at = sv + vlane + x / ND * C::ROWB + x % ND * 64;
        return __builtin_shufflevector(read_tr(at), read_tr(at + 8 * C::VG), 0, 1, 2, 3, 4, 5, 6, 7);
    };
    if (MODE != kPlain && masked) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                // row m of the product is place 2 b + m / 16 of group m % 16
                const int m = 8 * (i / 4) + i % 4;
                s[b][i] = C::ROWS * (m % 16 + 4 * half) + 2 * b + m / 16 < lim ? s[b][i] : -INFINITY;
            }
        if (MODE == kMasks)
#pragma unroll 1
            for (int x = 0; x < 16; ++x)
                odd |= any_not_finite(*reinterpret_cast<const bf16x8_t*>(sv + x * C::VG + lane * 16));
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
        const float a = !rise ? 1.f : st.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((st.m - mx) * c);
        st.m = rise ? mx : st.m;
        st.l *= a;
        if (LSE) st.exact *= a;
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[db][i] *= a;
    }
    const float ref = st.m == -INFINITY ? 0.f : st.m * c;
    bf16x8_t vf[PF];
#pragma unroll
    for (int x = 0; x < 2; ++x) vf[x] = v_at(x);
    u32x4_t pw[2 * NB];  // the weights as B operands: place y of every group
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], c, -ref));
            s[b][i] = p;
            if (LSE) st.exact += p;
            if (i & 1) {
                const uint32_t w = pack_bf16(s[b][i - 1], s[b][i]);
                pw[2 * b + i / 8][i % 8 / 2] = w;
                // the output is divided by the sum of the rounded weights, which is what V is
                // multiplied by; lse is of the unrounded ones
                st.l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w),
                                                       __builtin_bit_cast(bf16x2_t, 0x3f803f80u), st.l, false);
            }
        }
    if constexpr (MODE == kOdd) {
        // The product with what is finite, then, key by key, what is not: in a row that sees the
        // key, any positive weight of an infinity is that infinity, and NaN is NaN.
#pragma unroll
        for (int x = 0; x < 2 * NB * ND; ++x)
            o[x % ND] = mfma32(only_finite(v_at(x)), __builtin_bit_cast(bf16x8_t, pw[x / ND]), o[x % ND]);
#pragma unroll 1
        for (int key = 0; key < N; ++key) {
            const char* at = sv + key / C::ROWS * C::VG + key % C::ROWS * C::ROWB + 8 * half;
            const bool sees = key < lim;
#pragma unroll
            for (int db = 0; db < ND; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(at + 64 * db + 16 * (i / 4) + 2 * (i % 4)));
                    o[db][i] += sees && !(fabsf(x) <= 3.4028234e38f) ? x : 0.f;
                }
        }
    } else {
#pragma unroll
        for (int x = 2; x < PF; ++x) vf[x] = v_at(x);
#pragma unroll
        for (int x = 0; x < 2 * NB * ND; ++x) {
            o[x % ND] = mfma32(vf[x % PF], __builtin_bit_cast(bf16x8_t, pw[x / ND]), o[x % ND]);
            if (x + PF < 2 * NB * ND) vf[x % PF] = v_at(x + PF);
        }
    }
}

// Eight waves. Keys are staged two steps at a time. SPLIT 1: the waves have 32 rows each, 256 in
// all, and take both steps; a staged key serves 256 rows. SPLIT 2: 128 rows, four waves of them
// take the first steps and four the second, and are joined at the end: half the rows and half
// the time per workgroup, for calls that have too few tiles to keep all CUs busy evenly.
template <int D, bool LSE, int SPLIT>
__global__ void __launch_bounds__(64 * kBf16Waves, 2) prefill_bf16_kernel(AttnCall p)
{
    using C = Tile<uint16_t, D>;
    constexpr int N = C::N, M = 32 * C::WAVES / SPLIT, ND = D / 32;
    // separate arrays: the compiler then knows that reading one need not wait for the loads that
    // are filling another
    __shared__ __align__(16) char s_k0[32 * C::KG], s_k1[32 * C::KG];
    __shared__ __align__(16) char s_v0[32 * C::VG], s_v1[32 * C::VG];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5;
    const int rw = wave % (C::WAVES / SPLIT), turn = wave / (C::WAVES / SPLIT);  // 32 rows, steps
    Work w;
    if (!find_work<M>(p, blockIdx.x / p.d.h_kv, blockIdx.x % p.d.h_kv, lane, &w)) return;

    const int64_t ks = 2 * p.d.k_token, vs = 2 * p.d.v_token;
    const char* kb = static_cast<const char*>(p.k) + w.k0 * ks + 2 * w.head * p.d.k_head;
    const char* vb = static_cast<const char*>(p.v) + w.k0 * vs + 2 * w.head * p.d.v_head;
    constexpr int LPR = 64 / C::ROWS;  // lanes that load a row
    const int koff = (int)(lane / LPR * ks) + lane % LPR * 16, voff = (int)(lane / LPR * vs) + lane % LPR * 16;
    // K: row lane & 31 of a product is place (lane & 31) / 16 of group lane & 15; V: the reads of
    // 16 lanes cover groups 4 half + 0..3, 16 elements of each, the next 16 lanes the next 16
    const int klane = (lane & 15) * C::KG + ((lane >> 4) & 1) * C::ROWB + half * 16;
    const int vlane = (4 * half + ((lane >> 2) & 3)) * C::VG + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    auto fetch = [&](int row, char* sk, char* sv) __attribute__((always_inline)) {
        stage<D, C::KG>(kb, row, w.len_k, ks, sk, wave, koff);
        stage<D, C::VG>(vb, row, w.len_k, vs, sv, wave, voff);
    };

    // keys that a row sees: the workgroup's last row and all of its rows; the last of the wave's
    // and all of the wave's; this lane's
    auto limit_of = [&](int row) {
        return key_limit(w, (int)((uint32_t)(row < w.rows ? row : w.rows - 1) / (uint32_t)w.g), p.d.causal);
    };
    const int wfirst = w.row0 + 32 * rw;
    const int keys = limit_of(w.row0 + M - 1), all = limit_of(w.row0);
    if (keys > 0) fetch(0, s_k0, s_v0);
    const int wkeys = wfirst < w.rows ? limit_of(wfirst + 31) : 0, wall = limit_of(wfirst);

    // this lane's query: row r of the sequence's packed rows
    const int r = wfirst + (lane & 31), rc = r < w.rows ? r : w.rows - 1, pos = (int)((uint32_t)rc / (uint32_t)w.g);
    const int limit = key_limit(w, pos, p.d.causal);
    const uint16_t* qp = static_cast<const uint16_t*>(p.q) + (w.q0 + pos) * p.d.q_token +
                         (w.head * w.g + (rc - pos * w.g)) * p.d.q_head + 8 * half;
    // A negative scale becomes a positive one of the negated query: the maximum of the raw scores
    // is then that of the scaled ones. Zero becomes so small a one that every weight is 1, and
    // a masked score, -infinity, stays so.
    const uint32_t flip = p.d.scale < 0.f ? 0x80008000u : 0u;
    const float c = fmaxf(fabsf(p.d.scale) * kLog2e, 1e-37f);
    bf16x8_t q[D / 16];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        q[kk] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(qp + 16 * kk) ^ flip);

    f32x16_t o[ND];
    Stats st;
    bool odd = false;
    auto step = [&](auto mode, const char* sk, const char* sv, int j0) __attribute__((always_inline)) {
        constexpr int MODE = decltype(mode)::value;
        if (MODE != kPlain && j0 >= wkeys) return;  // nothing there for this wave's rows
        bf16_step<D, LSE, MODE>(sk, sv, klane, vlane, q, o, st, c, j0 + N > wall, limit - j0, lane, odd);
    };
    auto pair = [&](auto mode, const char* sk, const char* sv, int j0) __attribute__((always_inline)) {
        if constexpr (SPLIT == 1) {
#pragma unroll 1
            for (int t = 0; t < 2; ++t) step(mode, sk + t * 16 * C::KG, sv + t * 16 * C::VG, j0 + t * N);
        } else {
            step(mode, sk + turn * 16 * C::KG, sv + turn * 16 * C::VG, j0 + turn * N);
        }
    };
    // Two buffers: while a pair of steps is used the next one arrives. The barrier before a pair
    // has every wave's loads of it done, and every wave past the buffer that is refilled next.
    auto run = [&](auto mode, int j0) __attribute__((always_inline)) {
        for (; j0 < keys; j0 += 4 * N) {
            __syncthreads();
            if (j0 + 2 * N < keys) fetch(j0 + 2 * N, s_k1, s_v1);
            pair(mode, s_k0, s_v0, j0);
            if (j0 + 2 * N >= keys) break;
            __syncthreads();
            if (j0 + 4 * N < keys) fetch(j0 + 4 * N, s_k0, s_v0);
            pair(mode, s_k1, s_v1, j0 + 2 * N);
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
    int j0 = 0;
    for (; j0 + 4 * N <= all; j0 += 4 * N) {  // keys that all rows see
        __syncthreads();
        fetch(j0 + 2 * N, s_k1, s_v1);
        pair(std::integral_constant<int, kPlain>{}, s_k0, s_v0, j0);
        __syncthreads();
        if (j0 + 4 * N < keys) fetch(j0 + 4 * N, s_k0, s_v0);
        pair(std::integral_constant<int, kPlain>{}, s_k1, s_v1, j0 + 2 * N);
    }
    run(std::integral_constant<int, kMasks>{}, j0);
    if (__syncthreads_or(odd)) {  // rare: the whole tile again
        clear();
        fetch(0, s_k0, s_v0);
        run(std::integral_constant<int, kOdd>{}, 0);
    }

    if constexpr (SPLIT == 2) {
        // O of the second steps' waves through LDS: D / 2 registers of 64 lanes a wave, in the
        // buffers of K and V, a row group in each
        static_assert(D / 2 * 256 <= 32 * C::KG, "a wave's O fits a buffer");
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
        const float a0 = st.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((st.m - mm) * c);
        const float a1 = m1 == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m1 - mm) * c);
        st.m = mm;
        st.l = a0 * st.l + a1 * s_st[rw][1][lane];
        st.exact = a0 * st.exact + a1 * s_st[rw][2][lane];
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[db][i] = a0 * o[db][i] + a1 * so[(16 * db + i) * 64 + lane];
    }
    st.m *= c;
    write_row<uint16_t, D>(p, w, r, lane, o, st);
}

// fp32 inputs: the same with the 32x32x2 fp32 MFMA, whose two k slots are the lane halves.
template <int D>
__global__ void __launch_bounds__(64 * kWaves) prefill_f32_kernel(AttnCall p)
{
    constexpr int N = Tile<float, D>::N, M = Tile<float, D>::M, CH = D / 4, ND = D / 32;
    __shared__ __align__(16) char s_k[N * D * 4];
    __shared__ __align__(16) char s_v[N * D * 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, l31 = lane & 31;
    Work w;
    if (!find_work<M>(p, blockIdx.x / p.d.h_kv, blockIdx.x % p.d.h_kv, lane, &w)) return;
    const int g = w.g;

    const int r = w.row0 + 32 * wave + l31, rc = r < w.rows ? r : w.rows - 1, pos = rc / g;
    const int limit = key_limit(w, pos, p.d.causal);
    const float* qp = static_cast<const float*>(p.q) + (w.q0 + pos) * p.d.q_token +
                      (w.head * g + (rc - pos * g)) * p.d.q_head + 4 * half;
    f32x4_t q[D / 8];  // slot e of step kk: element 8 kk + 4 half + e
#pragma unroll
    for (int kk = 0; kk < D / 8; ++kk) q[kk] = *reinterpret_cast<const f32x4_t*>(qp + 8 * kk);

    const int last = (w.row0 + M < w.rows ? w.row0 + M : w.rows) - 1;
    const int keys = key_limit(w, last / g, p.d.causal);
    const int wrow = w.row0 + 32 * wave;
    const int all = key_limit(w, (wrow < w.rows ? wrow : w.rows - 1) / g, p.d.causal);

    const char* kb = static_cast<const char*>(p.k) + 4 * (w.k0 * p.d.k_token + w.head * p.d.k_head);
    const char* vb = static_cast<const char*>(p.v) + 4 * (w.k0 * p.d.v_token + w.head * p.d.v_head);
    const float c = p.d.scale * kLog2e;

    f32x16_t o[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] = 0.f;
    Stats st = {-INFINITY, 0.f, 0.f};

    for (int j0 = 0; j0 < keys; j0 += N) {
        __syncthreads();
        stage_f32<N, CH>(kb, j0, w.len_k, 4 * p.d.k_token, s_k, wave, lane);
        stage_f32<N, CH>(vb, j0, w.len_k, 4 * p.d.v_token, s_v, wave, lane);
        __syncthreads();

        float s[16];
        f32x16_t acc;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 8; ++kk) {
            const int ch = (2 * kk + half) ^ swz<CH>(l31);
            const f32x4_t a = *reinterpret_cast<const f32x4_t*>(s_k + l31 * (D * 4) + ch * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], q[kk][e], acc, 0, 0, 0);
        }
        const bool masked = j0 + N > all;
        const int lim = limit - j0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int key = 8 * (i / 4) + 4 * half + i % 4;
            s[i] = !masked || key < lim ? acc[i] * c : -INFINITY;
        }
        softmax_step<16, ND>(s, o, &st);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = 8 * (i / 4) + 4 * half + i % 4;
#pragma unroll
            for (int db = 0; db < ND; ++db) {
                const int ch = 8 * db + (l31 >> 2);
                const float a = *reinterpret_cast<const float*>(s_v + row * (D * 4) +
                                                                (ch ^ swz<CH>(row)) * 16 + 4 * (l31 & 3));
                if (masked && __any(!(fabsf(a) <= 3.4028234e38f))) {
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {  // the two keys of the product, one at a time
                        const f32x16_t y = __builtin_amdgcn_mfma_f32_32x32x2f32(half == x ? a : 0.f, s[i], o[db], 0, 0, 0);
                        const bool sees = 8 * (i / 4) + 4 * x + i % 4 < lim;
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[db][e] = sees ? y[e] : o[db][e];
                    }
                } else {
                    o[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, s[i], o[db], 0, 0, 0);
                }
            }
        }
    }
    st.exact = st.l;
    write_row<float, D>(p, w, r, lane, o, st);
}

template <int D, bool LSE, int SPLIT>
hipError_t launch_bf16(const AttnCall& c)
{
    const int64_t tiles = c.d.total_q * (c.d.h_q / c.d.h_kv) / (32 * kBf16Waves / SPLIT) + c.d.n;
    hipLaunchKernelGGL((prefill_bf16_kernel<D, LSE, SPLIT>), dim3((unsigned)(tiles * c.d.h_kv)), dim3(64 * kBf16Waves),
                       0, c.stream, c);
    return hipGetLastError();
}

template <int D>
hipError_t launch_split(const AttnCall& c)
{
    // Whole tiles of 256 rows where they fill the CUs, evenly: under a causal mask a prompt's
    // last tiles take twice the average, so there should be two for every CU. Measured (us, whole
    // against split): d = 256, 16/2 heads, 4096-token prompt (256 tiles) 236 / 178, 8192 (512)
    // 526 / 622, 4096 tokens after 28672 (256 equal tiles) 1910 / 2112.
    const int64_t tiles = c.d.total_q * c.d.h_q / 256;
    const bool split = tiles < (c.d.causal && c.d.total_k < 2 * c.d.total_q ? 512 : 256);
    if (c.lse) return split ? launch_bf16<D, true, 2>(c) : launch_bf16<D, true, 1>(c);
    return split ? launch_bf16<D, false, 2>(c) : launch_bf16<D, false, 1>(c);
}

template <int D>
hipError_t launch_f32(const AttnCall& c)
{
    const int64_t tiles = c.d.total_q * (c.d.h_q / c.d.h_kv) / Tile<float, D>::M + c.d.n;
    hipLaunchKernelGGL((prefill_f32_kernel<D>), dim3((unsigned)(tiles * c.d.h_kv)), dim3(64 * kWaves), 0, c.stream, c);
    return hipGetLastError();
}

template <int D>
hipError_t launch_d(const AttnCall& c)
{
    return c.d.dtype == GDN_BF16 ? launch_split<D>(c) : launch_f32<D>(c);
}

}  // namespace

int attn_prefill_rows(int32_t, int32_t)
{
    return 128;  // the smallest of the kernels' tiles
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
