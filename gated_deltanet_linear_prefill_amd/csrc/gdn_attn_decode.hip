// gdn_attn_decode.hip -- attention of one new token per sequence over the paged cache.
//
// Bound by the bytes of the cache: every K and V row is read once per KV head, for all of its
// G = h_q / h_kv query heads (up to 16 at a time). One workgroup takes one (sequence, KV head)
// and one range of positions; its waves take 32-position (16 for long rows) steps of the range
// in turn, each with its own softmax state, and are joined in LDS. When the pairs alone would
// not fill the chip the positions are split over more workgroups (ranges), whose sums go to the
// workspace and are joined by a second kernel. (Joining by the workgroup that ends last was
// slower: 4096 positions 20.8 us against 14, since every workgroup then has to write its cache
// lines back before it counts itself.)
//
// Measured: 64 sequences of 17 to 8192, 32/8 heads, d = 128, bf16 (897 MB) 167 us + 7.6 us of join,
// 5.4 TB/s in the first kernel (a large copy: 5.2 to 5.7); 32 sequences of 4096, fp32, 5.6 TB/s
// in all; one sequence of 131072 fp8 positions, 16/2 heads, d = 256 (135 MB) 29 + 4.3 us, 4.6 TB/s
// (fp32 queries over an fp8 cache, 64 sequences of 8192, 32/8 heads, d = 128: 3.3 TB/s; four
// heads fill a quarter of the fp32 matrix instructions' columns, which run at 70% of their rate);
// 333 bf16 positions 11.4 us, what one CU takes to load a KV head's 341 KB (with eight waves a
// workgroup 11.1).
//
// Registers only (16x16 MFMA, one query head per column). S^T = K Q^T: lane l (c = l & 15,
// g = l >> 4) loads row c of a 16-key block in 16-byte pieces, which are the A operand as they
// are, and receives the scores of head c for keys 4 g + 0..3. O^T = V^T P^T: those scores are
// the B operand of keys 4 g + i as they are, if lane (c, g) also brings the V rows of keys
// 4 g + i: it loads a piece of each of them, and the piece's element j gives the A operand
// whose row c is that element. So no operand passes through LDS or between lanes; for bf16
// the two keys of an operand dword are paired by a byte permute.
#include "gdn_attn_internal.hpp"

namespace gdn {
namespace {

constexpr int kWaves = 4;
constexpr int kRange = 32 * kWaves;    // ranges are multiples of this: a step of every wave
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// How a call is divided: range positions per workgroup, ranges per sequence.
struct Plan {
    int64_t range, ranges;
    int head_tiles;
};

Plan make_plan(const gdn_kv_cache* c, int32_t h_q, int64_t max_len)
{
    const int64_t cap = c->max_pages * c->page_size;
    const int64_t len = max_len < cap ? max_len : cap;
    Plan p;
    p.head_tiles = (h_q / c->h_kv - 1) / 16 + 1;
    const int64_t units = c->n * c->h_kv * p.head_tiles;
    const int64_t steps = len > 0 ? (len + kRange - 1) / kRange : 1;
    // Measured (us of a C call, one sequence, d = 256, 16/2 heads, bf16, in 1 / 2 / 4 ranges): 256
    // positions 9.2 / 10.3, 512 14.2 / 12.9 / 10.4, 1024 23.4 / 18.0 / 13.0; fp8 512 10.1 / 10.9 / 9.6,
    // 1024 15.1 / 13.7 / 11.0; d = 128, 32/8 heads 512 8.4 / 9.7 / 8.5, 1024 12.7 / 11.9 / 9.7. Up to
    // four steps stay together, which spares the workspace and the second launch (333 positions
    // 11.4, 8.7 and 7.2; in ranges of one step 10.3, 9.5 and 8.4); longer ones are cut into ranges
    // of two steps or more. Ranges of one step would be faster for long rows: bf16 d = 256 from
    // 384 positions on (512: 10.4 us; 1024 in 8: 10.8), fp32 d = 256 from 256 on (512 29.5 / 15.4). A
    // single sequence of 131072 fp8 positions 33 in 256 ranges (one workgroup a CU), 39 in 1024. A
    // batch's lengths differ: 64 sequences of up to 8192, 8 KV heads, 198 in one range each,
    // 187 in ranges of 2048, 176 of 1024, where late workgroups fill the CUs that are done.
    const int64_t most = units * steps;
    int64_t want = most / 8 < 4096 ? most / 8 : 4096;
    if (want < 256 || c->n == 1) want = 256;
    int64_t ranges = units > 0 ? (want + units - 1) / units : 1;
    if (ranges > (steps + 1) / 2) ranges = (steps + 1) / 2;
    if (steps <= 4) ranges = 1;
    if (units > 0 && ranges > 0x7fffffff / units) ranges = 0x7fffffff / units;  // the grid
    if (ranges < 1) ranges = 1;
    const int64_t per = (steps + ranges - 1) / ranges;
    p.range = per * kRange;
    p.ranges = (steps + per - 1) / per;
    return p;
}

// Workspace of one call: O sums [unit][range][16][D] fp32, then (m, l, exact l, -) of each.
struct Partials {
    float* o;
    float4* ml;
};

template <typename T, bool FP8, int D>
struct Cfg {
    // bytes of a K/V element, elements of a V row per lane and load, loads
    static constexpr int ES = FP8 ? 1 : (int)sizeof(T);
    static constexpr int VL = D / 16;                          // elements of a V row per lane
    static constexpr int EPL = VL * ES > 16 ? 16 / ES : VL;    // ... per load
    static constexpr int U = VL / EPL;
    static constexpr int KL = D * ES / 64;                     // 16-byte loads of a K row per lane
    static constexpr int EPK = 16 / ES;                        // elements of each
    // 16-position blocks of a step: K and V rows of a step stay in registers
    static constexpr int NB = D * ES > 512 ? 1 : 2, STEP = 16 * NB;
    static constexpr bool QLDS = D * ES >= 512;                // Q in LDS, rows of QSTRIDE bytes
    static constexpr int QSTRIDE = D * (int)sizeof(T) + 16;
};

template <int BYTES>
struct Piece;
template <> struct Piece<4> { typedef uint32_t type; };
template <> struct Piece<8> { typedef u32x2_t type; };
template <> struct Piece<16> { typedef u32x4_t type; };

template <typename P>
__device__ __forceinline__ uint32_t word(const P& p, int i)
{
    if constexpr (sizeof(P) == 4) return p;
    else return p[i];
}

__device__ __forceinline__ float round_bf16(float x)
{
    return (float)(__bf16)x;
}

__device__ __forceinline__ uint32_t cvt_bf16_fp8(uint32_t w, bool hi)
{
    return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}

template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(64 * kWaves, 2)
decode_attn_kernel(AttnDecodeCall p, int64_t range, int ranges, int head_tiles, int page_shift,
                   Partials part)
{
    using C = Cfg<T, FP8, D>;
    using VP = typename Piece<C::EPL * C::ES>::type;
    constexpr bool BF = sizeof(T) == 2;
    __shared__ __align__(16) float s_o[kWaves][16][D + 4];
    static_assert(16 * C::QSTRIDE <= (int)sizeof(s_o), "Q fits");
    __shared__ float s_m[kWaves][16];
    __shared__ float2 s_l[kWaves][16];
    char* const s_q = reinterpret_cast<char*>(&s_o[0][0][0]);  // until the waves are joined

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    // ranges of one index lie together in the grid: which XCD a workgroup runs on (its index
    // modulo 8) then does not depend on its range, and late ranges, which few sequences have,
    // spread over all XCDs
    const int64_t units = p.c.n * p.c.h_kv * head_tiles;
    const int rg = (int)(block_index() / units);
    const int64_t unit = block_index() % units;
    if (rg >= ranges) return;  // past the grid's end
    const int ht = (int)(unit % head_tiles);
    const int kvh = (int)(unit / head_tiles % p.c.h_kv);
    const int64_t seq = unit / head_tiles / p.c.h_kv;
    const int G = p.h_q / p.c.h_kv, heads = G - 16 * ht < 16 ? G - 16 * ht : 16;
    const int64_t cap = p.c.num_pages > 0 ? p.c.max_pages << page_shift : 0;
    int64_t len = p.lens[seq];
    len = len < p.max_len ? len : p.max_len;
    len = len < cap ? len : cap;
    const int64_t begin = rg * range;
    if (rg > 0 && begin >= len) return;  // the join does not read this range
    const bool whole = len <= range;     // nothing to join
    const int64_t end = begin + range < len ? begin + range : len;

    // Q as the B operand: column c is head 16 ht + c (heads past the group repeat the last), piece x
    // of element order (i * 4 + g) * EPK .. for load i of a K row. In registers, or in LDS where a
    // row's K, V and O leave no room.
    const T* qrow = static_cast<const T*>(p.q) + seq * p.q_token;
    const int head0 = kvh * G + 16 * ht;
    constexpr int QP = C::EPK * (int)sizeof(T) / 16;  // 16-byte pieces of a load's elements
    u32x4_t q[C::QLDS ? 1 : C::KL * QP];
    if constexpr (C::QLDS) {
        constexpr int CH = D * (int)sizeof(T) / 16;
        for (int x = threadIdx.x; x < 16 * CH; x += 64 * kWaves) {
            const int h = x / CH < heads ? x / CH : heads - 1;
            *reinterpret_cast<u32x4_t*>(s_q + x / CH * C::QSTRIDE + x % CH * 16) =
                *reinterpret_cast<const u32x4_t*>(qrow + (head0 + h) * p.q_head + x % CH * (16 / (int)sizeof(T)));
        }
    } else {
        const T* qp = qrow + (head0 + (c < heads ? c : heads - 1)) * p.q_head;
#pragma unroll
        for (int i = 0; i < C::KL; ++i)
#pragma unroll
            for (int x = 0; x < QP; ++x)
                q[i * QP + x] = *reinterpret_cast<const u32x4_t*>(qp + (i * 4 + g) * C::EPK + x * (16 / (int)sizeof(T)));
    }
    int qoff = c * C::QSTRIDE + g * C::EPK * (int)sizeof(T);
    auto q_at = [&](int i, int x) __attribute__((always_inline)) {
        if constexpr (C::QLDS)
            return *reinterpret_cast<const u32x4_t*>(s_q + qoff + i * 4 * C::EPK * (int)sizeof(T) + x * 16);
        else
            return q[i * QP + x];
    };
    if constexpr (C::QLDS) __syncthreads();

    f32x4_t o[C::VL];
#pragma unroll
    for (int j = 0; j < C::VL; ++j) o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f, exact = 0.f;
    const float cs = p.scale * kLog2e;
    const int32_t* table = p.c.page_table + seq * p.c.max_pages;
    const char* kpool = static_cast<const char*>(p.c.k);
    const char* vpool = static_cast<const char*>(p.c.v);

    u32x4_t kx[C::NB][C::KL];
    VP vx[4 * C::NB][C::U];
    uint32_t sk[C::NB], sv[C::NB];

    // Row of the pools where block b of the step at j0 begins; absent pages read page 0 (and are
    // masked), positions past the range's end the page of its last.
    auto block_row = [&](int64_t j0, int b, bool* there) {
        const int64_t pos = j0 + 16 * b;
        const int64_t page = table[(pos < end ? pos : end - 1) >> page_shift];
        *there = page >= 0 && page < p.c.num_pages;
        return (((*there ? page : 0) * p.c.h_kv + kvh) << page_shift) + (pos & (p.c.page_size - 1));
    };
    auto load_k = [&](const int64_t* row) {
#pragma unroll
        for (int b = 0; b < C::NB; ++b) {
            const char* kr = kpool + (row[b] + c) * (D * C::ES) + g * 16;
#pragma unroll
            for (int i = 0; i < C::KL; ++i) kx[b][i] = *reinterpret_cast<const u32x4_t*>(kr + i * 64);
            if constexpr (FP8) sk[b] = *reinterpret_cast<const uint32_t*>(p.c.k_scale + row[b] + 4 * g);
        }
    };
    auto load_v = [&](const int64_t* row) {
#pragma unroll
        for (int b = 0; b < C::NB; ++b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const char* vr = vpool + (row[b] + 4 * g + i) * (D * C::ES) + c * (C::EPL * C::ES);
#pragma unroll
                for (int u = 0; u < C::U; ++u)
                    vx[4 * b + i][u] = *reinterpret_cast<const VP*>(vr + u * (16 * C::EPL * C::ES));
            }
            if constexpr (FP8) sv[b] = *reinterpret_cast<const uint32_t*>(p.c.v_scale + row[b] + 4 * g);
        }
    };

    // The next step's K is loaded when this step's scores are done, its V when this step's sum
    // is: the registers are free then, and a wave always has loads in flight.
    int64_t row[C::NB];
    bool there[C::NB];
    const int64_t first = begin + wave * C::STEP;
    if (first < end) {
#pragma unroll
        for (int b = 0; b < C::NB; ++b) row[b] = block_row(first, b, &there[b]);
        load_k(row);
        load_v(row);
    }
    for (int64_t j0 = first; j0 < end; j0 += kWaves * C::STEP) {
        const int64_t next = j0 + kWaves * C::STEP;
        int64_t nrow[C::NB] = {};
        bool nthere[C::NB] = {};
        if (next < end)
#pragma unroll
            for (int b = 0; b < C::NB; ++b) nrow[b] = block_row(next, b, &nthere[b]);

        // scores
        if constexpr (C::QLDS) asm volatile("" : "+v"(qoff));  // read again in every step, not kept
        float s[4 * C::NB];
#pragma unroll
        for (int b = 0; b < C::NB; ++b) {
            f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < C::KL; ++i) {
                if constexpr (BF && !FP8) {
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, kx[b][i]), __builtin_bit_cast(bf16x8_t, q_at(i, 0)), acc, 0, 0, 0);
                } else if constexpr (BF) {
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const u32x4_t a = {cvt_bf16_fp8(kx[b][i][2 * f], false), cvt_bf16_fp8(kx[b][i][2 * f], true),
                                           cvt_bf16_fp8(kx[b][i][2 * f + 1], false), cvt_bf16_fp8(kx[b][i][2 * f + 1], true)};
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, q_at(i, f)), acc, 0, 0, 0);
                    }
                } else if constexpr (!FP8) {
                    const u32x4_t qq = q_at(i, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kx[b][i][e]), __uint_as_float(qq[e]), acc, 0, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const u32x4_t qq = q_at(i, e / 4);
                        const f32x2_t a = e & 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)kx[b][i][e / 4], true)
                                                : __builtin_amdgcn_cvt_pk_f32_fp8((int)kx[b][i][e / 4], false);
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[0], __uint_as_float(qq[e % 4]), acc, 0, 0, 0);
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[1], __uint_as_float(qq[e % 4 + 1]), acc, 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[4 * b + i] = acc[i] * cs;
                if constexpr (FP8) s[4 * b + i] *= scale_of((sk[b] >> (8 * i)) & 0xff);
            }
        }
        if (next < end) load_k(nrow);

        const bool masked = j0 + C::STEP > end || !there[0] || !there[C::NB - 1];
        if (masked)
#pragma unroll
            for (int i = 0; i < 4 * C::NB; ++i)
                if (!there[i / 4] || j0 + 16 * (i / 4) + 4 * g + i % 4 >= end) {
                    s[i] = -INFINITY;
                    // what lies there is anything: not into the product
#pragma unroll
                    for (int u = 0; u < C::U; ++u) vx[i][u] = VP{};
                    if constexpr (FP8) sv[i / 4] &= ~(0xffu << (8 * (i % 4)));
                }

        // softmax; the reference maximum moves only when weights would pass 2^8
        float mx = s[0];
#pragma unroll
        for (int i = 1; i < 4 * C::NB; ++i) mx = fmaxf(mx, s[i]);
        if (__any(mx > m && (m == -INFINITY || mx > m + 8.f))) {
            const auto a16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
            mx = fmaxf(__uint_as_float(a16[0]), __uint_as_float(a16[1]));
            const auto a32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
            mx = fmaxf(__uint_as_float(a32[0]), __uint_as_float(a32[1]));
            const float mn = fmaxf(m, mx);  // the same in all lanes of a head
            const float a = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= a;
            exact *= a;
#pragma unroll
            for (int j = 0; j < C::VL; ++j) o[j] *= a;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        // Weights. For the product with bf16 V they are rounded to bf16; l is of what V is multiplied
        // by, so that a rounding that all elements share cancels; lse is of the unrounded sum.
#pragma unroll
        for (int i = 0; i < 4 * C::NB; ++i) {
            s[i] = __builtin_amdgcn_exp2f(s[i] - ref);
            exact += s[i];
            if constexpr (BF) s[i] = round_bf16(s[i]);
            l += s[i];
            // exact, but for rows of V so small that the product is below the normal range
            if constexpr (FP8) s[i] *= scale_of((sv[i / 4] >> (8 * (i % 4))) & 0xff);
        }

        // O^T += V^T P^T; o[u * EPL + j] rows are elements 16 EPL u + EPL (4 g + i) + j
        if constexpr (BF) {
            const u32x4_t pw = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7])};
            const bf16x8_t pb = __builtin_bit_cast(bf16x8_t, pw);
            auto add = [&](int at, u32x4_t a) __attribute__((always_inline)) {
                o[at] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), pb, o[at], 0, 0, 0);
            };
#pragma unroll
            for (int u = 0; u < C::U; ++u) {
                if constexpr (!FP8) {
#pragma unroll
                    for (int j = 0; j < C::EPL; ++j) {
                        u32x4_t a;
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            a[x] = __builtin_amdgcn_perm(word(vx[2 * x + 1][u], j / 2), word(vx[2 * x][u], j / 2),
                                                         j & 1 ? 0x07060302u : 0x05040100u);
                        add(u * C::EPL + j, a);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < C::EPL; j += 2) {
                        u32x4_t a0, a1;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            // bytes j and j + 1 of two keys, interleaved
                            const uint32_t y = __builtin_amdgcn_perm(word(vx[2 * x + 1][u], j / 4), word(vx[2 * x][u], j / 4),
                                                                     j & 2 ? 0x07030602u : 0x05010400u);
                            a0[x] = cvt_bf16_fp8(y, false);
                            a1[x] = cvt_bf16_fp8(y, true);
                        }
                        add(u * C::EPL + j, a0);
                        add(u * C::EPL + j + 1, a1);
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4 * C::NB; ++i)
#pragma unroll
                for (int u = 0; u < C::U; ++u)
#pragma unroll
                    for (int j = 0; j < C::EPL; ++j) {
                        float a;
                        if constexpr (!FP8) a = __uint_as_float(word(vx[i][u], j));
                        else a = j & 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)word(vx[i][u], j / 4), true)[j & 1]
                                       : __builtin_amdgcn_cvt_pk_f32_fp8((int)word(vx[i][u], j / 4), false)[j & 1];
                        o[u * C::EPL + j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, s[i], o[u * C::EPL + j], 0, 0, 0);
                    }
        }
        if (next < end) load_v(nrow);
#pragma unroll
        for (int b = 0; b < C::NB; ++b) there[b] = nthere[b];
    }

    // join the waves: weights relative to the largest maximum. A wave that saw nothing but NaN
    // scores has m = -inf as one that saw no key has; its sums are NaN, and 0 x NaN hands them on
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    exact += __shfl_xor(exact, 16, 64);
    exact += __shfl_xor(exact, 32, 64);
    if (g == 0) {
        s_m[wave][c] = m;
        s_l[wave][c] = make_float2(l, exact);
    }
    __syncthreads();
    float mm = s_m[0][c];
#pragma unroll
    for (int x = 1; x < kWaves; ++x) mm = fmaxf(mm, s_m[x][c]);
    const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mm);
    if (c < heads) {
#pragma unroll
        for (int u = 0; u < C::U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < C::EPL; ++j)
                    s_o[wave][c][16 * C::EPL * u + C::EPL * (4 * g + i) + j] = o[u * C::EPL + j][i] * f;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < heads * (D / 4); x += 64 * kWaves) {
        const int hd = x / (D / 4), el = x % (D / 4) * 4;
        float top = s_m[0][hd];
#pragma unroll
        for (int y = 1; y < kWaves; ++y) top = fmaxf(top, s_m[y][hd]);
        f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
        float ls = 0.f, le = 0.f;
#pragma unroll
        for (int y = 0; y < kWaves; ++y) sum += *reinterpret_cast<const f32x4_t*>(&s_o[y][hd][el]);
#pragma unroll
        for (int y = 0; y < kWaves; ++y) {
            const float w = s_m[y][hd] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(s_m[y][hd] - top);
            ls += s_l[y][hd].x * w;
            le += s_l[y][hd].y * w;
        }
        if (whole) {
            const int64_t orow = seq * p.h_q + kvh * G + 16 * ht + hd;
            const float inv = ls > 0.f ? 1.f / ls : (ls == ls ? 0.f : ls);
            sum *= inv;
            T* out = static_cast<T*>(p.out) + orow * D + el;
            if constexpr (BF) *reinterpret_cast<u32x2_t*>(out) = u32x2_t{pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
            else *reinterpret_cast<f32x4_t*>(out) = sum;
            if (p.lse && el == 0) p.lse[orow] = le > 0.f ? (top + __builtin_amdgcn_logf(le)) * kLn2 : (le == le ? -INFINITY : le);
        } else {
            const int64_t at = (unit * ranges + rg) * 16 + hd;
            *reinterpret_cast<f32x4_t*>(part.o + at * D + el) = sum;
            if (el == 0) part.ml[at] = make_float4(top, ls, le, 0.f);
        }
    }
}

// Joins the ranges of one (sequence, head), 64 elements of it: the ranges' sums weighted by
// exp2(m - max m). 16 lanes hold the elements, the blockDim / 16 groups of them take the ranges
// in turn (few ranges need few groups: see join_threads); the order of the additions depends on
// the sizes only. Latency-bound: 4.4 us for 16 heads of 128 ranges, 7.6 us for 2048 of up to 8.
constexpr int kJoinGroups = 64;  // at most

int join_threads(int64_t ranges)
{
    const int64_t t = (ranges + 3) / 4 * 16;  // about four ranges a group
    return t < 64 ? 64 : t > 16 * kJoinGroups ? 16 * kJoinGroups : (int)((t + 63) / 64 * 64);
}

template <typename T, int D>
__global__ void __launch_bounds__(16 * kJoinGroups) decode_join_kernel(AttnDecodeCall p, int64_t range,
                                                                       int ranges, int head_tiles,
                                                                       int page_shift, Partials part)
{
    __shared__ f32x4_t s_o[kJoinGroups][16];
    __shared__ float2 s_l[kJoinGroups];
    __shared__ float s_m[kJoinGroups / 4];
    const int groups = blockDim.x / 16;
    const int64_t hrow = blockIdx.x / (D / 64);
    const int64_t seq = hrow / p.h_q;
    const int hq = (int)(hrow - seq * p.h_q);
    const int G = p.h_q / p.c.h_kv, kvh = hq / G, hg = hq - kvh * G, ht = hg / 16, hd = hg % 16;
    const int64_t cap = p.c.num_pages > 0 ? p.c.max_pages << page_shift : 0;
    int64_t len = p.lens[seq];
    len = len < p.max_len ? len : p.max_len;
    len = len < cap ? len : cap;
    if (len <= range) return;  // written by its only range
    const int used = (int)((len + range - 1) / range);
    const int64_t unit = (seq * p.c.h_kv + kvh) * head_tiles + ht;
    const float4* ml = part.ml + unit * ranges * 16 + hd;
    const int y = threadIdx.x / 16, el = (int)(blockIdx.x % (D / 64)) * 64 + threadIdx.x % 16 * 4;
    const float* po = part.o + (unit * ranges * 16 + hd) * D + el;

    float top = -INFINITY;
    for (int x = threadIdx.x; x < used; x += blockDim.x) top = fmaxf(top, ml[(int64_t)x * 16].x);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    if (threadIdx.x % 64 == 0) s_m[threadIdx.x / 64] = top;
    __syncthreads();
    for (int x = 0; x < (int)blockDim.x / 64; ++x) top = fmaxf(top, s_m[x]);

    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    float ls = 0.f, le = 0.f;
#pragma unroll 4
    for (int x = y; x < used; x += groups) {
        const float4 v = ml[(int64_t)x * 16];
        const f32x4_t a = *reinterpret_cast<const f32x4_t*>(po + (int64_t)x * 16 * D);
        const float f = v.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(v.x - top);
        ls += v.y * f;
        le += v.z * f;
        sum += a * f;
    }
    s_o[y][threadIdx.x % 16] = sum;
    if (threadIdx.x % 16 == 0) s_l[y] = make_float2(ls, le);
    __syncthreads();
    if (y != 0) return;
    float l = 0.f, e = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int x = 0; x < groups; ++x) {
        o += s_o[x][threadIdx.x];
        l += s_l[x].x;
        e += s_l[x].y;
    }
    o *= l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    T* out = static_cast<T*>(p.out) + hrow * D + el;
    if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2_t*>(out) = u32x2_t{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    else *reinterpret_cast<f32x4_t*>(out) = o;
    if (p.lse && el == 0) p.lse[hrow] = e > 0.f ? (top + __builtin_amdgcn_logf(e)) * kLn2 : (e == e ? -INFINITY : e);
}

template <typename T, bool FP8, int D>
hipError_t launch_t(const AttnDecodeCall& c)
{
    const Plan pl = make_plan(&c.c, c.h_q, c.max_len);
    const int64_t units = c.c.n * c.c.h_kv * pl.head_tiles;
    const int shift = __builtin_ctz((unsigned)c.c.page_size);
    Partials part;
    part.o = static_cast<float*>(c.ws);
    part.ml = reinterpret_cast<float4*>(part.o + units * pl.ranges * 16 * D);
    hipLaunchKernelGGL((decode_attn_kernel<T, FP8, D>), grid_of(units * pl.ranges), dim3(64 * kWaves), 0, c.stream, c,
                       pl.range, (int)pl.ranges, pl.head_tiles, shift, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || pl.ranges == 1) return e;
    hipLaunchKernelGGL((decode_join_kernel<T, D>), dim3((unsigned)(c.c.n * c.h_q * (D / 64))), dim3(join_threads(pl.ranges)), 0, c.stream, c,
                       pl.range, (int)pl.ranges, pl.head_tiles, shift, part);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_store(const AttnDecodeCall& c)
{
    return c.c.store == GDN_FP8 ? launch_t<T, true, D>(c) : launch_t<T, false, D>(c);
}

template <typename T>
hipError_t launch_d(const AttnDecodeCall& c)
{
    switch (c.c.d) {
        case 64: return launch_store<T, 64>(c);
        case 128: return launch_store<T, 128>(c);
        case 256: return launch_store<T, 256>(c);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

size_t attn_decode_workspace(const gdn_kv_cache* c, int32_t h_q, int64_t max_len)
{
    const Plan pl = make_plan(c, h_q, max_len);
    if (pl.ranges == 1) return 0;
    return (size_t)(c->n * c->h_kv * pl.head_tiles * pl.ranges) * 16 * (c->d * sizeof(float) + sizeof(float4));
}

hipError_t launch_attn_decode(const AttnDecodeCall& c)
{
    return c.dtype == GDN_BF16 ? launch_d<uint16_t>(c) : launch_d<float>(c);
}

}  // namespace gdn
