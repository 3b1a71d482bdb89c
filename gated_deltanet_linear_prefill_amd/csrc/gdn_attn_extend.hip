// gdn_attn_extend.hip -- attention of new tokens over the paged cache: a few rows per sequence.
//
// Rows. The G = h_q / h_kv heads of a KV head read the same keys, so the rows of one (sequence, KV
// head) are numbered position-major, row r being position r / G, head r % G, and a workgroup takes
// M = 16 CT of them, over a part of the positions that they see (gdn_extend.hpp).
//
// Positions. What a tile's rows see together is [0, sinks) and the stretch from the first row's window
// to the last row. Both are taken in whole 16-position blocks, which never cross a page, and numbered
// through ("virtual" positions); ranges and steps are of these, so that a window costs its own
// length and no page outside it is looked at.
//
// Bound by the bytes of the cache: one token of each of 64 sequences of up to 8192 positions, d = 128, 32/8
// heads, runs at 5.2 TB/s with the join (212 us), 16 sequences of 4 tokens at 4.0 (72 us, 4.7 of them the join's), 32
// behind a window of 4096, d = 256, at 4.1 (59 us). A wave takes 32 positions (16 for long rows) of K and V into
// registers, for all M rows, with its own softmax state; waves are joined in LDS, ranges by a second
// kernel through the workspace. 16x16 MFMA, one row per column: S^T = K Q^T takes 16-byte pieces of K
// rows as its A operand as they were loaded, and its result is the B operand of O^T = V^T P^T, if
// lane (c, g) brings pieces of the V rows of keys 4 g + i. No K, V or weight passes between lanes;
// Q is read from LDS. The next step's K is loaded when this step's scores are done, its V when this
// step's product is.
//
// A key that only some rows see may hold a NaN or an infinity, and 0 x NaN is NaN: in steps with
// masked keys such elements of V are left out of the product and added to the rows that see them.
#include "gdn_extend.hpp"

namespace gdn {
namespace {

constexpr int kWaves = 4;
constexpr int kRange = 32 * kWaves;  // ranges are multiples of this: a step of every wave
static_assert(kRange == kStep, "shares are of whole steps");

template <typename T, bool FP8, int D, int CT>
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
    static constexpr int QSTRIDE = D * (int)sizeof(T) + 16;    // bytes of a row of Q in LDS
    static constexpr int M = 16 * CT;
    // registers of O, K and V; with 512 a wave there is one wave a SIMD
    static constexpr int REGS = CT * VL * 4 + 2 * NB * KL * 4;
    static constexpr int PER_SIMD = REGS > (CT > 1 ? 159 : 192) ? 1 : 2;
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

template <typename P>
__device__ __forceinline__ void set_word(P& p, int i, uint32_t x)
{
    if constexpr (sizeof(P) == 4) p = x;
    else p[i] = x;
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

// All ones in the places of a word's elements of ES bytes that are NaN or infinite.
template <int ES>
__device__ __forceinline__ uint32_t odd_mask(uint32_t w)
{
    if constexpr (ES == 4) return (w & 0x7f800000u) == 0x7f800000u ? 0xffffffffu : 0u;
    else if constexpr (ES == 2) return ((((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 15) * 0xffffu;
    else return ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu;
}

// An element of a V row that is NaN or infinite, else 0.
template <typename T, bool FP8>
__device__ __forceinline__ float odd_element(const char* row, int e)
{
    if constexpr (FP8) {
        return (static_cast<uint8_t>(row[e]) & 0x7f) == 0x7f ? __uint_as_float(0x7fc00000u) : 0.f;
    } else {
        const float x = load1_f32(reinterpret_cast<const T*>(row) + e);
        return fabsf(x) <= 3.4028234e38f ? 0.f : x;
    }
}

template <typename T, bool FP8, int D, int CT>
__global__ void __launch_bounds__(64 * kWaves, (Cfg<T, FP8, D, CT>::PER_SIMD)) extend_kernel(ExtendArgs a)
{
    using C = Cfg<T, FP8, D, CT>;
    using VP = typename Piece<C::EPL * C::ES>::type;
    constexpr bool BF = sizeof(T) == 2;
    constexpr int M = C::M, NB = C::NB;
    const ExtendCall& p = a.c;
    constexpr int O_BYTES = kWaves * 16 * (D + 4) * 4, Q_BYTES = M * C::QSTRIDE;
    __shared__ __align__(16) char s_buf[O_BYTES > Q_BYTES ? O_BYTES : Q_BYTES];
    __shared__ float s_m[kWaves][M];
    __shared__ float2 s_l[kWaves][M];
    char* const s_q = s_buf;  // until the waves are joined
    float(*const s_o)[16][D + 4] = reinterpret_cast<float(*)[16][D + 4]>(s_buf);

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    Part part;
    if (!find_part<M>(a, block_index(), &part)) return;
    const Span& t = part.t;
    const int kvh = t.head;
    const int64_t begin64 = part.rg * part.range;
    if (part.rg > 0 && begin64 >= t.len) return;  // the join does not read this range
    const bool whole = t.len <= part.range;       // nothing to join
    const int begin = (int)begin64;
    const int end = t.len - begin < part.range ? t.len : (int)(begin64 + part.range);

    // Q: row r of the tile, rows past the sequence's repeat its last
    const int left = t.rows - t.row0, have = left < M ? left : M;
    constexpr int CH = D * (int)sizeof(T) / 16;
    for (int x = threadIdx.x; x < M * CH; x += 64 * kWaves) {
        const int r = t.row0 + (x / CH < have ? x / CH : have - 1), i = r / t.g;
        *reinterpret_cast<u32x4_t*>(s_q + x / CH * C::QSTRIDE + x % CH * 16) = *reinterpret_cast<const u32x4_t*>(
            static_cast<const T*>(p.q) + (int64_t)(t.q0 + i) * p.d.q_token +
            (int64_t)(kvh * t.g + r - i * t.g) * p.d.q_head + x % CH * (16 / (int)sizeof(T)));
    }
    int upto[CT];  // virtual positions that this lane's rows see end here
#pragma unroll
    for (int x = 0; x < CT; ++x)
        upto[x] = max(t.shift + (t.row0 + (16 * x + c < have ? 16 * x + c : have - 1)) / t.g + 1 - t.skip, 0);
    int qoff = c * C::QSTRIDE + g * C::EPK * (int)sizeof(T);
    auto q_at = [&](int ct, int i, int x) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4_t*>(s_q + qoff + ct * 16 * C::QSTRIDE + i * 4 * C::EPK * (int)sizeof(T) + x * 16);
    };
    __syncthreads();

    const int sinks = (int)p.d.sinks, window = (int)p.d.window;
    auto sees = [&](int v, int x) __attribute__((always_inline)) {
        return (v < upto[x]) & (!window | (v >= upto[x] - window) | (v < sinks));
    };
    // every row sees the positions before `all` that are in the last row's window, from `from` on, or sinks
    const int all = t.first + 1 - t.skip, from = window ? t.len - window : 0;
    f32x4_t o[CT][C::VL];
    float m[CT], l[CT], exact[CT];
#pragma unroll
    for (int x = 0; x < CT; ++x) {
#pragma unroll
        for (int j = 0; j < C::VL; ++j) o[x][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        m[x] = -INFINITY;
        l[x] = exact[x] = 0.f;
    }
    const float cs = p.d.scale * kLog2e;
    const int32_t* table = p.c.page_table + t.seq * p.c.max_pages;
    const char* kpool = static_cast<const char*>(p.c.k);
    const char* vpool = static_cast<const char*>(p.c.v);

    u32x4_t kx[NB][C::KL];
    VP vx[4 * NB][C::U];
    uint32_t sk[NB], sv[NB];

    // Row of the pools where block b of the step at virtual position j0 begins; absent pages read page 0
    // (and are masked), blocks past the range's end the last before it.
    auto block_row = [&](int j0, int b, bool* there) {
        const int v = j0 + 16 * b, pos = t.pos(v < end ? v : (end - 1) & ~15);
        const int64_t page = table[pos >> a.page_shift];
        *there = page >= 0 && page < p.c.num_pages;
        return (((*there ? page : 0) * p.c.h_kv + kvh) << a.page_shift) + (pos & (p.c.page_size - 1));
    };
    // A block's rows begin at a scalar address; what a lane adds to it is 32 bits, made from the lane's number
    // in every step: the registers are full, and an offset reloaded from scratch memory would wait for
    // the loads before it.
    uint32_t own = lane;
    auto load_k = [&](const int64_t* row) {
        asm volatile("" : "+v"(own));
        const uint32_t koff = (own & 15) * (D * C::ES) + (own >> 4) * 16, soff = (own >> 4) * 4;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const char* kr = kpool + row[b] * (D * C::ES);
#pragma unroll
            for (int i = 0; i < C::KL; ++i) kx[b][i] = *reinterpret_cast<const u32x4_t*>(kr + koff + i * 64);
            if constexpr (FP8) sk[b] = *reinterpret_cast<const uint32_t*>(p.c.k_scale + row[b] + soff);
        }
    };
    auto load_v = [&](const int64_t* row) {
        asm volatile("" : "+v"(own));
        const uint32_t voff = (own >> 4) * (4 * D * C::ES) + (own & 15) * (C::EPL * C::ES), soff = (own >> 4) * 4;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const char* vr = vpool + row[b] * (D * C::ES);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < C::U; ++u)
                    vx[4 * b + i][u] = *reinterpret_cast<const VP*>(vr + voff + i * (D * C::ES) + u * (16 * C::EPL * C::ES));
            if constexpr (FP8) sv[b] = *reinterpret_cast<const uint32_t*>(p.c.v_scale + row[b] + soff);
        }
    };

    int64_t row[NB];
    bool there[NB];
    const int first = begin + wave * C::STEP;
    if (first < end) {
#pragma unroll
        for (int b = 0; b < NB; ++b) row[b] = block_row(first, b, &there[b]);
        load_k(row);
        load_v(row);
    }
    // the host keeps lengths below 2^31 - 2^16, so that a step past the end is still an int
    for (int j0 = first; j0 < end; j0 += kWaves * C::STEP) {
        const int next = j0 + kWaves * C::STEP;
        int64_t nrow[NB] = {};
        bool nthere[NB] = {};
        if (next < end)
#pragma unroll
            for (int b = 0; b < NB; ++b) nrow[b] = block_row(next, b, &nthere[b]);

        // scores
        asm volatile("" : "+v"(qoff));  // read again in every step, not kept
        float s[CT][4 * NB];
        {
            f32x4_t acc[CT][NB];
#pragma unroll
            for (int x = 0; x < CT; ++x)
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[x][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < C::KL; ++i) {
                constexpr int QP = C::EPK * (int)sizeof(T) / 16;  // 16-byte pieces of a load's elements
#pragma unroll
                for (int f = 0; f < QP; ++f) {
                    u32x4_t k16[NB];
                    if constexpr (BF)
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            if constexpr (FP8)
                                k16[b] = u32x4_t{cvt_bf16_fp8(kx[b][i][2 * f], false), cvt_bf16_fp8(kx[b][i][2 * f], true),
                                                 cvt_bf16_fp8(kx[b][i][2 * f + 1], false), cvt_bf16_fp8(kx[b][i][2 * f + 1], true)};
                            else
                                k16[b] = kx[b][i];
                        }
#pragma unroll
                    for (int x = 0; x < CT; ++x) {
                        const u32x4_t qq = q_at(x, i, f);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            if constexpr (BF) {
                                acc[x][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, k16[b]),
                                                                                    __builtin_bit_cast(bf16x8_t, qq), acc[x][b], 0, 0, 0);
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float k1;
                                    if constexpr (FP8)
                                        k1 = e & 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)kx[b][i][f], true)[e & 1]
                                                   : __builtin_amdgcn_cvt_pk_f32_fp8((int)kx[b][i][f], false)[e & 1];
                                    else
                                        k1 = __uint_as_float(kx[b][i][e]);
                                    acc[x][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(k1, __uint_as_float(qq[e]), acc[x][b], 0, 0, 0);
                                }
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < CT; ++x)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[x][4 * b + i] = acc[x][b][i] * cs;
                        if constexpr (FP8) s[x][4 * b + i] *= scale_of((sk[b] >> (8 * i)) & 0xff);
                    }
        }
        if (next < end) load_k(nrow);

        bool masked = false;
#pragma unroll
        for (int b = 0; b < NB; ++b)
            masked |= !there[b] || j0 + 16 * b + 16 > all || (j0 + 16 * b < from && j0 + 16 * b + 16 > sinks);
        bool odd = false;
        uint32_t seen[CT];  // bits of this lane's keys
        if (masked) {
#pragma unroll
            for (int x = 0; x < CT; ++x) seen[x] = 0;
            uint32_t found = 0;
            asm volatile("" : "+v"(own));  // comparisons ahead of the branch would be made for every step
            const int mine = (int)(own >> 4) * 4;
#pragma unroll
            for (int i = 0; i < 4 * NB; ++i) {
                const int b = i / 4, v = j0 + 16 * b + mine + i % 4;
                const bool exists = there[b] && v < end;
                if (!exists) {  // what lies there is anything: not into the product
#pragma unroll
                    for (int u = 0; u < C::U; ++u) vx[i][u] = VP{};
                    if constexpr (FP8) sv[b] &= ~(0xffu << (8 * (i % 4)));
                }
#pragma unroll
                for (int x = 0; x < CT; ++x) {
                    const bool in = exists & sees(v, x);
                    s[x][i] = in ? s[x][i] : -INFINITY;
                    seen[x] |= (uint32_t)in << i;
                }
#pragma unroll
                for (int u = 0; u < C::U; ++u)
#pragma unroll
                    for (int w = 0; w < (int)sizeof(VP) / 4; ++w) found |= odd_mask<C::ES>(word(vx[i][u], w));
            }
            odd = __any(found != 0);
            if (odd)
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i)
#pragma unroll
                    for (int u = 0; u < C::U; ++u)
#pragma unroll
                        for (int w = 0; w < (int)sizeof(VP) / 4; ++w)
                            set_word(vx[i][u], w, word(vx[i][u], w) & ~odd_mask<C::ES>(word(vx[i][u], w)));
        }

        u32x4_t pw[CT];
#pragma unroll
        for (int x = 0; x < CT; ++x) {
            // softmax; the reference maximum moves only when weights would pass 2^8
            float mx = s[x][0];
#pragma unroll
            for (int i = 1; i < 4 * NB; ++i) mx = fmaxf(mx, s[x][i]);
            if (__any(mx > m[x] && (m[x] == -INFINITY || mx > m[x] + 8.f))) {
                const auto a16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
                mx = fmaxf(__uint_as_float(a16[0]), __uint_as_float(a16[1]));
                const auto a32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
                mx = fmaxf(__uint_as_float(a32[0]), __uint_as_float(a32[1]));
                const float mn = fmaxf(m[x], mx);  // the same in all lanes of a row
                const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[x] - mn);
                m[x] = mn;
                l[x] *= f;
                exact[x] *= f;
#pragma unroll
                for (int j = 0; j < C::VL; ++j) o[x][j] *= f;
            }
            const float ref = m[x] == -INFINITY ? 0.f : m[x];
            // Weights. For the product with bf16 V they are rounded to bf16; l is of what V is multiplied
            // by, so that a rounding that all elements share cancels; lse is of the unrounded sum.
#pragma unroll
            for (int i = 0; i < 4 * NB; ++i) {
                s[x][i] = __builtin_amdgcn_exp2f(s[x][i] - ref);
                exact[x] += s[x][i];
                if constexpr (BF) s[x][i] = round_bf16(s[x][i]);
                l[x] += s[x][i];
                // exact, but for rows of V so small that the product is below the normal range
                if constexpr (FP8) {
                    s[x][i] *= scale_of((sv[i / 4] >> (8 * (i % 4))) & 0xff);
                    if (masked && !(seen[x] >> i & 1)) s[x][i] = 0.f;
                }
            }
            if constexpr (BF)
                pw[x] = u32x4_t{pack_bf16(s[x][0], s[x][1]), pack_bf16(s[x][2], s[x][3]), pack_bf16(s[x][4], s[x][5]),
                                pack_bf16(s[x][6], s[x][7])};
        }

        // O^T += V^T P^T; o[.][u * EPL + j] rows are elements 16 EPL u + EPL (4 g + i) + j
        if constexpr (BF) {
            auto add = [&](int y, u32x4_t v) __attribute__((always_inline)) {
#pragma unroll
                for (int x = 0; x < CT; ++x)
                    o[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v),
                                                                      __builtin_bit_cast(bf16x8_t, pw[x]), o[x][y], 0, 0, 0);
            };
#pragma unroll
            for (int u = 0; u < C::U; ++u) {
                if constexpr (!FP8) {
#pragma unroll
                    for (int j = 0; j < C::EPL; ++j) {
                        u32x4_t v;
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            v[x] = __builtin_amdgcn_perm(word(vx[2 * x + 1][u], j / 2), word(vx[2 * x][u], j / 2),
                                                         j & 1 ? 0x07060302u : 0x05040100u);
                        add(u * C::EPL + j, v);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < C::EPL; j += 2) {
                        u32x4_t v0, v1;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            // bytes j and j + 1 of two keys, interleaved
                            const uint32_t y = __builtin_amdgcn_perm(word(vx[2 * x + 1][u], j / 4), word(vx[2 * x][u], j / 4),
                                                                     j & 2 ? 0x07030602u : 0x05010400u);
                            v0[x] = cvt_bf16_fp8(y, false);
                            v1[x] = cvt_bf16_fp8(y, true);
                        }
                        add(u * C::EPL + j, v0);
                        add(u * C::EPL + j + 1, v1);
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4 * NB; ++i)
#pragma unroll
                for (int u = 0; u < C::U; ++u)
#pragma unroll
                    for (int j = 0; j < C::EPL; ++j) {
                        float v;
                        if constexpr (!FP8) v = __uint_as_float(word(vx[i][u], j));
                        else v = j & 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)word(vx[i][u], j / 4), true)[j & 1]
                                       : __builtin_amdgcn_cvt_pk_f32_fp8((int)word(vx[i][u], j / 4), false)[j & 1];
#pragma unroll
                        for (int x = 0; x < CT; ++x)
                            o[x][u * C::EPL + j] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, s[x][i], o[x][u * C::EPL + j], 0, 0, 0);
                    }
        }
        if (odd) {
            // What was left out, key by key: in a row that sees the key any positive weight of an infinity
            // is that infinity, and NaN is NaN.
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (!there[b]) continue;
#pragma unroll 1
                for (int key = 0; key < 16 && j0 + 16 * b + key < end; ++key) {
                    const char* vr = vpool + (row[b] + key) * (D * C::ES);
                    const int v = j0 + 16 * b + key;
#pragma unroll
                    for (int y = 0; y < C::VL; ++y)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float e = odd_element<T, FP8>(vr, 16 * C::EPL * (y / C::EPL) + C::EPL * (4 * g + i) + y % C::EPL);
#pragma unroll
                            for (int x = 0; x < CT; ++x)
                                if (sees(v, x)) o[x][y][i] += e;
                        }
                }
            }
        }
        if (next < end) load_v(nrow);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            row[b] = nrow[b];
            there[b] = nthere[b];
        }
    }

    // Join the waves, 16 rows at a time: weights relative to the largest maximum. A wave that saw nothing
    // but NaN scores has m = -inf as one that saw no key has; its sums are NaN, and 0 x NaN hands them on.
#pragma unroll
    for (int x = 0; x < CT; ++x) {
        l[x] += __shfl_xor(l[x], 16, 64);
        l[x] += __shfl_xor(l[x], 32, 64);
        exact[x] += __shfl_xor(exact[x], 16, 64);
        exact[x] += __shfl_xor(exact[x], 32, 64);
        if (g == 0) {
            s_m[wave][16 * x + c] = m[x];
            s_l[wave][16 * x + c] = make_float2(l[x], exact[x]);
        }
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        __syncthreads();
        if (16 * ct >= have) break;
        float mm = s_m[0][16 * ct + c];
#pragma unroll
        for (int x = 1; x < kWaves; ++x) mm = fmaxf(mm, s_m[x][16 * ct + c]);
        const float f = m[ct] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[ct] - mm);
#pragma unroll
        for (int u = 0; u < C::U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < C::EPL; ++j)
                    s_o[wave][c][16 * C::EPL * u + C::EPL * (4 * g + i) + j] = o[ct][u * C::EPL + j][i] * f;
        __syncthreads();
        const int rows = have - 16 * ct < 16 ? have - 16 * ct : 16;
        for (int x = threadIdx.x; x < rows * (D / 4); x += 64 * kWaves) {
            const int y = x / (D / 4), el = x % (D / 4) * 4, tr = 16 * ct + y;
            float top = s_m[0][tr];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) top = fmaxf(top, s_m[w][tr]);
            f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
            float ls = 0.f, le = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) sum += *reinterpret_cast<const f32x4_t*>(&s_o[w][y][el]);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float v = s_m[w][tr] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(s_m[w][tr] - top);
                ls += s_l[w][tr].x * v;
                le += s_l[w][tr].y * v;
            }
            if (whole) {
                const int r = t.row0 + tr, i = r / t.g;
                const int64_t to = (int64_t)(t.q0 + i) * p.d.h_q + kvh * t.g + r - i * t.g;
                sum *= ls > 0.f ? 1.f / ls : (ls == ls ? 0.f : ls);
                T* out = static_cast<T*>(p.out) + to * D + el;
                if constexpr (BF) *reinterpret_cast<u32x2_t*>(out) = u32x2_t{pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
                else *reinterpret_cast<f32x4_t*>(out) = sum;
                if (p.lse && el == 0) p.lse[to] = le > 0.f ? (top + __builtin_amdgcn_logf(le)) * kLn2 : (le == le ? -INFINITY : le);
            } else {
                const int64_t to = part.at + tr;
                *reinterpret_cast<f32x4_t*>(a.part_o + to * D + el) = sum;
                if (el == 0) a.part_ml[to] = make_float4(top, ls, le, 0.f);
            }
        }
    }
}

// Joins the ranges of one row of a tile, 64 elements of it: the ranges' sums weighted by
// exp2(m - max m). 16 lanes hold the elements, the blockDim / 16 groups of them take the ranges in
// turn; the order of the additions depends on the sizes only.
constexpr int kJoinGroups = 64;  // at most

int join_threads(int64_t ranges)
{
    const int64_t t = (ranges + 3) / 4 * 16;  // about four ranges a group
    return t < 64 ? 64 : t > 16 * kJoinGroups ? 16 * kJoinGroups : (int)((t + 63) / 64 * 64);
}

template <typename T, int D, int M>
__global__ void __launch_bounds__(16 * kJoinGroups) extend_join_kernel(ExtendArgs a)
{
    __shared__ f32x4_t s_o[kJoinGroups][16];
    __shared__ float2 s_l[kJoinGroups];
    __shared__ float s_m[kJoinGroups / 4];
    const ExtendCall& p = a.c;
    const uint32_t units = (uint32_t)a.slots * (uint32_t)p.c.h_kv;
    const int groups = blockDim.x / 16;
    const int64_t tr64 = (int64_t)block_index() / (D / 64);
    const int64_t unit = tr64 / M;
    const int tr = (int)(tr64 - unit * M);
    if (unit >= units) return;  // past the grid's end
    Part part;
    if (!find_parts<M>(a, (uint32_t)unit, &part)) return;
    const Span& t = part.t;
    const int kvh = t.head, used = part.rg;
    if (t.row0 + tr >= t.rows) return;
    const int64_t step = part.step;
    const float4* ml = a.part_ml + part.at + tr;
    const int y = threadIdx.x / 16, el = (int)(block_index() % (D / 64)) * 64 + threadIdx.x % 16 * 4;
    const float* po = a.part_o + (part.at + tr) * D + el;

    float top = -INFINITY;
    for (int x = threadIdx.x; x < used; x += blockDim.x) top = fmaxf(top, ml[x * step].x);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    if (threadIdx.x % 64 == 0) s_m[threadIdx.x / 64] = top;
    __syncthreads();
    for (int x = 0; x < (int)blockDim.x / 64; ++x) top = fmaxf(top, s_m[x]);

    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    float ls = 0.f, le = 0.f;
#pragma unroll 4
    for (int x = y; x < used; x += groups) {
        const float4 v = ml[x * step];
        const f32x4_t sums = *reinterpret_cast<const f32x4_t*>(po + x * step * D);
        const float f = v.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(v.x - top);
        ls += v.y * f;
        le += v.z * f;
        sum += sums * f;
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
    const int r = t.row0 + tr, i = r / t.g;
    const int64_t to = (int64_t)(t.q0 + i) * p.d.h_q + kvh * t.g + r - i * t.g;
    T* out = static_cast<T*>(p.out) + to * D + el;
    if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2_t*>(out) = u32x2_t{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    else *reinterpret_cast<f32x4_t*>(out) = o;
    if (p.lse && el == 0) p.lse[to] = e > 0.f ? (top + __builtin_amdgcn_logf(e)) * kLn2 : (e == e ? -INFINITY : e);
}

// The same for few ranges of many rows: D / 4 lanes hold a row, first a range each for the weights, then four
// elements each of the weighted sum.
constexpr int kFewRanges = 16;

template <typename T, int D, int M>
__global__ void __launch_bounds__(256) extend_join_rows_kernel(ExtendArgs a)
{
    constexpr int LANES = D / 4, ROWS = 256 / LANES;
    static_assert(M % ROWS == 0 && LANES >= kFewRanges, "a tile is whole workgroups, a range has a lane");
    __shared__ float s_w[ROWS][kFewRanges];
    const ExtendCall& p = a.c;
    const uint32_t unit = block_index() / (M / ROWS);
    const int tr = (int)(block_index() % (M / ROWS)) * ROWS + threadIdx.x / LANES, lane = threadIdx.x % LANES;
    if (unit >= (uint32_t)a.slots * (uint32_t)p.c.h_kv) return;  // past the grid's end
    Part part;
    if (!find_parts<M>(a, unit, &part)) return;
    const Span& t = part.t;
    const int r = t.row0 + tr, used = part.rg;
    const int64_t at = part.at + tr, step = part.step;
    const float* from = a.part_o + at * D + lane * 4;
    const bool there = r < t.rows;
    float top = -INFINITY;
    for (int x = lane; x < used; x += LANES)
        if (there) top = fmaxf(top, a.part_ml[at + x * step].x);
#pragma unroll
    for (int off = LANES / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, LANES));
    float l = 0.f, e = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int x0 = 0; x0 < used; x0 += kFewRanges) {
        const int some = used - x0 < kFewRanges ? used - x0 : kFewRanges;
        if (lane < kFewRanges) {
            const float4 ml = lane < some && there ? a.part_ml[at + (x0 + lane) * step] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
            const float w = ml.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
            l += ml.y * w;
            e += ml.z * w;
            s_w[threadIdx.x / LANES][lane] = w;
        }
        __syncthreads();
        if (there)
#pragma unroll 8
            for (int x = 0; x < some; ++x)
                o += *reinterpret_cast<const f32x4_t*>(from + (x0 + x) * step * D) * s_w[threadIdx.x / LANES][x];
        __syncthreads();
    }
#pragma unroll
    for (int off = kFewRanges / 2; off >= 1; off >>= 1) {
        l += __shfl_xor(l, off, LANES);
        e += __shfl_xor(e, off, LANES);
    }
    l = __shfl(l, 0, LANES);
    if (!there) return;
    o *= l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    const int i = (int)((uint32_t)r / (uint32_t)t.g);
    const int64_t to = (t.q0 + i) * p.d.h_q + t.head * t.g + r - i * t.g;
    T* out = static_cast<T*>(p.out) + to * D + lane * 4;
    if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2_t*>(out) = u32x2_t{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    else *reinterpret_cast<f32x4_t*>(out) = o;
    if (p.lse && lane == 0) p.lse[to] = e > 0.f ? (top + __builtin_amdgcn_logf(e)) * kLn2 : (e == e ? -INFINITY : e);
}

template <typename T, int D, int M>
hipError_t launch_join(const ExtendArgs& a)
{
    const int64_t units = (int64_t)a.slots * a.c.c.h_kv;
    if (a.ranges <= kFewRanges) {  // (or about so many)
        hipLaunchKernelGGL((extend_join_rows_kernel<T, D, M>), grid_of(units * (M * D / 1024)), dim3(256), 0, a.c.stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((extend_join_kernel<T, D, M>), grid_of(units * M * (D / 64)), dim3(join_threads(a.ranges)), 0,
                       a.c.stream, a);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_join_m(const ExtendArgs& a, int m)
{
    switch (m) {
        case 16: return launch_join<T, D, 16>(a);
        case 32: return launch_join<T, D, 32>(a);
        case 64: return launch_join<T, D, 64>(a);
        case 128: return launch_join<T, D, 128>(a);
        case 256: return launch_join<T, D, 256>(a);
        default: return hipErrorInvalidValue;
    }
}

template <typename T>
hipError_t launch_join_d(const ExtendArgs& a, int m)
{
    switch (a.c.c.d) {
        case 64: return launch_join_m<T, 64>(a, m);
        case 128: return launch_join_m<T, 128>(a, m);
        case 256: return launch_join_m<T, 256>(a, m);
        default: return hipErrorInvalidValue;
    }
}

template <typename T, bool FP8, int D, int CT>
hipError_t launch_ct(const ExtendCall& c, const ExtendPlan& pl, void* ws)
{
    const ExtendArgs a = extend_args(c, pl, ws);
    hipLaunchKernelGGL((extend_kernel<T, FP8, D, CT>), grid_of(pl.workgroups()), dim3(64 * kWaves), 0, c.stream, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || pl.ranges == 1 ? e : launch_extend_join(a, pl.m);
}

template <typename T, bool FP8, int D>
hipError_t launch_t(const ExtendCall& c, const ExtendPlan& pl, void* ws)
{
    switch (pl.m) {
        case 16: return launch_ct<T, FP8, D, 1>(c, pl, ws);
        case 32: return launch_ct<T, FP8, D, 2>(c, pl, ws);
        default:
            if constexpr (D < 256) return launch_ct<T, FP8, D, 4>(c, pl, ws);
            else return hipErrorInvalidValue;
    }
}

template <typename T, int D>
hipError_t launch_store(const ExtendCall& c, const ExtendPlan& pl, void* ws)
{
    return c.c.store == GDN_FP8 ? launch_t<T, true, D>(c, pl, ws) : launch_t<T, false, D>(c, pl, ws);
}

template <typename T>
hipError_t launch_d(const ExtendCall& c, const ExtendPlan& pl, void* ws)
{
    switch (c.c.d) {
        case 64: return launch_store<T, 64>(c, pl, ws);
        case 128: return launch_store<T, 128>(c, pl, ws);
        case 256: return launch_store<T, 256>(c, pl, ws);
        default: return hipErrorInvalidValue;
    }
}

// Rows of a KV head up to which a sequence is taken by the kernel of this file; longer ones by the tiles of
// gdn_attn_extend_tile.hip, where the call is not small (narrow_tiles).
constexpr int kStreamRows = 64;

// Whether tiles are of 16 rows. Larger ones read the keys less often, but the ones of extend_kernel take up to 512
// registers, with one wave a SIMD whose every step waits for its loads, and the ones of gdn_attn_extend_tile.hip start and
// end slowly (15 to 20 us); tiles of 16 rows have two waves a SIMD, and the ones of a sequence share what they read in
// an L2 (pair_of). They win while what they ask for, the keys of every tile, stays below some 200 MB (fp32: 512, and
// 2048 of more than 64 rows, whose tiles are slowest), in up to 768 tiles, and for fp8 pages with d = 256, up to 64 rows. Measured
// (us, 16 / larger; MB). Up to 64 rows: d = 256, 16/2 heads 8 tokens after 4000 (33) 18 / 23, 16000 (134) 25 / 27, 32760 (268) 36 / 34,
// 8 sequences of 8 after up to 8192 (537) 43 / 37, 32 of 4 (1074) 110 / 74; fp8 8 after 32760 (134) 29 / 32, 32 of 4 to 8
// (537) 72 / 81, 64 of 8 after up to 16000 (2100) 296 / 352; d = 128, 32/8 heads 16 after 4000, fp8 (34) 18 / 25, 8 of 8 after up to
// 8192 (537) 46 / 41, 16 of 8, fp8 (537) 75 / 53; fp32, d = 256 8 after 4000 (67) 29 / 41, 8 of 4 after up to 8192 (537) 60 / 62. More rows:
// d = 256 16 after 4000 (67) 20 / 40, 128 after 1000 (151) 26 / 40, 256 after 1000 (336) 35 / 43, fp8 64 after 2000 (71) 24 / 66, 512 from the
// start (134) 18 / 43; d = 128 32 after 2000 (71) 18 / 25, 256 after 1000 (168) 30 / 30, 512 from the start (268) 22 / 18, 4 sequences of 20 to 200
// after up to 500 28 / 20, 16 of 60 from the start (126, 1920 tiles) 21 / 17, d = 256
// 64 of 10 to 20 after up to 100 (134, about 1000) 34 / 25; d = 64 16/16 heads 512 from the start (67) 11 / 14; fp32, d =
// 256 128 after 1000 (302) 50 / 225, 4000 (1110) 125 / 228, d = 128, 8/2 heads 64 after 4000 (138) 28 / 110, 16/2 heads 256 after 3000
// (1680) 93 / 114.
bool narrow_tiles(const gdn_kv_cache& c, const gdn_extend_dims& d, int64_t rows)
{
    const int64_t g = d.h_q / c.h_kv, each = (rows + 15) / 16, sparse = d.total_q * g / 16 + c.n;
    const int64_t tiles = (each <= sparse / c.n ? c.n * each : sparse) * c.h_kv;
    const int64_t step_bytes = (int64_t)kRange * 2 * c.d * (c.store == GDN_FP8 ? 1 : c.store == GDN_F32 ? 4 : 2);
    const int64_t steps = (extend_longest(c, d, 16) + kRange - 1) / kRange;
    if (c.n > 64) return false;  // more than Shares takes: a sequence's tiles would lie apart; no measured crossing
    if (rows <= 64 && c.d == 256 && c.store == GDN_FP8 && d.dtype == GDN_BF16) return true;
    const int64_t most = c.store != GDN_F32 ? 192 : rows <= 64 ? 512 : 2048;
    return tiles <= 768 && tiles * steps <= (most << 20) / step_bytes;
}

// How the sequences of up to `to` rows are taken.
ExtendPlan stream_plan(const gdn_kv_cache& c, const gdn_extend_dims& d, int64_t to)
{
    ExtendPlan p;
    const int64_t g = d.h_q / c.h_kv, most = d.max_q * g, rows = most < to ? most : to;
    const bool narrow = narrow_tiles(c, d, rows);
    p.m = rows <= 16 || narrow ? 16 : rows <= 32 || c.d == 256 ? 32 : 64;
    const int64_t packed = d.total_q * g / p.m + c.n, each = (rows + p.m - 1) / p.m;
    p.per_seq = each <= packed / c.n ? (int)each : 0;
    p.slots = p.per_seq ? c.n * each : packed;
    p.units = p.slots * c.h_kv;
    p.rows_from = 0;
    p.rows_to = (int)rows;
    const int64_t tiles = (d.total_q * g + p.m - 1) / p.m;
    const int64_t likely = tiles < p.slots ? tiles : p.slots, real = (likely > c.n ? likely : c.n) * c.h_kv;
    const int64_t len = extend_longest(c, d, p.m), steps = len > 0 ? (len + kRange - 1) / kRange : 1;
    // As many parts as fill the chip once: `fill` workgroups run at a time, and late ones cost a round. Where the
    // tiles alone do, parts of about eight steps, so that late ones fill the CUs that are done. Measured
    // (us, workgroups 256 / 512 / 640): 32 sequences behind a window of 4096, d = 256, 16/2 heads 59 / 69 / -; 24 of up to 8000, fp8,
    // d = 256 45 / 36 / -; 16 of 4 tokens after up to 8192, d = 128, 32/8 83 / 72 / 76; 8 of 16 tokens (64 rows) 57 / 67 / -. Up to
    // four steps stay together, which spares the second launch.
    // Up to 64 sequences are divided by their lengths, on the GPU, instead of by max_len (us, by max_len / by
    // lengths; all drawn up to the bound): 16 of 4 tokens as above 82 / 72, 64 of one token, up to 8192, d = 128, 32/8
    // heads 234 / 212, 40 of them 160 / 143, 32 behind a window 59 / 59. More than 64, which have no lane each, are
    // divided by max_len or not at all: 64 of one token after up to 16000, d = 256, 16/2 heads take 214, 65 take 438.
    const int64_t fill = (c.d == 256 && !(c.store == GDN_FP8 && p.m == 16)) || p.m == 64 ? 256 : 512;
    int64_t ranges = real >= fill ? (real * steps / 8 < 4096 ? real * steps / 8 : 4096) / real : fill / real;
    if (ranges > (steps + 1) / 2) ranges = (steps + 1) / 2;
    if (c.n > 1 && c.n <= 64 && real < fill && steps >= 16 && ranges < 2) ranges = 2;
    if (steps <= 4) ranges = 1;
    if (ranges > 0x7fffffff / p.units) ranges = 0x7fffffff / p.units;  // the grid
    if (ranges < 1) ranges = 1;
    const int64_t per = (steps + ranges - 1) / ranges;
    p.range = per * kRange;
    p.ranges = (steps + per - 1) / per;
    p.share = p.packed = 0;
    p.least = real >= fill ? 8 : 2;
    // Shares are found by lanes, one a sequence, with sums of 32 bits. One sequence is divided by its bound,
    // which spares 0.6 us of looking.
    if (c.n > 1 && c.n <= 64 && p.ranges > 1 && c.n * (d.total_q * g / p.m + 1) * c.h_kv < (1 << 30) / (steps + 1))
        p.share = real >= fill ? real * (p.ranges + 1) : fill;
    return p;
}

struct Plans {
    ExtendPlan stream, tiles;
    size_t stream_bytes;  // the tiles' workspace follows
};

// A tile of 128 rows with a few in use asks for bf16 pages at 7.8 TB/s (128 flops a byte at 1 PFLOP/s), more than
// memory gives, so that short sequences beside long ones are best left to the tiles, one launch: 24
// sequences of 1 to 700 tokens, of which few are short, 398 us and 72 + 5 less. fp8 and fp32 pages, a
// quarter and a third of that, are taken by the kernel of this file.
Plans make_plans(const gdn_kv_cache& c, const gdn_extend_dims& d)
{
    const int64_t most = d.max_q * (d.h_q / c.h_kv);
    const bool only_stream = most <= kStreamRows || narrow_tiles(c, d, most) || (d.dtype == GDN_F32 && c.store == GDN_FP8);
    const bool both = !only_stream && c.n > 1 && c.store != GDN_BF16;
    Plans p;
    p.stream.m = p.tiles.m = 0;
    if (only_stream || both) p.stream = stream_plan(c, d, only_stream ? most : kStreamRows);
    if (!only_stream) {
        p.tiles = extend_tile_plan(c, d);
        p.tiles.rows_from = both ? kStreamRows + 1 : 0;
        p.tiles.rows_to = 0x7fffffff;
    }
    p.stream_bytes = p.stream.workspace(c);
    return p;
}

}  // namespace

hipError_t launch_extend_join(const ExtendArgs& a, int m)
{
    return a.c.d.dtype == GDN_BF16 ? launch_join_d<uint16_t>(a, m) : launch_join_d<float>(a, m);
}

size_t attn_extend_workspace(const gdn_kv_cache& c, const gdn_extend_dims& d)
{
    const Plans p = make_plans(c, d);
    return p.stream_bytes + p.tiles.workspace(c);
}

hipError_t launch_attn_extend(const ExtendCall& c)
{
    const Plans p = make_plans(c.c, c.d);
    hipError_t e = hipSuccess;
    if (p.stream.m) e = c.d.dtype == GDN_BF16 ? launch_d<uint16_t>(c, p.stream, c.ws) : launch_d<float>(c, p.stream, c.ws);
    if (e == hipSuccess && p.tiles.m) e = launch_extend_tiles(c, p.tiles, static_cast<char*>(c.ws) + p.stream_bytes);
    return e;
}

}  // namespace gdn
