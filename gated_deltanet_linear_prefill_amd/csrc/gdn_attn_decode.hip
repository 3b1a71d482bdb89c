// gdn_attn_decode.hip -- attention of one new token per sequence over the paged cache.
//
// Bound by the bytes of the cache: every K and V row is read once per KV head, for all of its
// G = h_q / h_kv query heads (up to 16 at a time). One workgroup takes one (sequence, KV head)
// and one range of positions; its waves take 32-position steps of the range in turn, each with
// its own softmax state, and are joined in LDS. When the pairs alone would not fill the chip
// the positions are split over more workgroups (ranges), whose sums go to the workspace and
// are joined by a second kernel.
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

constexpr int kWaves = 4, kStep = 32;  // positions per wave and step
constexpr int kRange = kWaves * kStep; // ranges are multiples of this
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
    p.head_tiles = (h_q / c->h_kv + 15) / 16;
    const int64_t units = c->n * c->h_kv * p.head_tiles;
    const int64_t steps = len > 0 ? (len + kRange - 1) / kRange : 1;
    int64_t ranges = units > 0 ? (1024 + units - 1) / units : 1;
    if (ranges < (steps + 15) / 16) ranges = (steps + 15) / 16;
    if (units > 0 && ranges > 0x7fffffff / units) ranges = 0x7fffffff / units;  // one grid dimension
    if (ranges > steps) ranges = steps;
    const int64_t per = (steps + ranges - 1) / ranges;
    p.range = per * kRange;
    p.ranges = (steps + per - 1) / per;
    return p;
}

// Workspace of one call: O sums [unit][range][G][D] fp32, then (m, l) pairs.
struct Partials {
    float* o;
    float2* ml;
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

__device__ __forceinline__ uint32_t cvt_bf16_fp8(uint32_t w, bool hi)
{
    return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}

template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(64 * kWaves)
decode_attn_kernel(AttnDecodeCall p, int64_t range, int ranges, int head_tiles, int page_shift,
                   Partials part)
{
    using C = Cfg<T, FP8, D>;
    using VP = typename Piece<C::EPL * C::ES>::type;
    constexpr bool BF = sizeof(T) == 2;
    __shared__ float s_o[kWaves][16][D + 4];
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int rg = blockIdx.x % ranges;
    const int64_t unit = blockIdx.x / ranges;
    const int ht = (int)(unit % head_tiles);
    const int kvh = (int)(unit / head_tiles % p.c.h_kv);
    const int64_t seq = unit / head_tiles / p.c.h_kv;
    const int G = p.h_q / p.c.h_kv, heads = G - 16 * ht < 16 ? G - 16 * ht : 16;
    const int64_t cap = p.c.max_pages << page_shift;
    int64_t len = p.lens[seq];
    len = len < p.max_len ? len : p.max_len;
    len = len < cap ? len : cap;
    const int64_t begin = rg * range;
    if (ranges > 1 && begin >= len) return;  // the join does not read this range
    const int64_t end = begin + range < len ? begin + range : len;

    // Q as the B operand: column c is head 16 ht + c (heads past the group repeat the last)
    const int head = kvh * G + 16 * ht + (c < heads ? c : heads - 1);
    const T* qp = static_cast<const T*>(p.q) + seq * p.q_token + (int64_t)head * p.q_head;
    // element order of a K piece: load i brings elements (i * 4 + g) * EPK ..
    T q[D / 4];
#pragma unroll
    for (int i = 0; i < C::KL; ++i)
#pragma unroll
        for (int e = 0; e < C::EPK; e += 16 / (int)sizeof(T)) {
            const u32x4_t x = *reinterpret_cast<const u32x4_t*>(qp + (i * 4 + g) * C::EPK + e);
            __builtin_memcpy(q + i * C::EPK + e, &x, 16);
        }

    f32x4_t o[C::VL];
#pragma unroll
    for (int j = 0; j < C::VL; ++j) o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    const float cs = p.scale * kLog2e;
    const int32_t* table = p.c.page_table + seq * p.c.max_pages;
    const char* kpool = static_cast<const char*>(p.c.k);
    const char* vpool = static_cast<const char*>(p.c.v);

    for (int64_t j0 = begin + wave * kStep; j0 < end; j0 += kWaves * kStep) {
        float s[8];
        u32x4_t kx[2][C::KL];
        VP vx[8][C::U];
        uint32_t sk[2], sv[2];
        bool there[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int64_t pos = j0 + 16 * b;
            int64_t page = -1;
            if (pos < end) page = table[pos >> page_shift];
            there[b] = page >= 0 && page < p.c.num_pages;
            const int64_t row = ((page * p.c.h_kv + kvh) << page_shift) + (pos & (p.c.page_size - 1));
            if (there[b]) {
                const char* kr = kpool + (row + c) * (D * C::ES) + g * 16;
#pragma unroll
                for (int i = 0; i < C::KL; ++i) kx[b][i] = *reinterpret_cast<const u32x4_t*>(kr + i * 64);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const char* vr = vpool + (row + 4 * g + i) * (D * C::ES) + c * (C::EPL * C::ES);
#pragma unroll
                    for (int u = 0; u < C::U; ++u)
                        vx[4 * b + i][u] = *reinterpret_cast<const VP*>(vr + u * (16 * C::EPL * C::ES));
                }
                if constexpr (FP8) {
                    sk[b] = *reinterpret_cast<const uint32_t*>(p.c.k_scale + row + 4 * g);
                    sv[b] = *reinterpret_cast<const uint32_t*>(p.c.v_scale + row + 4 * g);
                }
            } else {
                sk[b] = sv[b] = 0;
#pragma unroll
                for (int i = 0; i < C::KL; ++i) kx[b][i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int u = 0; u < C::U; ++u) vx[4 * b + i][u] = VP{};
            }
        }

        // scores
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < C::KL; ++i) {
                if constexpr (BF && !FP8) {
                    bf16x8_t qq;
                    __builtin_memcpy(&qq, q + i * 8, 16);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, kx[b][i]), qq, acc, 0, 0, 0);
                } else if constexpr (BF) {
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        bf16x8_t qq;
                        __builtin_memcpy(&qq, q + i * 16 + f * 8, 16);
                        const u32x4_t a = {cvt_bf16_fp8(kx[b][i][2 * f], false), cvt_bf16_fp8(kx[b][i][2 * f], true),
                                           cvt_bf16_fp8(kx[b][i][2 * f + 1], false), cvt_bf16_fp8(kx[b][i][2 * f + 1], true)};
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), qq, acc, 0, 0, 0);
                    }
                } else if constexpr (!FP8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kx[b][i][e]), q[i * 4 + e], acc, 0, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const f32x2_t a = e & 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)kx[b][i][e / 4], true)
                                                : __builtin_amdgcn_cvt_pk_f32_fp8((int)kx[b][i][e / 4], false);
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[0], q[i * 16 + e], acc, 0, 0, 0);
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[1], q[i * 16 + e + 1], acc, 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = acc[i] * cs;
                if constexpr (FP8) x *= scale_of((sk[b] >> (8 * i)) & 0xff);
                const bool seen = there[b] && j0 + 16 * b + 4 * g + i < end;
                s[4 * b + i] = seen ? x : -INFINITY;
                // what lies behind the last position is anything: not into the product
                if (!seen) {
#pragma unroll
                    for (int u = 0; u < C::U; ++u) vx[4 * b + i][u] = VP{};
                    if constexpr (FP8) sv[b] &= ~(0xffu << (8 * i));
                }
            }
        }

        // softmax
        float mx = s[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        if (__any(mx > m)) {
            const float mn = fmaxf(m, mx);
            const float a = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= a;
#pragma unroll
            for (int j = 0; j < C::VL; ++j) o[j] *= a;
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = __builtin_amdgcn_exp2f(s[i] - ref);
            l += s[i];
            if constexpr (FP8) s[i] *= scale_of((sv[i / 4] >> (8 * (i % 4))) & 0xff);
        }

        // O^T += V^T P^T; o[u * EPL + j] rows are elements 16 EPL u + EPL (4 g + i) + j
        if constexpr (BF) {
            const u32x4_t pw = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7])};
            const bf16x8_t pb = __builtin_bit_cast(bf16x8_t, pw);
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
                        o[u * C::EPL + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), pb, o[u * C::EPL + j], 0, 0, 0);
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
                        o[u * C::EPL + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a0), pb, o[u * C::EPL + j], 0, 0, 0);
                        o[u * C::EPL + j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a1), pb, o[u * C::EPL + j + 1], 0, 0, 0);
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
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
    }

    // join the waves
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (g == 0) {
        s_m[wave][c] = m;
        s_l[wave][c] = l;
    }
    __syncthreads();
    float mm = s_m[0][c];
#pragma unroll
    for (int x = 1; x < kWaves; ++x) mm = fmaxf(mm, s_m[x][c]);
    const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mm);
#pragma unroll
    for (int u = 0; u < C::U; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < C::EPL; ++j)
                s_o[wave][c][16 * C::EPL * u + C::EPL * (4 * g + i) + j] = m == -INFINITY ? 0.f : o[u * C::EPL + j][i] * f;
    __syncthreads();
    for (int x = threadIdx.x; x < heads * (D / 4); x += 64 * kWaves) {
        const int hd = x / (D / 4), el = x % (D / 4) * 4;
        float top = s_m[0][hd];
#pragma unroll
        for (int y = 1; y < kWaves; ++y) top = fmaxf(top, s_m[y][hd]);
        f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
        float ls = 0.f;
#pragma unroll
        for (int y = 0; y < kWaves; ++y) {
            sum += *reinterpret_cast<const f32x4_t*>(&s_o[y][hd][el]);
            if (s_m[y][hd] != -INFINITY) ls += s_l[y][hd] * __builtin_amdgcn_exp2f(s_m[y][hd] - top);
        }
        if (ranges == 1) {
            const int64_t row = seq * p.h_q + kvh * G + 16 * ht + hd;
            const float inv = ls > 0.f ? 1.f / ls : (ls == ls ? 0.f : ls);
            sum *= inv;
            T* out = static_cast<T*>(p.out) + row * D + el;
            if constexpr (BF) *reinterpret_cast<u32x2_t*>(out) = u32x2_t{pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
            else *reinterpret_cast<f32x4_t*>(out) = sum;
            if (p.lse && el == 0) p.lse[row] = ls > 0.f ? (top + __builtin_amdgcn_logf(ls)) * kLn2 : (ls == ls ? -INFINITY : ls);
        } else {
            const int64_t at = (unit * ranges + rg) * 16 + hd;
            *reinterpret_cast<f32x4_t*>(part.o + at * D + el) = sum;
            if (el == 0) part.ml[at] = make_float2(top, ls);
        }
    }
}

// Joins the ranges of one (sequence, head): the rows' sums weighted by exp2(m - max m).
template <typename T, int D>
__global__ void __launch_bounds__(256) decode_join_kernel(AttnDecodeCall p, int64_t range, int ranges,
                                                          int head_tiles, int page_shift, Partials part)
{
    constexpr int TPR = D / 4, RPB = 256 / TPR;  // threads per row, ranges at a time
    __shared__ f32x4_t s_o[RPB][TPR];
    __shared__ float s_l[RPB];
    const int64_t seq = blockIdx.x / p.h_q;
    const int hq = (int)(blockIdx.x - seq * p.h_q);
    const int G = p.h_q / p.c.h_kv, kvh = hq / G, hg = hq - kvh * G, ht = hg / 16, hd = hg % 16;
    const int64_t cap = p.c.max_pages << page_shift;
    int64_t len = p.lens[seq];
    len = len < p.max_len ? len : p.max_len;
    len = len < cap ? len : cap;
    const int used = len <= 0 ? 0 : (int)((len + range - 1) / range);
    const int64_t unit = (seq * p.c.h_kv + kvh) * head_tiles + ht;
    const float2* ml = part.ml + unit * ranges * 16 + hd;
    const float* po = part.o + (unit * ranges * 16 + hd) * D;

    const int lane = threadIdx.x & 63;
    float top = -INFINITY;
    for (int x = lane; x < used; x += 64) top = fmaxf(top, ml[(int64_t)x * 16].x);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));

    const int y = threadIdx.x / TPR, el = threadIdx.x % TPR * 4;
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    float ls = 0.f;
    for (int x = y; x < used; x += RPB) {
        const float2 v = ml[(int64_t)x * 16];
        if (v.x == -INFINITY) continue;
        const float f = __builtin_amdgcn_exp2f(v.x - top);
        ls += v.y * f;
        sum += *reinterpret_cast<const f32x4_t*>(po + (int64_t)x * 16 * D + el) * f;
    }
    s_o[y][el / 4] = sum;
    if (el == 0) s_l[y] = ls;
    __syncthreads();
    if (y != 0) return;
    float l = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < RPB; ++x) {
        o += s_o[x][el / 4];
        l += s_l[x];
    }
    const int64_t row = seq * p.h_q + hq;
    o *= l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    T* out = static_cast<T*>(p.out) + row * D + el;
    if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2_t*>(out) = u32x2_t{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    else *reinterpret_cast<f32x4_t*>(out) = o;
    if (p.lse && el == 0) p.lse[row] = l > 0.f ? (top + __builtin_amdgcn_logf(l)) * kLn2 : (l == l ? -INFINITY : l);
}

template <typename T, bool FP8, int D>
hipError_t launch_t(const AttnDecodeCall& c)
{
    const Plan pl = make_plan(&c.c, c.h_q, c.max_len);
    const int64_t units = c.c.n * c.c.h_kv * pl.head_tiles;
    const int shift = __builtin_ctz((unsigned)c.c.page_size);
    Partials part;
    part.o = static_cast<float*>(c.ws);
    part.ml = reinterpret_cast<float2*>(part.o + units * pl.ranges * 16 * D);
    hipLaunchKernelGGL((decode_attn_kernel<T, FP8, D>), dim3((unsigned)(units * pl.ranges)), dim3(64 * kWaves), 0,
                       c.stream, c, pl.range, (int)pl.ranges, pl.head_tiles, shift, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || pl.ranges == 1) return e;
    hipLaunchKernelGGL((decode_join_kernel<T, D>), dim3((unsigned)(c.c.n * c.h_q)), dim3(256), 0, c.stream, c,
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
    return (size_t)(c->n * c->h_kv * pl.head_tiles * pl.ranges) * 16 * (c->d * sizeof(float) + sizeof(float2));
}

hipError_t launch_attn_decode(const AttnDecodeCall& c)
{
    return c.dtype == GDN_BF16 ? launch_d<uint16_t>(c) : launch_d<float>(c);
}

}  // namespace gdn
