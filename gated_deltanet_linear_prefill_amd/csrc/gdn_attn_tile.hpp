// gdn_attn_tile.hpp -- the step of attention that the prefill kernels share: 32 query rows of a wave over
// keys that lie in LDS, and how rows are written (not part of the C ABI). The matrix form is
// described in gdn_attn_prefill.hip.
#pragma once

#include <type_traits>

#include "gdn_attn_internal.hpp"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int clamp_to(int x, int hi)
{
    return x < 0 ? 0 : (x > hi ? hi : x);
}

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
// Call: out, lse and d.h_q; Work: the sequence's q0, rows, g and head.
template <typename T, int D, typename Call, typename Work>
__device__ __forceinline__ void write_rows(const Call& p, const Work& w, int first, int lane,
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

// What a row sees of a packed sequence: the keys below lim (which may be negative, or above N).
struct SeesBelow {
    static constexpr bool RARE = false;
    int lim;
    __device__ __forceinline__ bool operator()(int key) const { return key < lim; }
};

// One step of a wave's 32 rows over N staged keys at sk, sv (klane, vlane: this lane's offsets).
// This lane's row sees the keys of [0, N) for which sees(key) holds; or, with RARE and where it is so that
// rare(), those for which rarely(key) does.
template <typename T, int D, bool LSE, int MODE, typename Sees>
__device__ __forceinline__ void attn_step(const char* sk, const char* sv, int klane, int vlane,
                                          const u32x4_t (&q)[D / (32 / sizeof(T))], f32x16_t (&o)[D / 32],
                                          Stats& st, float c, bool masked, Sees sees, int lane, bool& odd)
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
        if constexpr (Sees::RARE) {
            // made here and not before the branch, for every step
            asm volatile("" : "+v"(sees.lo));
            if (sees.rare()) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[b][i] = sees.rarely(C::ROWS * (group_of(i) + 4 * half) + place_of(b, i)) ? s[b][i] : -INFINITY;
            } else {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[b][i] = sees(C::ROWS * (group_of(i) + 4 * half) + place_of(b, i)) ? s[b][i] : -INFINITY;
            }
        } else {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[b][i] = sees(C::ROWS * (group_of(i) + 4 * half) + place_of(b, i)) ? s[b][i] : -INFINITY;
        }
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
            bool seen;
            if constexpr (Sees::RARE) seen = sees.rare() ? sees.rarely(key) : sees(key);
            else seen = sees(key);
#pragma unroll
            for (int db = 0; db < ND; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = load1_f32(reinterpret_cast<const T*>(at) + 32 * db + 8 * (i / 4) + i % 4);
                    o[db][i] += seen && !is_finite(x) ? x : 0.f;
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

}  // namespace
}  // namespace gdn
