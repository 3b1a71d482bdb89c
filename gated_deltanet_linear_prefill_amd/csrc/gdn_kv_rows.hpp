// gdn_kv_rows.hpp -- device pieces shared by the kernels that write and read cache rows: where a packed
// row lives, 16 bytes of a row, and the fp8 store's quantisation (not part of the C ABI).
#pragma once

#include "gdn_attn_internal.hpp"

namespace gdn {

// Where a packed row lives: its (page, slot) as a row index of the pools, or -1; *mine: it belongs to
// a sequence, and *at is then its position there. `first` is the token of the wave's first lane.
// Call: KvCall or another with its c, start and cu.
template <typename Call>
__device__ __forceinline__ int64_t pool_row(const Call& p, int64_t token, int first, int h, int page_shift,
                                            bool* mine, int64_t* at)
{
    const gdn_kv_cache& c = p.c;
    int64_t seq = token, i = 0;
    *mine = true;
    if (p.cu) {
        int end;
        seq = find_seq(p.cu, (int)c.n, first, (int)token, &end);
        i = token - p.cu[seq];
        *mine = i >= 0 && token < end;
        if (!*mine) return -1;
    }
    const int64_t pos = (int64_t)p.start[seq] + i;
    *at = pos;
    if (pos < 0 || pos >= c.max_pages << page_shift) return -1;
    const int64_t page = c.page_table[seq * c.max_pages + (pos >> page_shift)];
    if (page < 0 || page >= c.num_pages) return -1;
    return ((page * c.h_kv + h) << page_shift) + (pos & (c.page_size - 1));
}

// 16 bytes of T: E elements.
template <typename T>
struct Some {
    static constexpr int E = 16 / (int)sizeof(T);
    u32x4_t x;
    __device__ __forceinline__ void load(const T* p) { x = *reinterpret_cast<const u32x4_t*>(p); }
    // What is stored is not read again soon, and the lanes of a store cover whole lines.
    __device__ __forceinline__ void store(T* p) const { __builtin_nontemporal_store(x, reinterpret_cast<u32x4_t*>(p)); }
    __device__ __forceinline__ void get(float* f) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                f[2 * i] = __uint_as_float(x[i] << 16);
                f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
            } else {
                f[i] = __uint_as_float(x[i]);
            }
        }
    }
    __device__ __forceinline__ void set(const float* f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = sizeof(T) == 2 ? pack_bf16(f[2 * i], f[2 * i + 1]) : __float_as_uint(f[i]);
    }
};

// E codes of a lane.
template <int E>
struct Codes;
template <> struct Codes<4> { typedef uint32_t type; };
template <> struct Codes<8> { typedef u32x2_t type; };
template <> struct Codes<16> { typedef u32x4_t type; };

template <typename W>
__device__ __forceinline__ uint32_t word_of(const W& w, int i)
{
    if constexpr (sizeof(W) == 4) return w;
    else return w[i];
}

// Codes and scale byte of a row held by LPR lanes. Not-finite elements take no part in the
// scale and become NaN codes.
template <int E, int LPR>
__device__ __forceinline__ typename Codes<E>::type quantise(const float* f, uint32_t* scale)
{
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float a = fabsf(f[i]);
        top = a <= 3.4028234e38f ? fmaxf(top, a) : top;  // false for NaN and infinity
    }
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    const uint32_t bits = __float_as_uint(top);
    // exponent - 8, one more when the mantissa is above 1.75; a subnormal top has exponent 0
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = bits == 0 ? 0 : max(e, -126);
    *scale = (uint32_t)(e + 127);
    const float r = exp2_int(-e);
    float y[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float a = f[i] * r;
        y[i] = fabsf(a) <= 448.f ? a : __uint_as_float(0x7fc00000u);
    }
    typename Codes<E>::type code;
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], w, true);
        if constexpr (E == 4) code = (uint32_t)w;
        else code[i] = (uint32_t)w;
    }
    return code;
}

template <int E>
__device__ __forceinline__ void dequantise(typename Codes<E>::type code, uint32_t scale, float* f)
{
    const float s = scale_of(scale);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)word_of(code, i), false);
        const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)word_of(code, i), true);
        f[4 * i] = a[0] * s;
        f[4 * i + 1] = a[1] * s;
        f[4 * i + 2] = b[0] * s;
        f[4 * i + 3] = b[1] * s;
    }
}

}  // namespace gdn
