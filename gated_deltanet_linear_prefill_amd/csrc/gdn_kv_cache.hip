// gdn_kv_cache.hip -- the paged key-value cache: rows written (quantised as they are written)
// and read back.
//
// A row is the d elements of one (token, KV head). D/8 adjacent lanes hold a row, eight
// elements each, of K and of V: 16-byte loads and stores for bf16, and with an fp8 store the
// row's largest magnitude is a few cross-lane maxima away. Both kernels only move bytes.
//
// fp8 store: with a = max |x| = m 2^x (1 <= m < 2), the scale 2^e with e = x - 8 + (m > 1.75)
// is the smallest power of two with a / 2^e <= 448 = 1.75 * 2^8. It comes from a's bits, and
// multiplying by 2^-e is exact, so each element is rounded once (to nearest even, by the
// conversion to e4m3).
#include "gdn_attn_internal.hpp"

namespace gdn {
namespace {

// Where a packed row lives: its (page, slot) as a row index of the pools, or -1.
template <typename TCu>
__device__ __forceinline__ int64_t pool_row(const gdn_kv_cache& c, const TCu* start, const TCu* cu,
                                            int64_t token, int h, int page_shift, bool* mine)
{
    int64_t seq = token, i = 0;
    *mine = true;
    if (cu) {
        seq = find_seq(cu, c.n, token);
        i = token - cu[seq];
        *mine = i >= 0 && token < cu[seq + 1];
        if (!*mine) return -1;
    }
    const int64_t pos = (int64_t)start[seq] + i;
    if (pos < 0 || pos >= c.max_pages << page_shift) return -1;
    const int64_t page = c.page_table[seq * c.max_pages + (pos >> page_shift)];
    if (page < 0 || page >= c.num_pages) return -1;
    return ((page * c.h_kv + h) << page_shift) + (pos & (c.page_size - 1));
}

// Eight elements as loaded: bf16 in 16 bytes, fp32 in 32.
template <typename T>
struct Eight;

template <>
struct Eight<uint16_t> {
    u32x4_t x;
    __device__ __forceinline__ void load(const uint16_t* p) { x = *reinterpret_cast<const u32x4_t*>(p); }
    __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<u32x4_t*>(p) = x; }
    __device__ __forceinline__ void get(float* f) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(x[i] << 16);
            f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float* f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    }
};

template <>
struct Eight<float> {
    f32x4_t a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = *reinterpret_cast<const f32x4_t*>(p);
        b = *reinterpret_cast<const f32x4_t*>(p + 4);
    }
    __device__ __forceinline__ void store(float* p) const
    {
        *reinterpret_cast<f32x4_t*>(p) = a;
        *reinterpret_cast<f32x4_t*>(p + 4) = b;
    }
    __device__ __forceinline__ void get(float* f) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[i] = a[i]; f[4 + i] = b[i]; }
    }
    __device__ __forceinline__ void set(const float* f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) { a[i] = f[i]; b[i] = f[4 + i]; }
    }
};

// Codes and scale byte of a row held by LPR lanes. Not-finite elements take no part in the
// scale and become NaN codes.
template <int LPR>
__device__ __forceinline__ u32x2_t quantise(const float* f, uint32_t* scale)
{
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
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
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = f[i] * r;
        y[i] = fabsf(a) <= 448.f ? a : __uint_as_float(0x7fc00000u);
    }
    u32x2_t code;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
        code[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], w, true);
    }
    return code;
}

__device__ __forceinline__ void dequantise(u32x2_t code, uint32_t scale, float* f)
{
    const float s = scale_of(scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[i], false);
        const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)code[i], true);
        f[4 * i] = a[0] * s;
        f[4 * i + 1] = a[1] * s;
        f[4 * i + 2] = b[0] * s;
        f[4 * i + 3] = b[1] * s;
    }
}

template <typename T, int D, bool FP8>
__global__ void __launch_bounds__(256) kv_write_kernel(KvCall p, int page_shift)
{
    constexpr int LPR = D / 8, RPB = 256 / LPR;
    const int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
    const int el = (threadIdx.x % LPR) * 8;
    const int64_t token = r / p.c.h_kv;
    const int h = (int)(r - token * p.c.h_kv);
    if (token >= p.total) return;  // whole rows leave together
    Eight<T> k, v;
    k.load(static_cast<const T*>(p.k) + token * p.k_token + h * p.k_head + el);
    v.load(static_cast<const T*>(p.v) + token * p.v_token + h * p.v_head + el);
    bool mine;
    const int64_t row = pool_row(p.c, p.start, p.cu, token, h, page_shift, &mine);
    if constexpr (FP8) {
        float f[8];
        uint32_t sk, sv;
        k.get(f);
        const u32x2_t ck = quantise<LPR>(f, &sk);
        v.get(f);
        const u32x2_t cv = quantise<LPR>(f, &sv);
        if (row < 0) return;
        *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.c.k) + row * D + el) = ck;
        *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.c.v) + row * D + el) = cv;
        if (el == 0) {
            p.c.k_scale[row] = (uint8_t)sk;
            p.c.v_scale[row] = (uint8_t)sv;
        }
    } else {
        if (row < 0) return;
        k.store(static_cast<T*>(p.c.k) + row * D + el);
        v.store(static_cast<T*>(p.c.v) + row * D + el);
    }
}

template <typename T, int D, bool FP8>
__global__ void __launch_bounds__(256) kv_read_kernel(KvCall p, int page_shift)
{
    constexpr int LPR = D / 8, RPB = 256 / LPR;
    const int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
    const int el = (threadIdx.x % LPR) * 8;
    const int64_t token = r / p.c.h_kv;
    const int h = (int)(r - token * p.c.h_kv);
    if (token >= p.total) return;
    bool mine;
    const int64_t row = pool_row(p.c, p.start, p.cu, token, h, page_shift, &mine);
    if (!mine) return;
    Eight<T> k, v;
    if (row < 0) {
        const float zero[8] = {};
        k.set(zero);
        v.set(zero);
    } else if constexpr (FP8) {
        const u32x2_t ck = *reinterpret_cast<const u32x2_t*>(static_cast<const uint8_t*>(p.c.k) + row * D + el);
        const u32x2_t cv = *reinterpret_cast<const u32x2_t*>(static_cast<const uint8_t*>(p.c.v) + row * D + el);
        float f[8];
        dequantise(ck, p.c.k_scale[row], f);
        k.set(f);
        dequantise(cv, p.c.v_scale[row], f);
        v.set(f);
    } else {
        k.load(static_cast<const T*>(p.c.k) + row * D + el);
        v.load(static_cast<const T*>(p.c.v) + row * D + el);
    }
    k.store(static_cast<T*>(p.k_out) + r * D + el);
    v.store(static_cast<T*>(p.v_out) + r * D + el);
}

template <typename T, int D, bool FP8>
hipError_t launch_t(const KvCall& c, bool write)
{
    const int64_t rows = c.total * c.c.h_kv, per = 256 / (D / 8);
    const dim3 grid((unsigned)((rows + per - 1) / per)), block(256);
    const int shift = __builtin_ctz((unsigned)c.c.page_size);
    if (write)
        hipLaunchKernelGGL((kv_write_kernel<T, D, FP8>), grid, block, 0, c.stream, c, shift);
    else
        hipLaunchKernelGGL((kv_read_kernel<T, D, FP8>), grid, block, 0, c.stream, c, shift);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_store(const KvCall& c, bool write)
{
    return c.c.store == GDN_FP8 ? launch_t<T, D, true>(c, write) : launch_t<T, D, false>(c, write);
}

template <typename T>
hipError_t launch_d(const KvCall& c, bool write)
{
    switch (c.c.d) {
        case 64: return launch_store<T, 64>(c, write);
        case 128: return launch_store<T, 128>(c, write);
        case 256: return launch_store<T, 256>(c, write);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch(const KvCall& c, bool write)
{
    return c.dtype == GDN_BF16 ? launch_d<uint16_t>(c, write) : launch_d<float>(c, write);
}

}  // namespace

hipError_t launch_kv_write(const KvCall& c)
{
    return launch(c, true);
}

hipError_t launch_kv_read(const KvCall& c)
{
    return launch(c, false);
}

}  // namespace gdn
