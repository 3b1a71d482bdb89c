// gdn_kv_cache.hip -- the paged key-value cache: rows written (quantised as they are written)
// and read back.
//
// A row is the d elements of one (token, KV head). Adjacent lanes hold a row, each as many elements
// of K and of V as it stores in 16 bytes, so that a store covers whole lines and can bypass the
// caches; with an fp8 store the row's largest magnitude is a few cross-lane maxima away.
//
// Both kernels are bound by the bytes they move, once each way. Measured: 24 packed prompts, 8 heads
// of d = 128, bf16 (109 MB each way) written in 41 us, 5.3 TB/s (a large copy: 5.2 to 5.7);
// 65536 fp8 tokens, 2 heads of d = 256, read as bf16 (34 + 134 + 34 MB) in 30 us, 6.7 TB/s, the pool
// staying in the last-level cache; as many written as fp8 in 40 us, 5.0 TB/s. With stores of 8
// bytes a lane through the caches 45 and 55 us.
// A decode step's write takes 3.3 us, less than its launch costs the host (8.7 us a call).
//
// fp8 store: with a = max |x| = m 2^x (1 <= m < 2), the scale 2^e with e = x - 8 + (m > 1.75)
// is the smallest power of two with a / 2^e <= 448 = 1.75 * 2^8. It comes from a's bits, and
// multiplying by 2^-e is exact, so each element is rounded once (to nearest even, by the
// conversion to e4m3).
#include "gdn_attn_internal.hpp"

namespace gdn {
namespace {

// Where a packed row lives: its (page, slot) as a row index of the pools, or -1; *mine: it belongs to
// a sequence. `first` is the token of the wave's first lane.
__device__ __forceinline__ int64_t pool_row(const KvCall& p, int64_t token, int first, int h, int page_shift,
                                            bool* mine)
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

// This thread's piece of a row.
template <int D, int E>
struct Piece {
    static constexpr int LPR = D / E, RPB = 256 / LPR;  // lanes a row, rows a workgroup
    int64_t r, row;  // packed row (token, head); row of the pools, or -1
    uint32_t token;
    int head, el;
    bool mine;
    __device__ __forceinline__ Piece(const KvCall& p, int page_shift)
    {
        el = (int)(threadIdx.x % LPR) * E;
        r = (int64_t)block_index() * RPB + threadIdx.x / LPR;
        token = (uint32_t)r / (uint32_t)p.c.h_kv;  // rows stay below 2^31, and r below 2^32
        head = (int)((uint32_t)r % (uint32_t)p.c.h_kv);
        mine = false;
        const int first = __builtin_amdgcn_readfirstlane((int)token);
        row = pool_row(p, token < p.total ? token : p.total - 1, first, head, page_shift, &mine);
        if (token >= p.total) {
            mine = false;
            row = -1;
        }
    }
};

// Elements a lane writes: 16 bytes of the pool.
template <typename T, bool FP8>
constexpr int write_elems = FP8 ? 16 : Some<T>::E;

template <typename T, int D, bool FP8>
__global__ void __launch_bounds__(256) kv_write_kernel(KvCall p, int page_shift)
{
    constexpr int E = write_elems<T, FP8>, PIECES = E / Some<T>::E;
    using P = Piece<D, E>;
    const P x(p, page_shift);
    if (x.row < 0) return;  // the lanes of a row leave together
    const T* kp = static_cast<const T*>(p.k) + x.token * p.k_token + x.head * p.k_head + x.el;
    const T* vp = static_cast<const T*>(p.v) + x.token * p.v_token + x.head * p.v_head + x.el;
    Some<T> k[PIECES], v[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        k[i].load(kp + i * Some<T>::E);
        v[i].load(vp + i * Some<T>::E);
    }
    const int64_t at = x.row * D + x.el;
    if constexpr (FP8) {
        float f[E];
        uint32_t sk, sv;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) k[i].get(f + i * Some<T>::E);
        const u32x4_t ck = quantise<E, P::LPR>(f, &sk);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) v[i].get(f + i * Some<T>::E);
        const u32x4_t cv = quantise<E, P::LPR>(f, &sv);
        __builtin_nontemporal_store(ck, reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(p.c.k) + at));
        __builtin_nontemporal_store(cv, reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(p.c.v) + at));
        if (x.el == 0) {
            p.c.k_scale[x.row] = (uint8_t)sk;
            p.c.v_scale[x.row] = (uint8_t)sv;
        }
    } else {
        k[0].store(static_cast<T*>(p.c.k) + at);
        v[0].store(static_cast<T*>(p.c.v) + at);
    }
}

template <typename T, int D, bool FP8>
__global__ void __launch_bounds__(256) kv_read_kernel(KvCall p, int page_shift)
{
    constexpr int E = Some<T>::E;
    using P = Piece<D, E>;
    [[maybe_unused]] typedef typename Codes<E>::type W;
    const P x(p, page_shift);
    if (!x.mine) return;
    Some<T> k, v;
    const int64_t at = x.row * D + x.el;
    if (x.row < 0) {
        k.x = v.x = u32x4_t{0, 0, 0, 0};
    } else if constexpr (FP8) {
        const W ck = *reinterpret_cast<const W*>(static_cast<const uint8_t*>(p.c.k) + at);
        const W cv = *reinterpret_cast<const W*>(static_cast<const uint8_t*>(p.c.v) + at);
        float f[E];
        dequantise<E>(ck, p.c.k_scale[x.row], f);
        k.set(f);
        dequantise<E>(cv, p.c.v_scale[x.row], f);
        v.set(f);
    } else {
        k.load(static_cast<const T*>(p.c.k) + at);
        v.load(static_cast<const T*>(p.c.v) + at);
    }
    k.store(static_cast<T*>(p.k_out) + x.r * D + x.el);
    v.store(static_cast<T*>(p.v_out) + x.r * D + x.el);
}

template <typename T, int D, bool FP8>
hipError_t launch_t(const KvCall& c, bool write)
{
    const int64_t rows = c.total * c.c.h_kv;
    const int per = write ? Piece<D, write_elems<T, FP8>>::RPB : Piece<D, Some<T>::E>::RPB;
    const dim3 grid = grid_of((rows + per - 1) / per), block(256);
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
