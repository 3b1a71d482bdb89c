// gdn_rope.hip -- norms and rotary positions of queries and keys, packed or on their way into the
// paged cache.
//
// A row is the d elements of one (token, head). Adjacent lanes hold a row, each two pieces of 16
// bytes: both halves of its pairs, so that the rotation stays in the lane and only the norm's sum
// (and an fp8 store's maximum) crosses lanes. A workgroup takes a few tokens, all heads of them: the
// sines and cosines of its tokens are computed once, one (token, pair) a thread, and read from LDS
// by every head.
//
// Bound by bytes: 30001 tokens of 32/8 heads, d = 128, all rotated by three axes, 113 us (5.4 TB/s read and
// written, a large copy's rate); 4096 tokens of 16/2 heads, d = 256, 15 us; a packed append of 24
// prompts, 8 KV heads, d = 128, 45 us (4.8 TB/s); 16384 tokens of 16/2 heads, d = 256, with an fp8 store 67 us. A
// lane's pieces lie beside its neighbours', the next row is loaded while one is worked on, and stores of
// whole lines bypass the caches: without these three 133, 49 and 91 us of the first, third and last.
//
// Angles. freq * pos, in turns, is formed in two 64-bit numbers (the product, and what its roundings leave: without it
// 4e-7 radians are lost by 2^31) and reduced there to a fraction of a turn in [-1/2, 1/2]; what its rounding to fp32
// leaves out is put back by one term of the addition theorems, so that sine and cosine are as good as the library's
// functions of an exact angle at any position.
#include "gdn_kv_rows.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;  // of a workgroup, at most

// scale * (cos, sin) of freq * pos.
__device__ __forceinline__ float2 turn(double pos, float freq, float scale)
{
    constexpr double kTurn = 0.15915494309189535, kRest = -9.839338337591243e-18;  // 1 / (2 pi) and what its rounding leaves
    const double angle = pos * (double)freq, left = __builtin_fma(pos, (double)freq, -angle);
    const double t = __builtin_fma(angle, kTurn, -__builtin_rint(angle * kTurn)) + (angle * kRest + left * kTurn);
    const float r = (float)t;
    const float rest = (float)(t - (double)r) * 6.2831853f;
    float s, c;
    sincospif(2.f * r, &s, &c);
    return make_float2(scale * (c - rest * s), scale * (s + rest * c));
}

enum { kPacked, kSame, kFp8 };  // where keys go: k_out, a pool of T, an fp8 pool

// First elements of the lane's two pieces: both halves of the same pairs, and behind the rotated elements a
// piece of either half of the rest, so that neighbouring lanes' pieces are neighbours in memory. Rows without
// such pairs: a piece of either half.
template <int D, int PIECE>
__device__ __forceinline__ void pieces_of(int lane, int rot, bool paired, int* a, int* b)
{
    const int split = paired ? rot : 0, first = lane * 2 * PIECE < split ? 0 : split;
    const int size = first < split ? split : D - split;  // of the part that the lane is in
    *a = first + (lane - first / (2 * PIECE)) * PIECE;
    *b = *a + size / 2;
}

template <typename T, int D, int STORE>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeCall p, int tok, int page_shift)
{
    constexpr int PIECE = Some<T>::E, E = 2 * PIECE, LPR = D / E, RPB = kThreads / LPR;
    __shared__ __align__(16) float s_cos[kThreads], s_sin[kThreads];
    __shared__ int64_t s_row[kTokens];
    const int half = p.f.rot / 2, per = half > 0 ? half : 1;
    const int64_t token0 = (int64_t)block_index() * tok;
    if (token0 >= p.total) return;  // past the grid's end
    const int tokens = p.total - token0 < tok ? (int)(p.total - token0) : tok;

    // This thread's rows: head h of the token t, then every RPB-th. The next one's pieces are loaded while one
    // is worked on, the first one's before the angles.
    const int lane = threadIdx.x % LPR;
    const int heads = p.h_q + p.h_kv * (STORE == kPacked ? 1 : 2);
    const bool paired = !p.f.interleaved;
    int ra, rb;  // pieces of a rotated row
    pieces_of<D, PIECE>(lane, p.f.rot, paired, &ra, &rb);
    const int va = lane * PIECE, vb = va + D / 2;  // of a V row
    // Where the lanes of a store cover whole lines it bypasses the caches.
    constexpr int LINE = 128 / (int)sizeof(T);
    constexpr bool WHOLE = D / 2 % LINE == 0;
    const bool whole = paired ? p.f.rot / 2 % LINE == 0 && (D - p.f.rot) / 2 % LINE == 0 : WHOLE;
    int t = 0, h = threadIdx.x / LPR;
    auto settle = [&]() __attribute__((always_inline)) {
        while (h >= heads) {
            h -= heads;
            ++t;
        }
    };
    Some<T> na, nb;
    auto load = [&]() __attribute__((always_inline)) {
        const int64_t token = token0 + t;
        const bool is_q = h < p.h_q, rotates = h < p.h_q + p.h_kv;
        const T* from = is_q       ? static_cast<const T*>(p.q) + token * p.q_token + h * p.q_head
                        : rotates  ? static_cast<const T*>(p.k) + token * p.k_token + (h - p.h_q) * p.k_head
                                   : static_cast<const T*>(p.v) + token * p.v_token + (h - p.h_q - p.h_kv) * p.v_head;
        na.load(from + (rotates ? ra : va));
        nb.load(from + (rotates ? rb : vb));
    };
    settle();
    if (t < tokens) load();

    {  // tok * per <= kThreads: every thread one (token, pair) at most
        const int y = threadIdx.x / per, x = threadIdx.x - y * per;
        const int64_t token = token0 + (y < tokens ? y : tokens - 1);
        int64_t at = 0;
        if constexpr (STORE != kPacked) {
            bool mine;
            const int64_t first = token0 + (int)(threadIdx.x & ~63u) / per;  // of the wave's first lane
            const int64_t row = pool_row(p, token, (int)(first < p.total ? first : p.total - 1), 0, page_shift, &mine, &at);
            if (x == 0 && y < tokens) s_row[y] = mine ? row : -2;
            if (!mine) at = 0;
        }
        if (half > 0 && y < tokens) {
            if (STORE == kPacked || p.f.pos) {
                int axis = p.f.axis ? p.f.axis[x] : 0;
                axis = axis < p.f.axes ? axis : p.f.axes - 1;
                at = p.f.pos[axis * p.total + token];
            }
            const float2 cs = turn((double)at, p.f.freq[x], p.f.rope_scale);
            s_cos[threadIdx.x] = cs.x;
            s_sin[threadIdx.x] = cs.y;
        }
    }
    __syncthreads();

    while (t < tokens) {
        const int64_t token = token0 + t;
        const int y = t;
        const bool is_q = h < p.h_q, is_k = !is_q && h < p.h_q + p.h_kv, rotates = is_q || is_k;
        const int head = is_q ? h : is_k ? h - p.h_q : h - p.h_q - p.h_kv;
        const int a = rotates ? ra : va, b = rotates ? rb : vb;
        Some<T> xa = na, xb = nb;
        h += RPB;
        settle();
        if (t < tokens) load();
        int64_t row = 0;
        if constexpr (STORE != kPacked) {
            row = s_row[y];
            if (row == -2 || (row < 0 && !is_q)) continue;  // the lanes of a row go together
            row += (int64_t)head << page_shift;
        }
        float f[E];
        xa.get(f);
        xb.get(f + PIECE);
        const T* weight = static_cast<const T*>(is_q ? p.f.q_weight : is_k ? p.f.k_weight : nullptr);
        if (weight) {
            auto sum_of = [&](float s) __attribute__((always_inline)) {
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < E; ++i) x += (f[i] * s) * (f[i] * s);
#pragma unroll
                for (int off = LPR / 2; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
                return x;
            };
            // Squares that leave fp32's range are taken of the row times a power of two, which is exact:
            // the norm has no other effect than on eps. 2^100 brings the smallest squares far into fp32's range.
            float unit = 1.f, sum = sum_of(1.f);
            if (!(sum <= 3.4028234e38f) || (sum < 0x1p-100f && p.f.eps < 0x1p-100f)) {
                unit = sum < 1.f ? 0x1p100f : 0x1p-70f;
                sum = sum_of(unit);
            }
            const float inv = 1.f / sqrtf(sum * (1.f / D) + p.f.eps * unit * unit);
            Some<T> wa, wb;
            wa.load(weight + a);
            wb.load(weight + b);
            float w[E];
            wa.get(w);
            wb.get(w + PIECE);
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = f[i] * unit * inv * (p.f.weight_bias + w[i]);
        }
        if (rotates && paired && a < p.f.rot) {  // PIECE pairs, an element of each in either piece
            float c[PIECE], s[PIECE];
            const int at = y * half + a;
#pragma unroll
            for (int i = 0; i < PIECE; i += 4) {
                *reinterpret_cast<f32x4_t*>(c + i) = *reinterpret_cast<const f32x4_t*>(s_cos + at + i);
                *reinterpret_cast<f32x4_t*>(s + i) = *reinterpret_cast<const f32x4_t*>(s_sin + at + i);
            }
#pragma unroll
            for (int i = 0; i < PIECE; ++i) {
                const float x = f[i], z = f[PIECE + i];
                f[i] = x * c[i] - z * s[i];
                f[PIECE + i] = z * c[i] + x * s[i];
            }
        }
        if (rotates && !paired) {  // PIECE / 2 pairs in each piece
#pragma unroll
            for (int half_row = 0; half_row < 2; ++half_row) {
                const int from = half_row ? b : a, at = y * half + from / 2;
                if (from < p.f.rot) {
#pragma unroll
                    for (int i = 0; i < PIECE / 2; ++i) {
                        const float c = s_cos[at + i], s = s_sin[at + i];
                        float& u = f[half_row * PIECE + 2 * i];
                        float& z = f[half_row * PIECE + 2 * i + 1];
                        const float x = u;
                        u = x * c - z * s;
                        z = z * c + x * s;
                    }
                }
            }
        }
        if (STORE == kFp8 && !is_q) {
            uint32_t scale;
            const auto code = quantise<E, LPR>(f, &scale);
            uint8_t* to = static_cast<uint8_t*>(is_k ? p.c.k : p.c.v) + row * D;
            typedef typename Codes<PIECE>::type W;
            W ca, cb;
            if constexpr (PIECE == 8) {
                ca = W{code[0], code[1]};
                cb = W{code[2], code[3]};
            } else {
                ca = code[0];
                cb = code[1];
            }
            *reinterpret_cast<W*>(to + a) = ca;
            *reinterpret_cast<W*>(to + b) = cb;
            if (lane == 0) (is_k ? p.c.k_scale : p.c.v_scale)[row] = (uint8_t)scale;
        } else {
            T* to = is_q ? static_cast<T*>(p.q_out) + (token * p.h_q + head) * D
                  : STORE == kPacked ? static_cast<T*>(p.k_out) + (token * p.h_kv + head) * D
                                     : static_cast<T*>(is_k ? p.c.k : p.c.v) + row * D;
            xa.set(f);
            xb.set(f + PIECE);
            if (rotates ? whole : WHOLE) {
                asm volatile("" ::: "memory");  // the compiler would make both ways' stores one, of the other kind
                __builtin_nontemporal_store(xa.x, reinterpret_cast<u32x4_t*>(to + a));
                __builtin_nontemporal_store(xb.x, reinterpret_cast<u32x4_t*>(to + b));
                asm volatile("" ::: "memory");
            } else {
                *reinterpret_cast<u32x4_t*>(to + a) = xa.x;
                *reinterpret_cast<u32x4_t*>(to + b) = xb.x;
            }
        }
    }
}

template <typename T, int D, int STORE>
hipError_t launch_t(const RopeCall& c)
{
    const int per = c.f.rot > 0 ? c.f.rot / 2 : 1;
    constexpr int RPB = kThreads * 2 * Some<T>::E / D;
    const int64_t heads = c.h_q + (int64_t)c.h_kv * (STORE == kPacked ? 1 : 2);
    int64_t tok = (4 * RPB + heads - 1) / heads, most = c.total / 2048;
    if (most > kThreads / per) most = kThreads / per;
    if (most > kTokens) most = kTokens;
    tok = tok > most ? most : tok;
    tok = tok < 1 ? 1 : tok;
    hipLaunchKernelGGL((rope_kernel<T, D, STORE>), grid_of((c.total + tok - 1) / tok), dim3(kThreads), 0, c.stream, c,
                       (int)tok, STORE == kPacked ? 0 : __builtin_ctz((unsigned)c.c.page_size));
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_store(const RopeCall& c, bool cache)
{
    return !cache ? launch_t<T, D, kPacked>(c) : c.c.store == GDN_FP8 ? launch_t<T, D, kFp8>(c) : launch_t<T, D, kSame>(c);
}

template <typename T>
hipError_t launch_d(const RopeCall& c, bool cache)
{
    switch (c.d) {
        case 64: return launch_store<T, 64>(c, cache);
        case 128: return launch_store<T, 128>(c, cache);
        case 256: return launch_store<T, 256>(c, cache);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_rope(const RopeCall& c, bool cache)
{
    return c.dtype == GDN_BF16 ? launch_d<uint16_t>(c, cache) : launch_d<float>(c, cache);
}

}  // namespace gdn
