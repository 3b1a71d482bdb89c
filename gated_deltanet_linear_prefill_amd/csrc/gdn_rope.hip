// gdn_rope.hip -- norms and rotary positions of queries and keys, packed or on their way into the
// paged cache.
//
// A row is the d elements of one (token, head). Adjacent lanes hold a row, each two pieces of 16
// bytes: both halves of its pairs, so that the rotation stays in the lane and only the norm's sum
// (and an fp8 store's maximum) crosses lanes. A workgroup takes a few tokens, all heads of them: the
// sines and cosines of its tokens are computed once, one (token, pair) a thread, and read from LDS
// by every head.
//
// Angles. freq * pos is formed in 64 bits and reduced there to a fraction of a turn in
// [-1/2, 1/2]; what its rounding to fp32 leaves out is put back by one term of the addition
// theorems, so that sine and cosine are good to about an ulp at any position.
#include "gdn_kv_rows.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;  // of a workgroup, at most

// scale * (cos, sin) of freq * pos.
__device__ __forceinline__ float2 turn(double pos, float freq, float scale)
{
    double t = pos * (double)freq * 0.15915494309189533577;  // turns
    t -= __builtin_rint(t);
    const float r = (float)t;
    const float rest = (float)(t - (double)r) * 6.2831853f;
    float s, c;
    sincospif(2.f * r, &s, &c);
    return make_float2(scale * (c - rest * s), scale * (s + rest * c));
}

enum { kPacked, kSame, kFp8 };  // where keys go: k_out, a pool of T, an fp8 pool

// First elements of the lane's two pieces of E / 2: halves of the same pairs, or neighbours.
__device__ __forceinline__ void pieces_of(int lane, int piece, int rot, bool paired, int* a, int* b)
{
    const bool split = paired && lane * 2 * piece < rot;
    *a = split ? lane * piece : lane * 2 * piece;
    *b = split ? lane * piece + rot / 2 : *a + piece;
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

    {  // tok * per <= kThreads: every thread one (token, pair) at most
        const int t = threadIdx.x / per, x = threadIdx.x - t * per;
        const int64_t token = token0 + (t < tokens ? t : tokens - 1);
        int64_t at = 0, row = 0;
        if constexpr (STORE != kPacked) {
            bool mine;
            const int64_t first = token0 + (int)(threadIdx.x & ~63u) / per;  // of the wave's first lane
            row = pool_row(p, token, (int)(first < p.total ? first : p.total - 1), 0, page_shift, &mine, &at);
            if (x == 0 && t < tokens) s_row[t] = mine ? row : -2;
            if (!mine) at = 0;
        }
        if (half > 0 && t < tokens) {
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

    const int lane = threadIdx.x % LPR;
    const int heads = p.h_q + p.h_kv * (STORE == kPacked ? 1 : 2);
    const bool paired = !p.f.interleaved;
    int ra, rb;  // pieces of a rotated row
    pieces_of(lane, PIECE, p.f.rot, paired, &ra, &rb);
    const bool turns = lane * E < p.f.rot;
    int t = 0, h = threadIdx.x / LPR;
    for (;; h += RPB) {
        while (h >= heads) {
            h -= heads;
            ++t;
        }
        if (t >= tokens) break;
        const int64_t token = token0 + t;
        const bool is_q = h < p.h_q, is_k = !is_q && h < p.h_q + p.h_kv;
        const int head = is_q ? h : is_k ? h - p.h_q : h - p.h_q - p.h_kv;
        int64_t row = 0;
        if constexpr (STORE != kPacked) {
            row = s_row[t];
            if (row == -2 || (row < 0 && !is_q)) continue;  // the lanes of a row go together
            row += (int64_t)head << page_shift;
        }
        const T* from = is_q ? static_cast<const T*>(p.q) + token * p.q_token + head * p.q_head
                      : is_k ? static_cast<const T*>(p.k) + token * p.k_token + head * p.k_head
                             : static_cast<const T*>(p.v) + token * p.v_token + head * p.v_head;
        const bool rotates = is_q || is_k;
        const int a = rotates ? ra : lane * E, b = rotates ? rb : lane * E + PIECE;
        Some<T> xa, xb;
        xa.load(from + a);
        xb.load(from + b);
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
            // the norm has no other effect than on eps.
            float unit = 1.f, sum = sum_of(1.f);
            if (!(sum <= 3.4028234e38f) || (sum < 0x1p-100f && p.f.eps < 0x1p-100f)) {
                unit = sum < 1.f ? 0x1p70f : 0x1p-70f;
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
        if (rotates && turns) {
            const int at = t * half + (paired ? ra : lane * PIECE);
            float c[PIECE], s[PIECE];
#pragma unroll
            for (int i = 0; i < PIECE; i += 4) {
                *reinterpret_cast<f32x4_t*>(c + i) = *reinterpret_cast<const f32x4_t*>(s_cos + at + i);
                *reinterpret_cast<f32x4_t*>(s + i) = *reinterpret_cast<const f32x4_t*>(s_sin + at + i);
            }
            if (paired) {
#pragma unroll
                for (int i = 0; i < PIECE; ++i) {
                    const float x = f[i], y = f[PIECE + i];
                    f[i] = x * c[i] - y * s[i];
                    f[PIECE + i] = y * c[i] + x * s[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < PIECE; ++i) {
                    const float x = f[2 * i], y = f[2 * i + 1];
                    f[2 * i] = x * c[i] - y * s[i];
                    f[2 * i + 1] = y * c[i] + x * s[i];
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
            *reinterpret_cast<u32x4_t*>(to + a) = xa.x;
            *reinterpret_cast<u32x4_t*>(to + b) = xb.x;
        }
    }
}

template <typename T, int D, int STORE>
hipError_t launch_t(const RopeCall& c)
{
    const int per = c.f.rot > 0 ? c.f.rot / 2 : 1;
    int64_t tok = c.total / 2048;
    const int most = kThreads / per < kTokens ? kThreads / per : kTokens;
    tok = tok < 1 ? 1 : tok > most ? most : tok;
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
