// gdn_attn_prefill.hip -- attention over packed prompts: causal or full, grouped heads.
//
// Rows. The G = h_q / h_kv heads of a KV head read the same keys, so a workgroup's tile is M
// packed query rows of one (sequence, KV head): row r is position r / G, head r % G of the
// group. A tile then reads each key once for all its heads, and its causal edge is M / G
// positions wide.
//
// Grid. The host does not know the sequences' lengths. Sequence s gets the tiles
// [floor(cu_q[s] G / M) + s, floor(cu_q[s + 1] G / M) + s + 1), which are disjoint, in order
// and enough for its ceil(len G / M); a workgroup finds its sequence by bisection and leaves
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
// rows past the end of a sequence are read as zeros, and in tiles that hold masked keys an
// operand with a non-finite V is taken key by key, kept only in the rows that see the key.
#include "gdn_attn_internal.hpp"

namespace gdn {
namespace {

constexpr int kWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T, int D>
struct Tile;

// bf16: 32 query rows per wave; 64 keys per step, 32 where a row's registers (its share of O
// and Q) take most of the 256 a wave has at two waves per SIMD
template <int D>
struct Tile<uint16_t, D> {
    static constexpr int N = D == 256 ? 32 : 64, M = 32 * kWaves;
};

// fp32: 32 query rows per wave, 32 keys per step
template <int D>
struct Tile<float, D> {
    static constexpr int N = 32, M = 32 * kWaves;
};

// A workgroup's tile: its sequence, rows and key count.
struct Work {
    int64_t q0, k0;     // first packed rows of the sequence
    int64_t len_q, len_k;
    int64_t row0, rows; // first packed (position, head) row, and how many the sequence has
    int head;           // KV head
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t hi)
{
    return x < 0 ? 0 : (x > hi ? hi : x);
}

// floor(cu[s] G / M) + s, the first tile of sequence s
__device__ __forceinline__ int64_t tile_base(const int32_t* cu, int64_t s, int64_t total, int g, int m)
{
    return clamp64(cu[s], total) * g / m + s;
}

template <int M>
__device__ __forceinline__ bool find_work(const AttnCall& p, int64_t tile, int head, Work* w)
{
    const gdn_attn_dims& d = p.d;
    const int g = d.h_q / d.h_kv;
    int64_t lo = 0, hi = d.n;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (tile_base(p.cu_q, mid, d.total_q, g, M) <= tile) lo = mid; else hi = mid;
    }
    const int64_t qa = clamp64(p.cu_q[lo], d.total_q), qb = clamp64(p.cu_q[lo + 1], d.total_q);
    const int64_t ka = clamp64(p.cu_k[lo], d.total_k), kb = clamp64(p.cu_k[lo + 1], d.total_k);
    w->q0 = qa;
    w->k0 = ka;
    w->len_q = qb - qa;
    w->len_k = kb > ka ? kb - ka : 0;
    w->rows = w->len_q * g;
    w->head = head;
    if (w->len_q <= 0) return false;
    const int64_t tiles = (w->rows + M - 1) / M, local = tile - tile_base(p.cu_q, lo, d.total_q, g, M);
    if (local < 0 || local >= tiles) return false;
    w->row0 = (tiles - 1 - local) * M;
    return true;
}

// Keys that a query row at position pos sees: [0, limit).
__device__ __forceinline__ int64_t key_limit(const Work& w, int64_t pos, int causal)
{
    if (!causal) return w.len_k;
    const int64_t lim = pos + 1 + w.len_k - w.len_q;
    return lim < 0 ? 0 : (lim > w.len_k ? w.len_k : lim);
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

// 16-byte chunk of a K row at which logical chunk c is kept: the rows that a wave's read
// touches together then lie in different banks. The loads to LDS apply it by choosing which
// chunk each lane fetches.
template <int CHUNKS>
__device__ __forceinline__ int swz_k(int row)
{
    return row & (CHUNKS < 16 ? CHUNKS - 1 : 15);
}

// The same for V rows: the transposing read takes pairs of chunks from four rows at a time.
template <int CHUNKS>
__device__ __forceinline__ int swz_v(int row)
{
    const int x = (row & 3) | ((row & 1) << 2);
    return (2 * x) & (CHUNKS - 1);
}

// Rows [row, row + N) of a strided [..][D] tensor into LDS, zeros from `valid` rows on.
// CHUNKS 16-byte chunks a row; swizzled.
template <int N, int CHUNKS, bool V>
__device__ __forceinline__ void stage(const char* base, int64_t row, int64_t valid, int64_t stride,
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
        const int src = cc ^ (V ? swz_v<CHUNKS>(rr) : swz_k<CHUNKS>(rr));
        load_to_lds(r, lds + at * 16, (int)(rr * stride) + src * 16);
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
    float m, l;  // reference maximum (-inf: nothing seen), sum of weights of this lane's keys
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
__device__ __forceinline__ void write_row(const AttnCall& p, const Work& w, int64_t r, int lane,
                                          const f32x16_t* o, const Stats& st)
{
    const int g = p.d.h_q / p.d.h_kv;
    const float l = other_half_sum(st.l);
    if (r >= w.rows) return;
    const int64_t pos = r / g, row = (w.q0 + pos) * p.d.h_q + (int64_t)w.head * g + (r - pos * g);
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    T* out = static_cast<T*>(p.out) + row * D + 4 * (lane >> 5);
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = o[db][4 * i] * inv, b = o[db][4 * i + 1] * inv;
            const float c = o[db][4 * i + 2] * inv, e = o[db][4 * i + 3] * inv;
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<u32x2_t*>(out + 32 * db + 8 * i) = u32x2_t{pack_bf16(a, b), pack_bf16(c, e)};
            else
                *reinterpret_cast<f32x4_t*>(out + 32 * db + 8 * i) = f32x4_t{a, b, c, e};
        }
    if (p.lse && lane < 32) p.lse[row] = l > 0.f ? (st.m + __builtin_amdgcn_logf(l)) * kLn2 : (l == l ? -INFINITY : l);
}

// One step of a wave's 32 rows over N staged keys. MASKED: some of the keys may not be seen by
// some of the rows: row `lane & 31` sees those below lim.
template <int D, bool MASKED>
__device__ __forceinline__ void bf16_step(const char* sk, const char* sv, const bf16x8_t (&q)[D / 16],
                                          f32x16_t (&o)[D / 32], Stats& st, float c, int lim, int lane)
{
    constexpr int N = Tile<uint16_t, D>::N, CH = D / 8, ND = D / 32;
    const int half = lane >> 5, l31 = lane & 31;
    f32x16_t s[N / 32];
#pragma unroll
    for (int b = 0; b < N / 32; ++b) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
        const int row = 32 * b + l31;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int ch = (2 * kk + half) ^ swz_k<CH>(row);
            const bf16x8_t a = *reinterpret_cast<const bf16x8_t*>(sk + row * (D * 2) + ch * 16);
            s[b] = mfma32(a, q[kk], s[b]);
        }
    }
    // key of register i of block b: 32 b + 8 (i / 4) + 4 half + i % 4
    float mx = -INFINITY;
#pragma unroll
    for (int b = 0; b < N / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (MASKED) s[b][i] = 32 * b + 8 * (i / 4) + 4 * half + i % 4 < lim ? s[b][i] : -INFINITY;
            mx = fmaxf(mx, s[b][i]);
        }
    mx = other_half_max(mx);
    // the reference maximum moves only when weights would pass 2^8: O is then rescaled
    const bool rise = mx > st.m && (st.m == -INFINITY || (mx - st.m) * c > 8.f);
    if (__any(rise)) {
        const float a = !rise ? 1.f : st.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((st.m - mx) * c);
        st.m = rise ? mx : st.m;
        st.l *= a;
#pragma unroll
        for (int db = 0; db < ND; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[db][i] *= a;
    }
    const float ref = st.m == -INFINITY ? 0.f : st.m * c;
#pragma unroll
    for (int b = 0; b < N / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], c, -ref));
            if (MASKED) p = 32 * b + 8 * (i / 4) + 4 * half + i % 4 < lim ? p : 0.f;
            s[b][i] = p;
            st.l += p;
        }
#pragma unroll
    for (int t = 0; t < N / 16; ++t) {
        u32x4_t pw;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pw[i] = pack_bf16(s[t / 2][8 * (t & 1) + 2 * i], s[t / 2][8 * (t & 1) + 2 * i + 1]);
        const bf16x8_t pb = __builtin_bit_cast(bf16x8_t, pw);
        const int i16 = lane & 15, gg = (lane >> 4) & 1;
        const int row = 16 * t + 4 * half + (i16 >> 2);
#pragma unroll
        for (int db = 0; db < ND; ++db) {
            const int ch = 4 * db + 2 * gg + ((i16 >> 1) & 1), in = 8 * (i16 & 1);
            const bf16x4_t a0 = read_tr(sv + row * (D * 2) + (ch ^ swz_v<CH>(row)) * 16 + in);
            const bf16x4_t a1 = read_tr(sv + (row + 8) * (D * 2) + (ch ^ swz_v<CH>(row + 8)) * 16 + in);
            const bf16x8_t a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
            if (MASKED && any_not_finite(a)) {
#pragma unroll 1
                for (int key = 0; key < 16; ++key) {
                    // key 8 (j / 4) + 4 half + j % 4 sits in slot j of this half
                    const int slot = 4 * (key >> 3) + (key & 3);
                    const bool mine = ((key >> 2) & 1) == half;
                    u32x4_t one = __builtin_bit_cast(u32x4_t, a);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        one[i] &= mine && (slot >> 1) == i ? (slot & 1 ? 0xffff0000u : 0xffffu) : 0u;
                    const f32x16_t x = mfma32(__builtin_bit_cast(bf16x8_t, one), pb, o[db]);
                    const bool sees = 16 * t + key < lim;
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[db][i] = sees ? x[i] : o[db][i];
                }
            } else {
                o[db] = mfma32(a, pb, o[db]);
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(64 * kWaves, 2) prefill_bf16_kernel(AttnCall p)
{
    constexpr int N = Tile<uint16_t, D>::N, M = Tile<uint16_t, D>::M, CH = D / 8, ND = D / 32;
    __shared__ __align__(16) char s_k[2][N * D * 2];
    __shared__ __align__(16) char s_v[2][N * D * 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Work w;
    if (!find_work<M>(p, blockIdx.x / p.d.h_kv, blockIdx.x % p.d.h_kv, &w)) return;
    const int g = p.d.h_q / p.d.h_kv;

    // this lane's query: row r of the sequence's packed rows
    const int64_t r = w.row0 + 32 * wave + (lane & 31);
    const int64_t rc = r < w.rows ? r : w.rows - 1, pos = rc / g;
    const uint16_t* qp = static_cast<const uint16_t*>(p.q) + (w.q0 + pos) * p.d.q_token +
                         ((int64_t)w.head * g + (rc - pos * g)) * p.d.q_head + 8 * (lane >> 5);
    // a negative scale becomes a positive one of the negated query: the maximum of the raw
    // scores is then that of the scaled ones
    const uint32_t flip = p.d.scale < 0.f ? 0x80008000u : 0u;
    const float c = fabsf(p.d.scale) * kLog2e;
    bf16x8_t q[D / 16];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        q[kk] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(qp + 16 * kk) ^ flip);

    // keys that the workgroup's last row sees, that all of its rows see, and per lane
    const int64_t last = (w.row0 + M < w.rows ? w.row0 + M : w.rows) - 1;
    const int64_t keys = key_limit(w, last / g, p.d.causal);
    const int64_t all = key_limit(w, w.row0 / g, p.d.causal);
    const int64_t limit = key_limit(w, pos, p.d.causal);
    const int64_t wlast = w.row0 + 32 * wave + 31 < w.rows ? w.row0 + 32 * wave + 31 : w.rows - 1;
    const int64_t wkeys = key_limit(w, wlast / g, p.d.causal);

    const char* kb = static_cast<const char*>(p.k) + 2 * (w.k0 * p.d.k_token + w.head * p.d.k_head);
    const char* vb = static_cast<const char*>(p.v) + 2 * (w.k0 * p.d.v_token + w.head * p.d.v_head);

    f32x16_t o[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] = 0.f;
    Stats st = {-INFINITY, 0.f};

    // Two buffers: while a step's keys are used the next step's arrive. The barrier at the top
    // of a step has every wave's loads of it done, and every wave past the buffer refilled next.
    const int64_t steps = (keys + N - 1) / N, plain = all / N;
    if (steps > 0) {
        stage<N, CH, false>(kb, 0, w.len_k, 2 * p.d.k_token, s_k[0], wave, lane);
        stage<N, CH, true>(vb, 0, w.len_k, 2 * p.d.v_token, s_v[0], wave, lane);
    }
    int64_t x = 0;
    for (; x < plain; ++x) {
        __syncthreads();
        if (x + 1 < steps) {
            stage<N, CH, false>(kb, (x + 1) * N, w.len_k, 2 * p.d.k_token, s_k[(x + 1) & 1], wave, lane);
            stage<N, CH, true>(vb, (x + 1) * N, w.len_k, 2 * p.d.v_token, s_v[(x + 1) & 1], wave, lane);
        }
        bf16_step<D, false>(s_k[x & 1], s_v[x & 1], q, o, st, c, N, lane);
    }
    for (; x < steps; ++x) {
        __syncthreads();
        if (x + 1 < steps) {
            stage<N, CH, false>(kb, (x + 1) * N, w.len_k, 2 * p.d.k_token, s_k[(x + 1) & 1], wave, lane);
            stage<N, CH, true>(vb, (x + 1) * N, w.len_k, 2 * p.d.v_token, s_v[(x + 1) & 1], wave, lane);
        }
        if (x * N >= wkeys) continue;  // nothing here for this wave's rows
        const int64_t left = limit - x * N;
        bf16_step<D, true>(s_k[x & 1], s_v[x & 1], q, o, st, c, (int)(left < 0 ? 0 : left < N ? left : N), lane);
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
    if (!find_work<M>(p, blockIdx.x / p.d.h_kv, blockIdx.x % p.d.h_kv, &w)) return;
    const int g = p.d.h_q / p.d.h_kv;

    const int64_t r = w.row0 + 32 * wave + l31;
    const int64_t pos = (r < w.rows ? r : w.rows - 1) / g, hh = (r < w.rows ? r : w.rows - 1) - pos * g;
    const int64_t limit = key_limit(w, pos, p.d.causal);
    const float* qp = static_cast<const float*>(p.q) + (w.q0 + pos) * p.d.q_token +
                      ((int64_t)w.head * g + hh) * p.d.q_head + 4 * half;
    f32x4_t q[D / 8];  // slot e of step kk: element 8 kk + 4 half + e
#pragma unroll
    for (int kk = 0; kk < D / 8; ++kk) q[kk] = *reinterpret_cast<const f32x4_t*>(qp + 8 * kk);

    const int64_t last = (w.row0 + M < w.rows ? w.row0 + M : w.rows) - 1;
    const int64_t keys = key_limit(w, last / g, p.d.causal);
    const int64_t wrow = w.row0 + 32 * wave;
    const int64_t all = key_limit(w, (wrow < w.rows ? wrow : w.rows - 1) / g, p.d.causal);

    const char* kb = static_cast<const char*>(p.k) + 4 * (w.k0 * p.d.k_token + w.head * p.d.k_head);
    const char* vb = static_cast<const char*>(p.v) + 4 * (w.k0 * p.d.v_token + w.head * p.d.v_head);
    const float c = p.d.scale * kLog2e;

    f32x16_t o[ND];
#pragma unroll
    for (int db = 0; db < ND; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] = 0.f;
    Stats st = {-INFINITY, 0.f};

    for (int64_t j0 = 0; j0 < keys; j0 += N) {
        __syncthreads();
        stage<N, CH, false>(kb, j0, w.len_k, 4 * p.d.k_token, s_k, wave, lane);
        stage<N, CH, false>(vb, j0, w.len_k, 4 * p.d.v_token, s_v, wave, lane);
        __syncthreads();

        float s[16];
        f32x16_t acc;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 8; ++kk) {
            const int ch = (2 * kk + half) ^ swz_k<CH>(l31);
            const f32x4_t a = *reinterpret_cast<const f32x4_t*>(s_k + l31 * (D * 4) + ch * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], q[kk][e], acc, 0, 0, 0);
        }
        const bool masked = j0 + N > all;
        const int lim = (int)(limit - j0 < N ? limit - j0 : N);
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
                                                                (ch ^ swz_k<CH>(row)) * 16 + 4 * (l31 & 3));
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
    write_row<float, D>(p, w, r, lane, o, st);
}

template <typename T, int D>
hipError_t launch_t(const AttnCall& c)
{
    const int64_t rows = c.d.total_q * (c.d.h_q / c.d.h_kv);
    const int64_t tiles = rows / Tile<T, D>::M + c.d.n;
    const dim3 grid((unsigned)(tiles * c.d.h_kv)), block(64 * kWaves);
    if constexpr (sizeof(T) == 2)
        hipLaunchKernelGGL((prefill_bf16_kernel<D>), grid, block, 0, c.stream, c);
    else
        hipLaunchKernelGGL((prefill_f32_kernel<D>), grid, block, 0, c.stream, c);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_d(const AttnCall& c)
{
    switch (c.d.d) {
        case 64: return launch_t<T, 64>(c);
        case 128: return launch_t<T, 128>(c);
        case 256: return launch_t<T, 256>(c);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

int attn_prefill_rows(int32_t, int32_t)
{
    return 32 * kWaves;
}

hipError_t launch_attn_prefill(const AttnCall& c)
{
    return c.d.dtype == GDN_BF16 ? launch_d<uint16_t>(c) : launch_d<float>(c);
}

}  // namespace gdn
