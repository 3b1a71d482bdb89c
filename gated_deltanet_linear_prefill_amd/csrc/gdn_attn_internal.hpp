// gdn_attn_internal.hpp -- shared host/device pieces of the attention entry points (not part
// of the C ABI).
#pragma once

#include "gdn_internal.hpp"

namespace gdn {

// Validated calls: sizes and strides checked, pointers present, aligned and disjoint.
struct KvCall {
    gdn_kv_cache c;
    int64_t total;
    int32_t dtype;
    const void *k, *v;  // written from
    int64_t k_token, k_head, v_token, v_head;
    void *k_out, *v_out;  // read into
    const int32_t *start, *cu;
    hipStream_t stream;
};

struct AttnCall {
    gdn_attn_dims d;
    const void *q, *k, *v;
    const int32_t *cu_q, *cu_k;
    void* out;
    float* lse;
    void* ws;
    hipStream_t stream;
    // Set by the launcher: tiles of all KV heads, ranges of a tile's keys, and where their sums go,
    // [unit][range][row]: o [d] and (m, l, exact l, -).
    int units, ranges;
    float* part_o;
    float4* part_ml;
};

struct AttnDecodeCall {
    gdn_kv_cache c;
    int32_t h_q, dtype;
    float scale;
    int64_t max_len;
    const void* q;
    int64_t q_token, q_head;
    const int32_t* lens;
    void* out;
    float* lse;
    void* ws;
    hipStream_t stream;
};

// gdn_qk_norm_rope (no cache: h_kv heads of k to k_out) and gdn_kv_append.
struct RopeCall {
    gdn_norm_rope f;
    gdn_kv_cache c;
    int64_t total;
    int32_t h_q, h_kv, d, dtype;
    const void *q, *k, *v;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;
    void *q_out, *k_out;
    const int32_t *start, *cu;
    hipStream_t stream;
};

// max_len is bounded by the page table, max_q by total_q; window 0 and sinks 0 where there is no window.
struct ExtendCall {
    gdn_kv_cache c;
    gdn_extend_dims d;
    const void* q;
    const int32_t *cu_q, *lens;
    void* out;
    float* lse;
    void* ws;
    hipStream_t stream;
};

hipError_t launch_kv_write(const KvCall& c);
hipError_t launch_kv_read(const KvCall& c);
hipError_t launch_attn_prefill(const AttnCall& c);
hipError_t launch_attn_decode(const AttnDecodeCall& c);
hipError_t launch_rope(const RopeCall& c, bool cache);
hipError_t launch_attn_extend(const ExtendCall& c);

// Query rows (positions x heads of a KV head) a prefill workgroup handles, for the grid bound.
int attn_prefill_rows(int32_t d, int32_t dtype);
// Workspace of a checked prefill call with n > 0 (0: not split).
size_t attn_prefill_workspace(const gdn_attn_dims& d);
// Workspace of a decode call (0: not split), from the sizes the host knows.
size_t attn_decode_workspace(const gdn_kv_cache* c, int32_t h_q, int64_t max_len);
// Workspace of a checked extend call with rows (0: not split).
size_t attn_extend_workspace(const gdn_kv_cache& c, const gdn_extend_dims& d);

// A grid of at least `blocks` workgroups. A launch holds fewer than 2^32 threads in one dimension (more
// are not refused: workgroups are missing), so long ones go on in the second; workgroups have
// at most 1024 threads. Those whose block_index() is past the call's own leave.
constexpr int64_t kGridLine = INT64_C(1) << 21;

inline dim3 grid_of(int64_t blocks)
{
    return blocks <= kGridLine ? dim3((unsigned)blocks)
                               : dim3((unsigned)kGridLine, (unsigned)((blocks + kGridLine - 1) / kGridLine));
}

// ---------------------------------------------------------------- device helpers
// The workgroup's number in a grid of grid_of: below 2^31 + kGridLine.
__device__ __forceinline__ uint32_t block_index()
{
    return blockIdx.y * (uint32_t)kGridLine + blockIdx.x;
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Two floats as packed bf16 (round to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e)
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The factor of a scale byte: 2^(b - 127); byte 0, which no write makes, counts as 0.
__device__ __forceinline__ float scale_of(uint32_t b)
{
    return __uint_as_float(b << 23);
}

// The sequence a packed row belongs to: the last s in [0, n) with cu[s] <= row (0 if none), for a
// wave whose lanes' rows start at `first` and lie close together: 64 sequences are compared with
// the first row at a time, one a lane, and each lane goes on from there, in doubling steps over
// what may be many empty sequences and back by halves. Whatever cu holds, the answer is a valid
// sequence index. *end: cu of the next one.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, int first, int row, int* end)
{
    const int lane = threadIdx.x & 63;
    int s = 0;
    for (int span = n; span > 1;) {  // the sequence is in [s, s + span)
        const int step = (span + 63) / 64;
        const bool before = lane * step < span && (lane == 0 || cu[s + lane * step] <= first);
        const int x = 63 - __builtin_clzll(__ballot(before) | 1);  // the last lane not past the row
        s += x * step;
        span = span - x * step < step ? span - x * step : step;
    }
    *end = cu[s + 1];
    if (*end <= row && s + 1 < n) {
        int step = 1;
        for (; step < n - s && cu[s + step] <= row; step *= 2) s += step;
        for (int stop = step < n - s ? s + step : n; stop - s > 1;) {  // the sequence is in [s, stop)
            const int mid = s + (stop - s) / 2;
            if (cu[mid] <= row) s = mid;
            else stop = mid;
        }
        *end = cu[s + 1];
    }
    return s;
}

}  // namespace gdn
