// gdn_checks.hpp -- host-side argument checks shared by the C entry points (not part of the
// C ABI): address ranges, alignment, overflow, status of a launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

struct Range {
    uintptr_t lo, hi;  // [lo, hi); empty when lo == hi
};

inline bool overlap(Range a, Range b)
{
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t* r)
{
    return !__builtin_mul_overflow(a, b, r);
}

inline Range range_of(const void* p, int64_t elems, size_t esize)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, p ? lo + (uintptr_t)elems * esize : lo};
}

inline bool aligned(const void* p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline gdn_status finish(hipError_t e)
{
    if (e == hipErrorInvalidConfiguration) return GDN_ERR_SHAPE;  // more workgroups than a launch holds
    return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // namespace gdn
