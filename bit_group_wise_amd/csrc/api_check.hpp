// api_check.hpp -- argument checks that the entry points share (host code).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "q4.h"
#include "q4_common.hpp"

namespace q4 {

inline bool format_ok(q4_format f)
{
    return f == Q4_NF4 || f == Q4_INT4_SYM || f == Q4_INT4_ASYM || f == Q4_NF4_DQ || f == Q4_FP4;
}
inline bool dtype_ok(q4_dtype t) { return t == Q4_F16 || t == Q4_BF16; }
inline bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }
inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Checks shared by every entry point that takes a quantized weight.
inline q4_status check_weight(q4_format f, int g, const void *codes, const void *scales, const void *zeros, int64_t N,
                              int64_t K)
{
    if (!format_ok(f) || !group_ok(g))
        return Q4_EUNSUPPORTED;
    if (!codes || !scales)
        return Q4_EINVAL;
    if (N <= 0 || K <= 0 || K % g != 0)
        return Q4_EINVAL;
    if ((f == Q4_INT4_ASYM) != (zeros != nullptr))
        return Q4_EINVAL;
    const uintptr_t sa = f == Q4_NF4_DQ ? 16 : (f32_absmax(f) ? 4 : 2);
    if (!aligned(codes, 16) || !aligned(scales, sa))
        return Q4_EALIGN;
    return Q4_OK;
}

inline q4_status from_hip(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_EHIP; }

}  // namespace q4
