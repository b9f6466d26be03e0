// experts_api.hip -- the C ABI of the products through experts' weights
// (declared in include/q4.h): host-side argument validation and dispatch.  As
// in q4_api.hip, every check runs before the first HIP call.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_check.hpp"
#include "q4.h"
#include "q4_internal.hpp"
#include "rows.hpp"

namespace {

using namespace q4;

// Weight, groups and arrays of a product of `rows` rows.
q4_status check_experts(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a)
{
    if (a.experts <= 0 || a.N <= 0 || a.K <= 0)
        return Q4_EINVAL;
    if (a.experts > Q4_EXPERTS_MAX || a.N > INT32_MAX / a.experts)
        return Q4_EUNSUPPORTED;
    q4_status st = check_weight(f, g, a.codes, a.scales, a.zeros, a.experts * a.N, a.K);
    if (st != Q4_OK)
        return st;
    if (!dtype_ok(act_t) || a.K > Q4_GEMM_MAX_K)
        return Q4_EUNSUPPORTED;
    if (!a.offsets || a.rows < 0 || a.xrows < 0)
        return Q4_EINVAL;
    // row numbers fit 31 bits with room for a tile, and the largest grid 31
    if (a.rows > Q4_EXPERTS_MAX_ROWS || (a.N / 16 + 1) * most_pieces(a.rows, a.experts, 16) > INT32_MAX)
        return Q4_EUNSUPPORTED;
    if (!aligned(a.offsets, 4) || !aligned(a.index, 4))
        return Q4_EALIGN;
    if (a.rows == 0)
        return Q4_OK;
    if (!a.x || !a.y || (a.index ? a.xrows == 0 : a.xrows != a.rows))
        return Q4_EINVAL;
    // gathered rows are addressed with 32 bits from the first
    if (a.index && a.xrows > INT32_MAX / (2 * a.K))
        return Q4_EUNSUPPORTED;
    if (!aligned(a.x, 16) || !aligned(a.y, 2))
        return Q4_EALIGN;
    return Q4_OK;
}

}  // namespace

extern "C" {

q4_status q4_experts_gemm(q4_format f, int g, q4_dtype act_t, const void *x, int64_t x_rows, const int32_t *index,
                          const int32_t *offsets, int64_t rows, int experts, const uint8_t *codes,
                          const void *scales, const uint8_t *zeros, int64_t N, int64_t K, void *y, void *stream)
{
    const ExpertsArgs a{x, x_rows, index, offsets, rows, experts, codes, scales, zeros, N, K, y};
    const q4_status st = check_experts(f, g, act_t, a);
    if (st != Q4_OK || rows == 0)
        return st;
    return from_hip(launch_experts(f, g, act_t, a, (hipStream_t)stream));
}

q4_status q4_experts_gemm_dx(q4_format f, int g, q4_dtype act_t, const void *dy, const int32_t *offsets, int64_t rows,
                             int experts, const uint8_t *codes, const void *scales, const uint8_t *zeros, int64_t N,
                             int64_t K, void *dx, void *stream)
{
    const ExpertsArgs a{dy, rows, nullptr, offsets, rows, experts, codes, scales, zeros, N, K, dx};
    const q4_status st = check_experts(f, g, act_t, a);
    if (st != Q4_OK)
        return st;
    if (N % 8 != 0 || N > Q4_GEMM_DX_MAX_N || N * (K / 2) > Q4_GEMV_CHAIN_MAX_CODES ||
        (K + 127) / 128 * most_pieces(rows, experts, 64) > INT32_MAX)
        return Q4_EUNSUPPORTED;
    if (rows == 0)
        return Q4_OK;
    if (!aligned(dx, 16))
        return Q4_EALIGN;
    return from_hip(launch_experts_dx(f, g, act_t, a, (hipStream_t)stream));
}

}  // extern "C"


hipError_t q4::launch_experts(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s)
{
    switch (experts_kernel(a.rows, a.experts, a.N, a.K)) {
    case ExpertsKernel::stream1:
        return launch_experts_stream(f, g, act_t, a, 1, s);
    case ExpertsKernel::stream2:
        return launch_experts_stream(f, g, act_t, a, 2, s);
    case ExpertsKernel::skinny:
        return launch_experts_skinny(f, g, act_t, a, s);
    case ExpertsKernel::tile64:
        return launch_experts_tile64(f, g, act_t, a, s);
    case ExpertsKernel::tile128:
        return launch_experts_tile128(f, g, act_t, a, s);
    default:
        return launch_experts_tile256(f, g, act_t, a, s);
    }
}
