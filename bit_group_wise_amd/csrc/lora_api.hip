// lora_api.hip -- the C ABI of low-rank adapters beside a weight (declared in
// include/q4.h): host-side argument validation and dispatch.  As in
// q4_api.hip, every check runs before the first HIP call.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_check.hpp"
#include "q4.h"
#include "q4_internal.hpp"

namespace {

using namespace q4;

// Sizes of a product and its adapters.
q4_status check_sizes(int64_t M, int64_t N, int64_t K, int adapters, int rank)
{
    if (M < 0 || N <= 0 || K <= 0 || adapters <= 0 || rank <= 0)
        return Q4_EINVAL;
    if (M > Q4_LORA_MAX_ROWS || N > INT32_MAX || K > Q4_GEMM_MAX_K || adapters > Q4_LORA_MAX_ADAPTERS)
        return Q4_EUNSUPPORTED;
    if (rank % 8 != 0 || rank > Q4_LORA_MAX_RANK)
        return Q4_EUNSUPPORTED;
    // the grids count tiles of at least 64 rows by 128 columns (M and the sides
    // below 2^44 / 2^13 tiles)
    if (M * N >= (int64_t)1 << 44 || M * K >= (int64_t)1 << 44)
        return Q4_EUNSUPPORTED;
    // an adapter's matrices are addressed with 32 bits
    if (N > INT32_MAX / (2 * rank) || K > INT32_MAX / (2 * rank))
        return Q4_EUNSUPPORTED;
    return Q4_OK;
}

q4_status check_lora(q4_format f, int g, q4_dtype act_t, int64_t M, const void *codes, const void *scales,
                     const void *zeros, int64_t N, int64_t K, const q4_lora *l)
{
    q4_status st = check_weight(f, g, codes, scales, zeros, N, K);
    if (st != Q4_OK)
        return st;
    if (!dtype_ok(act_t))
        return Q4_EUNSUPPORTED;
    if (!l || !l->a || !l->b)
        return Q4_EINVAL;
    st = check_sizes(M, N, K, l->adapters, l->rank);
    if (st != Q4_OK)
        return st;
    if (!aligned(l->a, 16) || !aligned(l->b, 16) || !aligned(l->scale, 4) || !aligned(l->ids, 4))
        return Q4_EALIGN;
    return Q4_OK;
}

}  // namespace

extern "C" {

size_t q4_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int adapters, int rank, int backward)
{
    if (check_sizes(M, N, K, adapters, rank) != Q4_OK || M == 0)
        return 0;
    return (size_t)lora_layout(M, N, K, adapters, rank, backward != 0).bytes;
}

q4_status q4_lora_gemm(q4_format f, int g, q4_dtype act_t, const void *x, int64_t M, const uint8_t *codes,
                       const void *scales, const uint8_t *zeros, int64_t N, int64_t K, const q4_lora *lora, void *y,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    q4_status st = check_lora(f, g, act_t, M, codes, scales, zeros, N, K, lora);
    if (st != Q4_OK || M == 0)
        return st;
    if (!x || !y || !workspace)
        return Q4_EINVAL;
    if (!aligned(x, 16) || !aligned(y, 2) || !aligned(workspace, 256))
        return Q4_EALIGN;
    const LoraLayout w = lora_layout(M, N, K, lora->adapters, lora->rank, 0);
    if (workspace_bytes < (size_t)w.bytes)
        return Q4_EINVAL;
    const hipStream_t s = (hipStream_t)stream;
    DownArgs d{};
    d.x = x;
    d.a = lora->a;
    d.scale = lora->scale;
    d.ids = lora->ids;
    d.h = workspace;
    d.sums = (float *)((char *)workspace + w.sums);
    d.rows = M;
    d.N = (int)N;
    d.K = (int)K;
    d.adapters = lora->adapters;
    d.rank = lora->rank;
    const hipError_t e = launch_down(act_t, d, w.plan, s);
    if (e != hipSuccess)
        return Q4_EHIP;
    const LoraArgs a{x,          M,         codes,          scales,     zeros, N, K, lora->b,
                     lora->ids, lora->adapters, lora->rank, d.h, w.plan.parts, y, w.out_parts, d.sums};
    switch (lora_kernel(M, N)) {
    case LoraKernel::skinny:
        return from_hip(launch_lora_skinny(f, g, act_t, a, s));
    case LoraKernel::tile64:
        return from_hip(launch_lora_tile64(f, g, act_t, a, s));
    case LoraKernel::tile128:
        return from_hip(launch_lora_tile128(f, g, act_t, a, s));
    default:
        return from_hip(launch_lora_tile256(f, g, act_t, a, s));
    }
}

q4_status q4_lora_backward(q4_format f, int g, q4_dtype act_t, const void *dy, const void *x, int64_t M,
                           const uint8_t *codes, const void *scales, const uint8_t *zeros, int64_t N, int64_t K,
                           const q4_lora *lora, void *dx, void *da, void *db, void *workspace, size_t workspace_bytes,
                           void *stream)
{
    q4_status st = check_lora(f, g, act_t, M, codes, scales, zeros, N, K, lora);
    if (st != Q4_OK)
        return st;
    if (N % 8 != 0 || N > Q4_GEMM_DX_MAX_N || N * (K / 2) > Q4_GEMV_CHAIN_MAX_CODES)
        return Q4_EUNSUPPORTED;
    if ((!da) != (!db) || (!dx && !da && M > 0))
        return Q4_EINVAL;
    if (!aligned(dx, 16) || !aligned(da, 16) || !aligned(db, 16))
        return Q4_EALIGN;
    if (M > 0) {
        if (!dy || (da && !x) || !workspace)
            return Q4_EINVAL;
        if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(workspace, 256))
            return Q4_EALIGN;
    }
    if (M == 0 && !da)  // (dX of no rows, which may be NULL)
        return Q4_OK;
    const LoraLayout w = lora_layout(M, N, K, lora->adapters, lora->rank, 1);
    if (M > 0 && workspace_bytes < (size_t)w.bytes)
        return Q4_EINVAL;
    const hipStream_t s = (hipStream_t)stream;
    DownArgs d{};
    d.x = da ? x : nullptr;
    d.dy = dy;
    d.a = lora->a;
    d.b = lora->b;
    d.scale = lora->scale;
    d.ids = lora->ids;
    d.h = workspace;
    d.u = (char *)workspace + w.u;
    d.sums = (float *)((char *)workspace + w.sums);
    d.rows = M;
    d.N = (int)N;
    d.K = (int)K;
    d.adapters = lora->adapters;
    d.rank = lora->rank;
    hipError_t e = M > 0 ? launch_down(act_t, d, w.plan, s) : hipSuccess;
    if (e == hipSuccess && dx && M > 0) {
        const LoraArgs a{dy,        M,         codes,          scales,     zeros, N, K, lora->a,
                         lora->ids, lora->adapters, lora->rank, d.u, w.plan.parts, dx, w.out_parts, d.sums};
        e = launch_lora_dx(f, g, act_t, a, s);
    }
    if (e == hipSuccess && da) {
        const GradArgs a{x, dy, lora->ids, (const uint16_t *)d.h, (const uint16_t *)d.u,
                         d.sums, M, (int)N, (int)K, lora->adapters, lora->rank,
                         w.splits, da, db};
        e = launch_lora_grad(act_t, a, s);
    }
    return from_hip(e);
}

}  // extern "C"
