// experts_skinny.hip -- the product of few rows an expert, y[r] = x[index[r]] .
// What_e^T for the rows r of each expert e and any K: skinny.hpp's product over
// pieces of up to 16 rows of one expert.
#include "rows.hpp"
#include "skinny.hpp"

namespace q4 {
namespace {

template <int FMT, int ACT, int RB>
__global__ __launch_bounds__(kSkBlock) void experts_skinny_kernel(
    const uint16_t *__restrict__ x, int xrows, const int32_t *__restrict__ index,
    const int32_t *__restrict__ offsets, int rows, int experts, const uint8_t *__restrict__ codes,
    const void *__restrict__ scales, const uint8_t *__restrict__ zeros, int N, int K, int gshift,
    int nblocks, uint16_t *__restrict__ y)
{
    int nb;
    const Piece p = find_piece<16>(offsets, experts, rows, blockIdx.x, nblocks, nb);
    if (p.group < 0)
        return;
    const SkTask task{p.hi - p.lo, nb * 16 * RB, N, (int64_t)p.group * N, (int64_t)experts * N,
                      index ? index + p.lo : nullptr, xrows};
    skinny_product<FMT, ACT, RB, 1, kSkGather>(task, index ? x : x + (int64_t)p.lo * K, codes, scales, zeros, K,
                                                gshift, y + (int64_t)p.lo * N);
}

// Two blocks of weight rows a workgroup: each reads x once for both.
template <int FMT>
hipError_t launch_es(q4_dtype act_t, const ExpertsArgs &a, int gshift, hipStream_t s)
{
    constexpr int RB = 2;
    const int64_t nblocks = (a.N + 16 * RB - 1) / (16 * RB);
    const int64_t blocks = nblocks * most_pieces(a.rows, a.experts, 16);
    if (blocks > 0x7fffffffll)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(kSkBlock);
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((experts_skinny_kernel<FMT, Q4_BF16, RB>), grid, block, 0, s,
                           (const uint16_t *)a.x, (int)a.xrows, a.index, a.offsets, (int)a.rows, a.experts, a.codes,
                           a.scales, a.zeros, (int)a.N, (int)a.K, gshift, (int)nblocks, (uint16_t *)a.y);
    else
        hipLaunchKernelGGL((experts_skinny_kernel<FMT, Q4_F16, RB>), grid, block, 0, s,
                           (const uint16_t *)a.x, (int)a.xrows, a.index, a.offsets, (int)a.rows, a.experts, a.codes,
                           a.scales, a.zeros, (int)a.N, (int)a.K, gshift, (int)nblocks, (uint16_t *)a.y);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_skinny(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s)
{
    const int gshift = g == 32 ? 5 : (g == 64 ? 6 : 7);
    switch (f) {
    case Q4_NF4:
        return launch_es<Q4_NF4>(act_t, a, gshift, s);
    case Q4_FP4:
        return launch_es<Q4_FP4>(act_t, a, gshift, s);
    case Q4_NF4_DQ:
        return launch_es<Q4_NF4_DQ>(act_t, a, gshift, s);
    case Q4_INT4_SYM:
        return launch_es<Q4_INT4_SYM>(act_t, a, gshift, s);
    default:
        return launch_es<Q4_INT4_ASYM>(act_t, a, gshift, s);
    }
}

}  // namespace q4
