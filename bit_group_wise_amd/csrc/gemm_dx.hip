// gemm_dx.hip -- the backward product dX[M, K] = dY[M, N] . What[N, K]: the
// grid of gemm_dx_tile.hpp's tiles.
#include "gemm_dx_tile.hpp"

namespace q4 {
namespace {

template <int FMT, int ACT>
__global__ __launch_bounds__(kBlock) void gemm_dx_kernel(const uint16_t *__restrict__ dy, int M,
                                                         const uint8_t *__restrict__ codes,
                                                         const void *__restrict__ scales,
                                                         const uint8_t *__restrict__ zeros, int N,
                                                         int K, int gshift, int mtiles,
                                                         uint16_t *__restrict__ dx)
{
    Q4_DX_TILE_LDS(FMT);
    const DxTile tile{(int)(blockIdx.x % (unsigned)mtiles) * TM, M, (int)(blockIdx.x / (unsigned)mtiles) * TK, 0, N};
    dx_tile<FMT, ACT, kDxDense, kWMF>(tile, dy, codes, scales, zeros, N, K, gshift, dx, ys, wt, ptbl);
}

template <int FMT>
hipError_t launch_dx_fmt(q4_dtype act_t, int gshift, const void *dy, int64_t M,
                         const uint8_t *codes, const void *scales, const uint8_t *zeros, int64_t N,
                         int64_t K, void *dx, hipStream_t s)
{
    const int mtiles = (int)((M + TM - 1) / TM);
    const int64_t ktiles = (K + TK - 1) / TK;
    const dim3 grid((unsigned)(mtiles * ktiles)), block(kBlock);
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((gemm_dx_kernel<FMT, Q4_BF16>), grid, block, 0, s, (const uint16_t *)dy,
                           (int)M, codes, scales, zeros, (int)N, (int)K, gshift, mtiles,
                           (uint16_t *)dx);
    else
        hipLaunchKernelGGL((gemm_dx_kernel<FMT, Q4_F16>), grid, block, 0, s, (const uint16_t *)dy,
                           (int)M, codes, scales, zeros, (int)N, (int)K, gshift, mtiles,
                           (uint16_t *)dx);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_dx(q4_format f, int g, q4_dtype act_t, const void *dy, int64_t M,
                          const uint8_t *codes, const void *scales, const uint8_t *zeros,
                          int64_t N, int64_t K, void *dx, hipStream_t s)
{
    const int gshift = g == 32 ? 5 : (g == 64 ? 6 : 7);
    switch (f) {
    case Q4_NF4:
        return launch_dx_fmt<Q4_NF4>(act_t, gshift, dy, M, codes, scales, zeros, N, K, dx, s);
    case Q4_FP4:
        return launch_dx_fmt<Q4_FP4>(act_t, gshift, dy, M, codes, scales, zeros, N, K, dx, s);
    case Q4_NF4_DQ:
        return launch_dx_fmt<Q4_NF4_DQ>(act_t, gshift, dy, M, codes, scales, zeros, N, K, dx, s);
    case Q4_INT4_SYM:
        return launch_dx_fmt<Q4_INT4_SYM>(act_t, gshift, dy, M, codes, scales, zeros, N, K, dx, s);
    default:
        return launch_dx_fmt<Q4_INT4_ASYM>(act_t, gshift, dy, M, codes, scales, zeros, N, K, dx, s);
    }
}

}  // namespace q4
