// gemm.hip -- the prefill GEMM, y[M, N] = x[M, K] . What^T for any M: the grid
// of gemm_tile.hpp's tiles.
#include "gemm_tile.hpp"

namespace q4 {
namespace {

template <int FMT, int ACT, int G>
__global__ __launch_bounds__(kBlock) void gemm_kernel(const uint16_t *__restrict__ x, int M,
                                                      const uint8_t *__restrict__ codes,
                                                      const void *__restrict__ scales,
                                                      const uint8_t *__restrict__ zeros, int N,
                                                      int K, int mtiles, int vec_y,
                                                      uint16_t *__restrict__ y)
{
    Q4_GEMM_TILE_LDS(FMT, kMF);
    const Tile tile{(int)(blockIdx.x % (unsigned)mtiles) * BM, M, (int)(blockIdx.x / (unsigned)mtiles) * BN,
                    N, 0, N, nullptr, 0};
    gemm_tile<FMT, ACT, G, kDense, kMF>(tile, x, codes, scales, zeros, K, vec_y, y, xs0, xs1, ptbl);
}

template <int FMT, int G>
hipError_t launch_g(q4_dtype act_t, const void *x, int64_t M, const uint8_t *codes,
                    const void *scales, const uint8_t *zeros, int64_t N, int64_t K, void *y,
                    hipStream_t s)
{
    const int64_t mt = (M + BM - 1) / BM, nt = (N + BN - 1) / BN;
    if (mt * nt > 0x7fffffffll)
        return hipErrorInvalidValue;
    // 16-byte output stores need 16-byte rows
    const int vec_y = (N % 8 == 0 && ((uintptr_t)y & 15) == 0) ? 1 : 0;
    dim3 grid((unsigned)(mt * nt)), block(kBlock);
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((gemm_kernel<FMT, Q4_BF16, G>), grid, block, 0, s, (const uint16_t *)x,
                           (int)M, codes, scales, zeros, (int)N, (int)K, (int)mt, vec_y,
                           (uint16_t *)y);
    else
        hipLaunchKernelGGL((gemm_kernel<FMT, Q4_F16, G>), grid, block, 0, s, (const uint16_t *)x,
                           (int)M, codes, scales, zeros, (int)N, (int)K, (int)mt, vec_y,
                           (uint16_t *)y);
    return hipGetLastError();
}

template <int FMT>
hipError_t launch_fmt(int g, q4_dtype act_t, const void *x, int64_t M, const uint8_t *codes,
                      const void *scales, const uint8_t *zeros, int64_t N, int64_t K, void *y,
                      hipStream_t s)
{
    switch (g) {
    case 32:
        return launch_g<FMT, 32>(act_t, x, M, codes, scales, zeros, N, K, y, s);
    case 64:
        return launch_g<FMT, 64>(act_t, x, M, codes, scales, zeros, N, K, y, s);
    default:
        return launch_g<FMT, 128>(act_t, x, M, codes, scales, zeros, N, K, y, s);
    }
}

}  // namespace

hipError_t launch_gemm(q4_format f, int g, q4_dtype act_t, const void *x, int64_t M,
                       const uint8_t *codes, const void *scales, const uint8_t *zeros, int64_t N,
                       int64_t K, void *y, hipStream_t s)
{
    switch (f) {
    case Q4_NF4:
        return launch_fmt<Q4_NF4>(g, act_t, x, M, codes, scales, zeros, N, K, y, s);
    case Q4_FP4:
        return launch_fmt<Q4_FP4>(g, act_t, x, M, codes, scales, zeros, N, K, y, s);
    case Q4_NF4_DQ:
        return launch_fmt<Q4_NF4_DQ>(g, act_t, x, M, codes, scales, zeros, N, K, y, s);
    case Q4_INT4_SYM:
        return launch_fmt<Q4_INT4_SYM>(g, act_t, x, M, codes, scales, zeros, N, K, y, s);
    default:
        return launch_fmt<Q4_INT4_ASYM>(g, act_t, x, M, codes, scales, zeros, N, K, y, s);
    }
}

}  // namespace q4
