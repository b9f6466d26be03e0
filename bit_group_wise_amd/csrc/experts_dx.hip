// experts_dx.hip -- the gradient through experts' weights, dX[r] = dY[r] .
// What_e for the rows r of each expert e: gemm_dx_tile.hpp's tiles over pieces
// of up to 256 rows of one expert, shorter pieces as tiles of fewer rows.
#include "gemm_dx_tile.hpp"
#include "rows.hpp"

namespace q4 {
namespace {

// WMF: pieces of up to 64 WMF rows.
template <int FMT, int ACT, int WMF>
__global__ __launch_bounds__(kBlock) void experts_dx_kernel(
    const uint16_t *__restrict__ dy, const int32_t *__restrict__ offsets, int rows, int experts,
    const uint8_t *__restrict__ codes, const void *__restrict__ scales, const uint8_t *__restrict__ zeros, int N,
    int K, int gshift, int ktiles, uint16_t *__restrict__ dx)
{
    Q4_DX_TILE_LDS(FMT);
    int kt;
    const Piece p = find_piece_long_first<64 * WMF>(offsets, experts, rows, blockIdx.x, ktiles, kt);
    if (p.group < 0)
        return;
    const DxTile tile{p.lo, p.hi, kt * TK, (int64_t)p.group * N, (int64_t)experts * N};
    // the tile of as many quarters of its rows as the piece needs
    const int n = p.hi - p.lo;
#define Q4_TILE(MF) dx_tile<FMT, ACT, kDxGroup, MF>(tile, dy, codes, scales, zeros, N, K, gshift, dx, ys, wt, ptbl)
    if (WMF == 4 && n > 192)
        Q4_TILE(4);
    else if (WMF == 4 && n > 128)
        Q4_TILE(3);
    else if (WMF >= 2 && n > 64)
        Q4_TILE(2);
    else
        Q4_TILE(1);
#undef Q4_TILE
}

template <int FMT, int WMF>
hipError_t launch_edx_rows(q4_dtype act_t, const ExpertsArgs &a, int gshift, hipStream_t s)
{
    const int64_t ktiles = (a.K + TK - 1) / TK;
    const int64_t blocks = ktiles * most_pieces(a.rows, a.experts, 64 * WMF);
    if (blocks > 0x7fffffffll)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(kBlock);
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((experts_dx_kernel<FMT, Q4_BF16, WMF>), grid, block, 0, s, (const uint16_t *)a.x, a.offsets,
                           (int)a.rows, a.experts, a.codes, a.scales, a.zeros, (int)a.N, (int)a.K, gshift,
                           (int)ktiles, (uint16_t *)a.y);
    else
        hipLaunchKernelGGL((experts_dx_kernel<FMT, Q4_F16, WMF>), grid, block, 0, s, (const uint16_t *)a.x, a.offsets,
                           (int)a.rows, a.experts, a.codes, a.scales, a.zeros, (int)a.N, (int)a.K, gshift,
                           (int)ktiles, (uint16_t *)a.y);
    return hipGetLastError();
}

template <int FMT>
hipError_t launch_edx(q4_dtype act_t, const ExpertsArgs &a, int gshift, hipStream_t s)
{
    return experts_dx_rows(a.rows, a.K) == 64 ? launch_edx_rows<FMT, 1>(act_t, a, gshift, s)
                                              : launch_edx_rows<FMT, 4>(act_t, a, gshift, s);
}

}  // namespace

hipError_t launch_experts_dx(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s)
{
    const int gshift = g == 32 ? 5 : (g == 64 ? 6 : 7);
    switch (f) {
    case Q4_NF4:
        return launch_edx<Q4_NF4>(act_t, a, gshift, s);
    case Q4_FP4:
        return launch_edx<Q4_FP4>(act_t, a, gshift, s);
    case Q4_NF4_DQ:
        return launch_edx<Q4_NF4_DQ>(act_t, a, gshift, s);
    case Q4_INT4_SYM:
        return launch_edx<Q4_INT4_SYM>(act_t, a, gshift, s);
    default:
        return launch_edx<Q4_INT4_ASYM>(act_t, a, gshift, s);
    }
}

}  // namespace q4
