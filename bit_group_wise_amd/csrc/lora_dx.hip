// lora_dx.hip -- dX = dY . What + u . A, the gradient through a frozen weight
// and the adapters beside it: gemm_dx_tile.hpp's tiles, begun with the
// adapters' part.
#include "gemm_dx_tile.hpp"

namespace q4 {
namespace {

template <int FMT, int ACT, int WMF>
__global__ __launch_bounds__(kBlock) void lora_dx_kernel(const uint16_t *__restrict__ dy, int M,
                                                         const uint8_t *__restrict__ codes,
                                                         const void *__restrict__ scales,
                                                         const uint8_t *__restrict__ zeros, int N, int K, int gshift,
                                                         int mtiles, LowRank low, uint16_t *__restrict__ dx)
{
    Q4_DX_TILE_LDS(FMT);
    const DxTile tile{(int)(blockIdx.x % (unsigned)mtiles) * (64 * WMF), M, (int)(blockIdx.x / (unsigned)mtiles) * TK, 0, N};
    dx_tile<FMT, ACT, kDxLora, WMF>(tile, dy, codes, scales, zeros, N, K, gshift, dx, ys, wt, ptbl, &low);
}

template <int FMT, int WMF>
hipError_t launch_ldx_rows(q4_dtype act_t, const LoraArgs &a, int gshift, hipStream_t s)
{
    const int64_t mtiles = (a.M + 64 * WMF - 1) / (64 * WMF), ktiles = (a.K + TK - 1) / TK;
    if (mtiles * ktiles > 0x7fffffffll)
        return hipErrorInvalidValue;
    const LowRank low{nullptr, 0, (const uint16_t *)a.low, a.rank, a.adapters, a.M, a.ids, (const uint16_t *)a.w};
    const dim3 grid((unsigned)(mtiles * ktiles)), block(kBlock);
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((lora_dx_kernel<FMT, Q4_BF16, WMF>), grid, block, 0, s, (const uint16_t *)a.x, (int)a.M,
                           a.codes, a.scales, a.zeros, (int)a.N, (int)a.K, gshift, (int)mtiles, low, (uint16_t *)a.y);
    else
        hipLaunchKernelGGL((lora_dx_kernel<FMT, Q4_F16, WMF>), grid, block, 0, s, (const uint16_t *)a.x, (int)a.M,
                           a.codes, a.scales, a.zeros, (int)a.N, (int)a.K, gshift, (int)mtiles, low, (uint16_t *)a.y);
    return hipGetLastError();
}

// Tiles of 256 rows, or of 128 or 64 where those too are one round of
// workgroups or less (256 compute units): a short tile takes less time, but a
// weight's column is dequantized once a tile.  dX alone, rank 16, in us, with
// tiles of 256 / 128 / 64 rows: 512 rows of 4096 x 4096 NF4 g 64 (64 tiles of
// 256) 80 / 64 / 57, 768 rows (96) 81 / 64 / 100, 1024 rows (128) 81 / 65 / 100;
// 333 rows of 1024 x 1024 (16) 30 / 23 / 20.
template <int FMT>
hipError_t launch_ldx(q4_dtype act_t, const LoraArgs &a, int gshift, hipStream_t s)
{
    const int64_t tiles = (a.M + 255) / 256 * ((a.K + TK - 1) / TK);
    if (tiles <= 64)
        return launch_ldx_rows<FMT, 1>(act_t, a, gshift, s);
    if (tiles <= 128)
        return launch_ldx_rows<FMT, 2>(act_t, a, gshift, s);
    return launch_ldx_rows<FMT, 4>(act_t, a, gshift, s);
}

}  // namespace

hipError_t launch_lora_dx(q4_format f, int g, q4_dtype act_t, const LoraArgs &a, hipStream_t s)
{
    const int gshift = g == 32 ? 5 : (g == 64 ? 6 : 7);
    switch (f) {
    case Q4_NF4:
        return launch_ldx<Q4_NF4>(act_t, a, gshift, s);
    case Q4_FP4:
        return launch_ldx<Q4_FP4>(act_t, a, gshift, s);
    case Q4_NF4_DQ:
        return launch_ldx<Q4_NF4_DQ>(act_t, a, gshift, s);
    case Q4_INT4_SYM:
        return launch_ldx<Q4_INT4_SYM>(act_t, a, gshift, s);
    default:
        return launch_ldx<Q4_INT4_ASYM>(act_t, a, gshift, s);
    }
}

}  // namespace q4
