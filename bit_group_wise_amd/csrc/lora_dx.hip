// lora_dx.hip -- dX = dY . What + u . A, the gradient through a frozen weight
// and the adapters beside it: gemm_dx_tile.hpp's tiles, begun with the
// adapters' part.  A few tiles, each a workgroup that goes through all N weight
// rows, leave most of the card idle, so there N is cut into parts, whose
// binary32 sums a second kernel adds in order and rounds.
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
    Q4_DX_LORA_LDS(FMT);
    const DxTile tile{(int)(blockIdx.x % (unsigned)mtiles) * (64 * WMF), M, (int)(blockIdx.x / (unsigned)mtiles) * TK, 0, N};
    dx_tile<FMT, ACT, kDxLora, WMF>(tile, dy, codes, scales, zeros, N, K, gshift, dx, ys, wt, ptbl, us, &low);
}

template <int FMT, int ACT>
__global__ __launch_bounds__(kBlock) void lora_dx_part_kernel(const uint16_t *__restrict__ dy, int M,
                                                              const uint8_t *__restrict__ codes,
                                                              const void *__restrict__ scales,
                                                              const uint8_t *__restrict__ zeros, int N, int K,
                                                              int gshift, int mtiles, LowRank low,
                                                              float *__restrict__ sums)
{
    Q4_DX_LORA_LDS(FMT);
    const int steps = (N + TN - 1) / TN, part = blockIdx.y, parts = gridDim.y;
    const int first = steps * part / parts, last = steps * (part + 1) / parts;
    const DxTile tile{(int)(blockIdx.x % (unsigned)mtiles) * 64, M, (int)(blockIdx.x / (unsigned)mtiles) * TK, 0, N,
                      first, last - first, sums + (int64_t)part * M * K};
    dx_tile<FMT, ACT, kDxLoraPart, 1>(tile, dy, codes, scales, zeros, N, K, gshift, nullptr, ys, wt, ptbl, us, &low);
}

template <int ACT>
__global__ __launch_bounds__(256) void lora_dx_join_kernel(const float *__restrict__ sums, int64_t size, int parts,
                                                           uint16_t *__restrict__ dx)
{
    const int64_t at = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (at >= size)
        return;
    f32x4 v = *(const f32x4 *)(sums + at);
    for (int i = 1; i < parts; ++i) {
        const f32x4 u = *(const f32x4 *)(sums + i * size + at);
        v = f32x4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
    }
    *(u32x2 *)(dx + at) = u32x2{pack2<ACT>(v[0], v[1]), pack2<ACT>(v[2], v[3])};
}

template <int FMT, int ACT>
hipError_t launch_ldx_parts(const LoraArgs &a, int gshift, hipStream_t s)
{
    const int64_t mtiles = (a.M + 63) / 64, ktiles = (a.K + TK - 1) / TK;
    const LowRank low{nullptr, 0, (const uint16_t *)a.low, a.rank, a.adapters, a.M, a.ids, (const uint16_t *)a.w};
    hipLaunchKernelGGL((lora_dx_part_kernel<FMT, ACT>), dim3((unsigned)(mtiles * ktiles), (unsigned)a.out_parts),
                       dim3(kBlock), 0, s, (const uint16_t *)a.x, (int)a.M, a.codes, a.scales, a.zeros, (int)a.N,
                       (int)a.K, gshift, (int)mtiles, low, a.sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int64_t size = a.M * a.K;
    hipLaunchKernelGGL((lora_dx_join_kernel<ACT>), dim3((unsigned)((size / 4 + 255) / 256)), dim3(256), 0, s, a.sums,
                       size, a.out_parts, (uint16_t *)a.y);
    return hipGetLastError();
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

template <int FMT>
hipError_t launch_ldx(q4_dtype act_t, const LoraArgs &a, int gshift, hipStream_t s)
{
    if (a.out_parts > 1)
        return act_t == Q4_BF16 ? launch_ldx_parts<FMT, Q4_BF16>(a, gshift, s)
                                : launch_ldx_parts<FMT, Q4_F16>(a, gshift, s);
    switch (lora_dx_rows(a.M, a.K)) {
    case 64:
        return launch_ldx_rows<FMT, 1>(act_t, a, gshift, s);
    case 128:
        return launch_ldx_rows<FMT, 2>(act_t, a, gshift, s);
    default:
        return launch_ldx_rows<FMT, 4>(act_t, a, gshift, s);
    }
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
