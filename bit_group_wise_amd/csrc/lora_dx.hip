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
    Q4_DX_TILE_LDS(FMT);
    const DxTile tile{(int)(blockIdx.x % (unsigned)mtiles) * (64 * WMF), M, (int)(blockIdx.x / (unsigned)mtiles) * TK, 0, N};
    dx_tile<FMT, ACT, kDxLora, WMF>(tile, dy, codes, scales, zeros, N, K, gshift, dx, ys, wt, ptbl, &low);
}

constexpr int kPartSteps = 8;  // least steps of TN rows of a part

template <int FMT, int ACT>
__global__ __launch_bounds__(kBlock) void lora_dx_part_kernel(const uint16_t *__restrict__ dy, int M,
                                                              const uint8_t *__restrict__ codes,
                                                              const void *__restrict__ scales,
                                                              const uint8_t *__restrict__ zeros, int N, int K,
                                                              int gshift, int mtiles, LowRank low,
                                                              float *__restrict__ sums)
{
    Q4_DX_TILE_LDS(FMT);
    const int steps = (N + TN - 1) / TN, part = blockIdx.y, parts = gridDim.y;
    const int first = steps * part / parts, last = steps * (part + 1) / parts;
    const DxTile tile{(int)(blockIdx.x % (unsigned)mtiles) * 64, M, (int)(blockIdx.x / (unsigned)mtiles) * TK, 0, N,
                      first, last - first, sums + (int64_t)part * M * K};
    dx_tile<FMT, ACT, kDxLoraPart, 1>(tile, dy, codes, scales, zeros, N, K, gshift, nullptr, ys, wt, ptbl, &low);
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
    if (a.out_parts > 1)
        return act_t == Q4_BF16 ? launch_ldx_parts<FMT, Q4_BF16>(a, gshift, s)
                                : launch_ldx_parts<FMT, Q4_F16>(a, gshift, s);
    if (tiles <= 64)
        return launch_ldx_rows<FMT, 1>(act_t, a, gshift, s);
    if (tiles <= 128)
        return launch_ldx_rows<FMT, 2>(act_t, a, gshift, s);
    return launch_ldx_rows<FMT, 4>(act_t, a, gshift, s);
}

}  // namespace

// Parts of N: as many as give every compute unit a workgroup, of at least
// kPartSteps steps.  dX alone in us, NF4 g 64, rank 16, whole / in parts of at
// least 16 / of 8 steps: 1 row, N 7640, K 1024 89 / 27 / 24; 16 rows of 4096 x
// 4096 53 / 26 / 23; 64 of 14336 x 4096 162 / 43 / 42; 16 of 2048 x 4096 32 / 25 /
// 21; 333 of 4096 x 2048 55 / 39 / 39; 333 of 1024 x 1024 (16 steps) 19.6 / 19.6 / 18.8.
int lora_dx_parts(int64_t M, int64_t N, int64_t K)
{
    const int64_t tiles = (M + 63) / 64 * ((K + TK - 1) / TK), steps = (N + TN - 1) / TN;
    const int64_t parts = tiles > 0 && tiles < 256 ? 256 / tiles : 1, most = steps / kPartSteps;
    return (int)(parts < most ? parts : (most > 1 ? most : 1));
}

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
