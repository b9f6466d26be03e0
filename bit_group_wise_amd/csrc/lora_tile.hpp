// lora_tile.hpp -- y = x . What^T + h . B^T for many rows: gemm_tile.hpp's
// tiles of 16 Q4_LORA_MF rows, begun with the adapters' part.
#pragma once

#ifndef Q4_LORA_MF
#define Q4_LORA_MF 16
#endif

#include "gemm_tile.hpp"

namespace q4 {
namespace {

constexpr int kTileMF = Q4_LORA_MF;
constexpr int kTileRows = 16 * kTileMF;

template <int FMT, int ACT, int G>
__global__ __launch_bounds__(kBlock) void lora_tile_kernel(const uint16_t *__restrict__ x, int M,
                                                           const uint8_t *__restrict__ codes,
                                                           const void *__restrict__ scales,
                                                           const uint8_t *__restrict__ zeros, int N, int K, int mtiles,
                                                           int vec_y, LowRank low, uint16_t *__restrict__ y)
{
    Q4_GEMM_TILE_LDS(FMT, kTileMF);
    const Tile tile{(int)(blockIdx.x % (unsigned)mtiles) * kTileRows, M, (int)(blockIdx.x / (unsigned)mtiles) * BN,
                    N, 0, N, nullptr, 0};
    gemm_tile<FMT, ACT, G, kLora, kTileMF>(tile, x, codes, scales, zeros, K, vec_y, y, xs0, xs1, ptbl, &low);
}

template <int FMT, int G>
hipError_t launch_g(q4_dtype act_t, const LoraArgs &a, hipStream_t s)
{
    const int64_t mt = (a.M + kTileRows - 1) / kTileRows, nt = (a.N + BN - 1) / BN;
    if (mt * nt > 0x7fffffffll)
        return hipErrorInvalidValue;
    // 16-byte output stores need 16-byte rows
    const int vec_y = (a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0) ? 1 : 0;
    const LowRank low{nullptr, 0, (const uint16_t *)a.low, a.rank, a.adapters, a.M, a.ids, (const uint16_t *)a.w};
    const dim3 grid((unsigned)(mt * nt)), block(kBlock);
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((lora_tile_kernel<FMT, Q4_BF16, G>), grid, block, 0, s, (const uint16_t *)a.x, (int)a.M,
                           a.codes, a.scales, a.zeros, (int)a.N, (int)a.K, (int)mt, vec_y, low, (uint16_t *)a.y);
    else
        hipLaunchKernelGGL((lora_tile_kernel<FMT, Q4_F16, G>), grid, block, 0, s, (const uint16_t *)a.x, (int)a.M,
                           a.codes, a.scales, a.zeros, (int)a.N, (int)a.K, (int)mt, vec_y, low, (uint16_t *)a.y);
    return hipGetLastError();
}

template <int FMT>
hipError_t launch_fmt(int g, q4_dtype act_t, const LoraArgs &a, hipStream_t s)
{
    switch (g) {
    case 32:
        return launch_g<FMT, 32>(act_t, a, s);
    case 64:
        return launch_g<FMT, 64>(act_t, a, s);
    default:
        return launch_g<FMT, 128>(act_t, a, s);
    }
}

}  // namespace

hipError_t Q4_LORA_LAUNCH(q4_format f, int g, q4_dtype act_t, const LoraArgs &a, hipStream_t s)
{
    switch (f) {
    case Q4_NF4:
        return launch_fmt<Q4_NF4>(g, act_t, a, s);
    case Q4_FP4:
        return launch_fmt<Q4_FP4>(g, act_t, a, s);
    case Q4_NF4_DQ:
        return launch_fmt<Q4_NF4_DQ>(g, act_t, a, s);
    case Q4_INT4_SYM:
        return launch_fmt<Q4_INT4_SYM>(g, act_t, a, s);
    default:
        return launch_fmt<Q4_INT4_ASYM>(g, act_t, a, s);
    }
}

}  // namespace q4
