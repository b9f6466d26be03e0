// lora_tile.hpp -- y = x . What^T + h . B^T for many rows: gemm_tile.hpp's
// tiles of 16 Q4_LORA_MF rows, begun with the adapters' part.  The shortest
// tiles may share out K: with few of them most of the card would idle while
// each goes through all of it.  A second kernel adds the parts' binary32 sums
// in order and rounds.
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

template <int FMT, int ACT, int G>
__global__ __launch_bounds__(kBlock) void lora_tile_part_kernel(const uint16_t *__restrict__ x, int M,
                                                                const uint8_t *__restrict__ codes,
                                                                const void *__restrict__ scales,
                                                                const uint8_t *__restrict__ zeros, int N, int K,
                                                                int mtiles, LowRank low, float *__restrict__ sums)
{
    Q4_GEMM_TILE_LDS(FMT, kTileMF);
    const int spans = (K + kSpanK - 1) / kSpanK, part = blockIdx.y, parts = gridDim.y;
    const int pitch = (N + 3) & ~3;
    const Tile tile{(int)(blockIdx.x % (unsigned)mtiles) * kTileRows, M, (int)(blockIdx.x / (unsigned)mtiles) * BN,
                    N, 0, N, nullptr, 0, spans * part / parts * kSpanK, spans * (part + 1) / parts * kSpanK,
                    sums + (int64_t)part * M * pitch, pitch};
    gemm_tile<FMT, ACT, G, kLoraPart, kTileMF>(tile, x, codes, scales, zeros, K, 0, nullptr, xs0, xs1, ptbl, &low);
}

// Four values of a row a thread (N4 fours a row).
template <int ACT>
__global__ __launch_bounds__(256) void lora_tile_join_kernel(const float *__restrict__ sums, int64_t fours, int N,
                                                             int N4, int parts, int vec_y, uint16_t *__restrict__ y)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= fours)
        return;
    f32x4 v = *(const f32x4 *)(sums + 4 * at);
    for (int i = 1; i < parts; ++i) {
        const f32x4 u = *(const f32x4 *)(sums + 4 * (i * fours + at));
        v = f32x4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
    }
    const int64_t m = at / N4;
    const int n = 4 * (int)(at - m * N4);
    const u32x2 p{pack2<ACT>(v[0], v[1]), pack2<ACT>(v[2], v[3])};
    uint16_t *to = y + m * N + n;
    if (vec_y) {
        *(u32x2 *)to = p;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < N)
                to[e] = (uint16_t)(p[e >> 1] >> (16 * (e & 1)));
    }
}

template <int FMT, int ACT, int G>
hipError_t launch_parts(const LoraArgs &a, hipStream_t s)
{
    const int64_t mt = (a.M + kTileRows - 1) / kTileRows, nt = (a.N + BN - 1) / BN;
    const LowRank low{nullptr, 0, (const uint16_t *)a.low, a.rank, a.adapters, a.M, a.ids, (const uint16_t *)a.w};
    hipLaunchKernelGGL((lora_tile_part_kernel<FMT, ACT, G>), dim3((unsigned)(mt * nt), (unsigned)a.out_parts),
                       dim3(kBlock), 0, s, (const uint16_t *)a.x, (int)a.M, a.codes, a.scales, a.zeros, (int)a.N,
                       (int)a.K, (int)mt, low, a.sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int64_t n4 = (a.N + 3) / 4, fours = a.M * n4;
    const int vec_y = (a.N % 4 == 0 && ((uintptr_t)a.y & 7) == 0) ? 1 : 0;
    hipLaunchKernelGGL((lora_tile_join_kernel<ACT>), dim3((unsigned)((fours + 255) / 256)), dim3(256), 0, s, a.sums,
                       fours, (int)a.N, (int)n4, a.out_parts, vec_y, (uint16_t *)a.y);
    return hipGetLastError();
}

template <int FMT, int G>
hipError_t launch_g(q4_dtype act_t, const LoraArgs &a, hipStream_t s)
{
    const int64_t mt = (a.M + kTileRows - 1) / kTileRows, nt = (a.N + BN - 1) / BN;
    if (mt * nt > 0x7fffffffll)
        return hipErrorInvalidValue;
    if constexpr (kTileMF == 4) {
        if (a.out_parts > 1)
            return act_t == Q4_BF16 ? launch_parts<FMT, Q4_BF16, G>(a, s) : launch_parts<FMT, Q4_F16, G>(a, s);
    }
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
