// experts_tile.hpp -- the product of many rows an expert, y[r] = x[index[r]] .
// What_e^T for the rows r of each expert e: gemm_tile.hpp's tiles over pieces
// of up to Q4_EXPERTS_MF blocks of 16 rows of one expert.  A shorter piece, an
// expert's last or only one, runs as a tile of three quarters, half or a
// quarter of the rows: its products take that much less.
#pragma once

#include "gemm_tile.hpp"
#include "rows.hpp"

namespace q4 {
namespace {

constexpr int kPieceMF = Q4_EXPERTS_MF;

template <int FMT, int ACT, int G>
__global__ __launch_bounds__(kBlock, Q4_EXPERTS_WAVES_PER_SIMD) void experts_tile_kernel(
    const uint16_t *__restrict__ x, int xrows, const int32_t *__restrict__ index,
    const int32_t *__restrict__ offsets, int rows, int experts, const uint8_t *__restrict__ codes,
    const void *__restrict__ scales, const uint8_t *__restrict__ zeros, int N, int K, int ntiles, int vec_y,
    uint16_t *__restrict__ y)
{
    Q4_GEMM_TILE_LDS(FMT, kPieceMF);
    int nt;
    const Piece p = find_piece_long_first<16 * kPieceMF>(offsets, experts, rows, blockIdx.x, ntiles, nt);
    if (p.group < 0)
        return;
    const Tile tile{p.lo, p.hi, nt * BN, N, (int64_t)p.group * N, (int64_t)experts * N, index, xrows};
    // the tile of as many quarters of its rows as the piece needs
    const int n = p.hi - p.lo;
#define Q4_TILE(MF) gemm_tile<FMT, ACT, G, kGather, MF>(tile, x, codes, scales, zeros, K, vec_y, y, xs0, xs1, ptbl)
    if (kPieceMF == 4 || n > 12 * kPieceMF) {
        Q4_TILE(kPieceMF);
    } else if constexpr (kPieceMF > 4) {
        if (n > 8 * kPieceMF) {
            Q4_TILE(kPieceMF * 3 / 4);
        } else if (kPieceMF == 8 || n > 4 * kPieceMF) {
            Q4_TILE(kPieceMF / 2);
        } else if constexpr (kPieceMF > 8) {
            Q4_TILE(kPieceMF / 4);
        }
    }
#undef Q4_TILE
}

template <int FMT, int G>
hipError_t launch_g(q4_dtype act_t, const ExpertsArgs &a, hipStream_t s)
{
    const int64_t ntiles = (a.N + BN - 1) / BN;
    const int64_t blocks = ntiles * most_pieces(a.rows, a.experts, 16 * kPieceMF);
    if (blocks > 0x7fffffffll)
        return hipErrorInvalidValue;
    // 16-byte output stores need 16-byte rows
    const int vec_y = (a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0) ? 1 : 0;
    const dim3 grid((unsigned)blocks), block(kBlock);
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((experts_tile_kernel<FMT, Q4_BF16, G>), grid, block, 0, s, (const uint16_t *)a.x,
                           (int)a.xrows, a.index, a.offsets, (int)a.rows, a.experts, a.codes, a.scales, a.zeros,
                           (int)a.N, (int)a.K, (int)ntiles, vec_y, (uint16_t *)a.y);
    else
        hipLaunchKernelGGL((experts_tile_kernel<FMT, Q4_F16, G>), grid, block, 0, s, (const uint16_t *)a.x,
                           (int)a.xrows, a.index, a.offsets, (int)a.rows, a.experts, a.codes, a.scales, a.zeros,
                           (int)a.N, (int)a.K, (int)ntiles, vec_y, (uint16_t *)a.y);
    return hipGetLastError();
}

template <int FMT>
hipError_t launch_fmt(int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s)
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

hipError_t Q4_EXPERTS_LAUNCH(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, hipStream_t s)
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
