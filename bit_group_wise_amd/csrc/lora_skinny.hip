// lora_skinny.hip -- y = x . What^T + h . B^T for few rows: skinny.hpp's
// product, begun with the adapters' part.
#include "skinny.hpp"

namespace q4 {
namespace {

constexpr int kSkMaxRows = 64;  // activation rows per launch (4 blocks of 16)

// Waves for the adapters' part, as the registers allow: 8 with one block of
// activation rows (16 rows of 16 adapters of rank 16 beside 11008 x 4096 NF4 g
// 64: 22 -> 20 us for this kernel, 17 with their loads in flight across
// adapters), 4 with two, none with four.
constexpr int extra_waves(int mt) { return mt == 1 ? 8 : (mt == 2 ? 4 : 0); }

template <int FMT, int ACT, int RB, int MT>
__global__ __launch_bounds__(kSkBlock + 64 * extra_waves(MT)) void lora_skinny_kernel(const uint16_t *__restrict__ x, int M,
                                                               const uint8_t *__restrict__ codes,
                                                               const void *__restrict__ scales,
                                                               const uint8_t *__restrict__ zeros, int N, int K,
                                                               int gshift, LowRank low, uint16_t *__restrict__ y)
{
    const SkTask task{M, (int)(blockIdx.x * 16 * RB), N, 0, N, nullptr, 0};
    skinny_product<FMT, ACT, RB, MT, kSkLora, extra_waves(MT)>(task, x, codes, scales, zeros, K, gshift, y, &low);
}

template <int FMT, int RB, int MT>
hipError_t launch_ls_mt(q4_dtype act_t, const LoraArgs &a, const LowRank &low, int gshift, hipStream_t s)
{
    const dim3 grid((unsigned)((a.N + 16 * RB - 1) / (16 * RB))), block(kSkBlock + 64 * extra_waves(MT));
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((lora_skinny_kernel<FMT, Q4_BF16, RB, MT>), grid, block, 0, s, (const uint16_t *)a.x,
                           (int)a.M, a.codes, a.scales, a.zeros, (int)a.N, (int)a.K, gshift, low, (uint16_t *)a.y);
    else
        hipLaunchKernelGGL((lora_skinny_kernel<FMT, Q4_F16, RB, MT>), grid, block, 0, s, (const uint16_t *)a.x,
                           (int)a.M, a.codes, a.scales, a.zeros, (int)a.N, (int)a.K, gshift, low, (uint16_t *)a.y);
    return hipGetLastError();
}

template <int FMT, int RB>
hipError_t launch_ls_rb(q4_dtype act_t, const LoraArgs &a, const LowRank &low, int gshift, hipStream_t s)
{
    if (a.M <= 16)
        return launch_ls_mt<FMT, RB, 1>(act_t, a, low, gshift, s);
    if (a.M <= 32)
        return launch_ls_mt<FMT, RB, 2>(act_t, a, low, gshift, s);
    return launch_ls_mt<FMT, RB, 4>(act_t, a, low, gshift, s);
}

// Row blocks per workgroup as in gemv_mfma.hip.
template <int FMT>
hipError_t launch_ls_fmt(q4_dtype act_t, const LoraArgs &a, const LowRank &low, int gshift, hipStream_t s)
{
    const int64_t nb = (a.N + 15) / 16;
    const int64_t cus = device_cu_count();
    const int64_t rb = (nb + cus - 1) / cus;
    if (rb >= 4)
        return launch_ls_rb<FMT, 4>(act_t, a, low, gshift, s);
    if (rb == 3)
        return launch_ls_rb<FMT, 3>(act_t, a, low, gshift, s);
    if (rb == 2)
        return launch_ls_rb<FMT, 2>(act_t, a, low, gshift, s);
    return launch_ls_rb<FMT, 1>(act_t, a, low, gshift, s);
}

}  // namespace

hipError_t launch_lora_skinny(q4_format f, int g, q4_dtype act_t, const LoraArgs &a, hipStream_t s)
{
    const int gshift = g == 32 ? 5 : (g == 64 ? 6 : 7);
    for (int64_t m0 = 0; m0 < a.M; m0 += kSkMaxRows) {
        LoraArgs b = a;
        b.M = a.M - m0 < kSkMaxRows ? a.M - m0 : kSkMaxRows;
        b.x = (const uint16_t *)a.x + m0 * a.K;
        b.y = (uint16_t *)a.y + m0 * a.N;
        const LowRank low{(const float *)a.low + m0 * a.rank, a.parts, nullptr, a.rank, a.adapters, a.M,
                          a.ids ? a.ids + m0 : nullptr, (const uint16_t *)a.w};
        hipError_t e;
        switch (f) {
        case Q4_NF4:
            e = launch_ls_fmt<Q4_NF4>(act_t, b, low, gshift, s);
            break;
        case Q4_FP4:
            e = launch_ls_fmt<Q4_FP4>(act_t, b, low, gshift, s);
            break;
        case Q4_NF4_DQ:
            e = launch_ls_fmt<Q4_NF4_DQ>(act_t, b, low, gshift, s);
            break;
        case Q4_INT4_SYM:
            e = launch_ls_fmt<Q4_INT4_SYM>(act_t, b, low, gshift, s);
            break;
        default:
            e = launch_ls_fmt<Q4_INT4_ASYM>(act_t, b, low, gshift, s);
            break;
        }
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace q4
