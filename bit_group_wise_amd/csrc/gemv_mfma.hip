// gemv_mfma.hip -- the skinny product of skinny.hpp for one weight (q4_gemv
// with 3 <= M <= 16, q4_gemm with M <= 96).
#include "skinny.hpp"

namespace q4 {
namespace {

constexpr int kSkMaxRows = 64;  // activation rows per launch (4 blocks of 16)

template <int FMT, int ACT, int RB, int MT>
__global__ __launch_bounds__(kSkBlock) void gemv_mfma_kernel(
    const uint16_t *__restrict__ x, int M, const uint8_t *__restrict__ codes,
    const void *__restrict__ scales, const uint8_t *__restrict__ zeros, int N, int K, int gshift,
    uint16_t *__restrict__ y)
{
    const SkTask task{M, (int)(blockIdx.x * 16 * RB), N, 0, N, nullptr, 0};
    skinny_product<FMT, ACT, RB, MT, kSkDense>(task, x, codes, scales, zeros, K, gshift, y);
}

template <int FMT, int RB, int MT>
hipError_t launch_sk_mt(q4_dtype act_t, const void *x, int M, const uint8_t *codes,
                        const void *scales, const uint8_t *zeros, int64_t N, int64_t K, int gshift,
                        void *y, hipStream_t s)
{
    const unsigned blocks = (unsigned)((N + 16 * RB - 1) / (16 * RB));
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((gemv_mfma_kernel<FMT, Q4_BF16, RB, MT>), dim3(blocks), dim3(kSkBlock),
                           0, s, (const uint16_t *)x, M, codes, scales, zeros, (int)N, (int)K,
                           gshift, (uint16_t *)y);
    else
        hipLaunchKernelGGL((gemv_mfma_kernel<FMT, Q4_F16, RB, MT>), dim3(blocks), dim3(kSkBlock),
                           0, s, (const uint16_t *)x, M, codes, scales, zeros, (int)N, (int)K,
                           gshift, (uint16_t *)y);
    return hipGetLastError();
}

// Activation blocks of 16 rows per launch: 1, 2 or 4 (M <= 16, 32, 64).
template <int FMT, int RB>
hipError_t launch_sk_rb(q4_dtype act_t, const void *x, int M, const uint8_t *codes,
                        const void *scales, const uint8_t *zeros, int64_t N, int64_t K, int gshift,
                        void *y, hipStream_t s)
{
    if (M <= 16)
        return launch_sk_mt<FMT, RB, 1>(act_t, x, M, codes, scales, zeros, N, K, gshift, y, s);
    if (M <= 32)
        return launch_sk_mt<FMT, RB, 2>(act_t, x, M, codes, scales, zeros, N, K, gshift, y, s);
    return launch_sk_mt<FMT, RB, 4>(act_t, x, M, codes, scales, zeros, N, K, gshift, y, s);
}

// Row blocks per workgroup: the blocks spread over the compute units
// (ceil(blocks / units), at most 4), so that no unit holds more than its
// share and x is read once for several blocks.  (With a number of
// workgroups between one and two per unit, the units holding two finish
// last: 688 blocks as 344 pairs ran a third longer than as 230 triples.)
template <int FMT>
hipError_t launch_sk_fmt(q4_dtype act_t, const void *x, int M, const uint8_t *codes,
                         const void *scales, const uint8_t *zeros, int64_t N, int64_t K,
                         int gshift, void *y, hipStream_t s)
{
    const int64_t nb = (N + 15) / 16;
    const int64_t cus = device_cu_count();
    const int64_t rb = (nb + cus - 1) / cus;
    if (rb >= 4)
        return launch_sk_rb<FMT, 4>(act_t, x, M, codes, scales, zeros, N, K, gshift, y, s);
    if (rb == 3)
        return launch_sk_rb<FMT, 3>(act_t, x, M, codes, scales, zeros, N, K, gshift, y, s);
    if (rb == 2)
        return launch_sk_rb<FMT, 2>(act_t, x, M, codes, scales, zeros, N, K, gshift, y, s);
    return launch_sk_rb<FMT, 1>(act_t, x, M, codes, scales, zeros, N, K, gshift, y, s);
}

}  // namespace

hipError_t launch_gemv_mfma(q4_format f, int g, q4_dtype act_t, const void *x, int64_t M,
                            const uint8_t *codes, const void *scales, const uint8_t *zeros,
                            int64_t N, int64_t K, void *y, hipStream_t s)
{
    const int gshift = g == 32 ? 5 : (g == 64 ? 6 : 7);
    // up to kSkMaxRows activation rows per launch; more run as consecutive
    // launches over row slices of x and y (each reads every weight once)
    for (int64_t m0 = 0; m0 < M; m0 += kSkMaxRows) {
        const int mc = (int)(M - m0 < kSkMaxRows ? M - m0 : kSkMaxRows);
        const void *xc = (const uint16_t *)x + m0 * K;
        void *yc = (uint16_t *)y + m0 * N;
        hipError_t e;
        switch (f) {
        case Q4_NF4:
            e = launch_sk_fmt<Q4_NF4>(act_t, xc, mc, codes, scales, zeros, N, K, gshift, yc, s);
            break;
        case Q4_FP4:
            e = launch_sk_fmt<Q4_FP4>(act_t, xc, mc, codes, scales, zeros, N, K, gshift, yc, s);
            break;
        case Q4_NF4_DQ:
            e = launch_sk_fmt<Q4_NF4_DQ>(act_t, xc, mc, codes, scales, zeros, N, K, gshift, yc, s);
            break;
        case Q4_INT4_SYM:
            e = launch_sk_fmt<Q4_INT4_SYM>(act_t, xc, mc, codes, scales, zeros, N, K, gshift, yc, s);
            break;
        default:
            e = launch_sk_fmt<Q4_INT4_ASYM>(act_t, xc, mc, codes, scales, zeros, N, K, gshift, yc, s);
            break;
        }
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace q4
