// experts_stream.hip -- the product of few rows an expert, y[r] = x[index[r]] .
// What_e^T for the rows r of each expert e, for K up to 4096: resident
// workgroups that stream row block after row block of the weights.
//
// Method as skinny.hpp (weights dequantized to the 16-bit type, 16x16x32
// matrix-core products, binary32 sums).  With few rows the product is bound by
// reading the asked experts' weights once; what a grid of one workgroup per
// block of weight rows loses on that is latency: offsets, index, first loads
// and the joining of the sums come one after another and outlast the few steps
// of K that a wave then has (64 experts of 2048 x 4096 INT4-asym g 32, 512
// rows: 161 us, 1.9 TB/s).
//  * The launch's work is all blocks of 16 weight rows of all pieces (up to
//    16 MT rows of one expert), one after another; workgroup i of G takes an
//    equal share of consecutive ones, so most of its blocks belong to one
//    piece.
//  * The waves (16 or 8) split K: lane quad q of wave w has the 32 S values from
//    32 S (4 w + q), in S steps of 32 (S = 1, 2 or 4).  Its part of x stays in registers
//    for all blocks of a piece.
//  * A block's codes and scales are 16 S contiguous bytes and S * 32 / g scales
//    a lane; the loads of the next two or three blocks are in flight while one
//    is dequantized and multiplied.
//  * The waves' partial 16 x 16 tiles of a few blocks meet in LDS at once (two
//    buffers, one barrier), and a wave each sums one, in wave order.
#include "q4_common.hpp"
#include "q4_internal.hpp"
#include "q4_mfma.hpp"
#include "rows.hpp"

namespace q4 {
namespace {

constexpr uint32_t kPast = 0x80000000u;

// A lane's share of a block of 16 weight rows: S times 32 codes of one row and
// their groups' scales as stored (and zero-points, from the byte of the first;
// NF4_DQ: the constants of the first group's run and the next).
template <int FMT, int G, int S>
struct Share {
    static constexpr int ng = S * 32 / G > 0 ? S * 32 / G : 1;  // groups
    u32x4 c[S];
    static constexpr int words = f32_absmax(FMT) ? ng : (FMT == Q4_NF4_DQ || ng == 1 ? 1 : ng / 2);
    uint32_t s[words];
    uint32_t z[FMT == Q4_NF4_DQ ? 2 : 1];
    int first;  // place of the first group: asym its nibble in z, NF4_DQ its number in its run
};

template <int FMT, int ACT, int G, int WAVES, int S, int MT>
__global__ __launch_bounds__(64 * WAVES) void experts_stream_kernel(
    const uint16_t *__restrict__ x, int xrows, const int32_t *__restrict__ index,
    const int32_t *__restrict__ offsets, int rows, int experts, const uint8_t *__restrict__ codes,
    const void *__restrict__ scales, const uint8_t *__restrict__ zeros, int N, int K, int vec_y,
    uint16_t *__restrict__ y)
{
    constexpr int LF = level_fmt(FMT);
    constexpr int ss = f32_absmax(FMT) ? 4 : (FMT == Q4_NF4_DQ ? 1 : 2);
    constexpr int kRing = WAVES == 16 ? 2 : 3;  // blocks in flight: as the registers hold
    constexpr int ng = Share<FMT, G, S>::ng;
    __shared__ float2 ptbl[LF == Q4_NF4 ? 256 : 1];
    constexpr int kTiles = WAVES == 16 ? 4 : 8;  // whose sums meet at once
    constexpr int kBatch = kTiles / MT;          // ... and blocks
    __shared__ f32x4 part[2][WAVES][kTiles][64];

    const int lane = threadIdx.x & 63;
    const int wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int Gn = K / G;
    const int row_bytes = K >> 1;
    if constexpr (LF == Q4_NF4) {
        if (threadIdx.x < 256)
            ptbl[threadIdx.x] = float2{level_entry<FMT>(threadIdx.x & 15), level_entry<FMT>(threadIdx.x >> 4)};
        __syncthreads();
    }
    const int nblocks = (N + 15) / 16;
    GroupLane lanes{};
    int upto = 0;
    const int total = count_pieces<16 * MT>(offsets, experts, rows, lanes, upto);
    const int64_t all = (int64_t)total * nblocks;
    const int64_t begin = all * blockIdx.x / gridDim.x, end = all * (blockIdx.x + 1) / gridDim.x;
    const int k0 = 32 * S * (4 * wave + q);  // the lane's first k
    // Offsets of what is not there get their highest bit set, past every view
    // (a select would become a branch with a load and a full wait of its own):
    // by the lane's step past K, and by the step past the workgroup's blocks.
    uint32_t past[S];
#pragma unroll
    for (int s = 0; s < S; ++s)
        past[s] = k0 + 32 * s < K ? 0u : kPast;

    int turn = 0, slot = 0;  // batches done (the LDS buffer), and blocks of this one
    for (int64_t at = begin; at < end;) {
        // the piece, and its blocks nb .. nend - 1
        const int pi = (int)(at / nblocks), nb = (int)(at % nblocks);
        const int nend = (int)min((int64_t)nblocks, nb + (end - at));
        at += nend - nb;
        const Piece p = experts > 64 ? piece_at<16 * MT>(offsets, experts, rows, pi)
                                     : piece_in<16 * MT>(lanes, upto, 0, pi);
        const int M = p.hi - p.lo;
        const int64_t w0 = (int64_t)p.group * N;  // the expert's first weight row

        // the lane's part of x: row r of each 16, k0 .. k0 + 32 S - 1
        u32x4 xf[MT][S][4];
        {
            const __amdgpu_buffer_rsrc_t xr = index ? buffer_view(x, (int64_t)xrows * K * 2)
                                                    : buffer_view(x + (int64_t)p.lo * K, (int64_t)M * K * 2);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                int m = 16 * mt + r;
                bool in = m < M;
                if (index) {
                    m = in ? index[p.lo + m] : 0;
                    in = in && (uint32_t)m < (uint32_t)xrows;
                }
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        xf[mt][s][d] = __builtin_amdgcn_raw_buffer_load_b128(
                            xr, (int)((2u * (uint32_t)(m * K + k0 + 32 * s + 8 * d)) | past[s] | (in ? 0u : kPast)), 0,
                            0);
            }
        }
        const __amdgpu_buffer_rsrc_t cr = buffer_view(codes + w0 * row_bytes, (int64_t)N * row_bytes);
        // scales and zero-points: to the end of the padded arrays, so that no word
        // of a meaningful entry is cut by a view's end (which would make it zero)
        const int64_t g0 = w0 * Gn, groups = (int64_t)experts * N * Gn;  // flat number of the expert's first group, and of all
        const int64_t s_total = padded_meta_bytes(FMT == Q4_NF4_DQ ? dq_scales_bytes(groups) : groups * ss);
        const __amdgpu_buffer_rsrc_t sr = buffer_view((const char *)scales + g0 * ss, s_total - g0 * ss);
        __amdgpu_buffer_rsrc_t zr = sr;
        if constexpr (FMT == Q4_INT4_ASYM)
            zr = buffer_view(zeros + (g0 >> 1), padded_meta_bytes((groups + 1) / 2) - (g0 >> 1));
        if constexpr (FMT == Q4_NF4_DQ)
            zr = buffer_view((const char *)scales + dq_s2_offset(groups) + 4 * (g0 / kDqRun),
                         s_total - dq_s2_offset(groups) - 4 * (g0 / kDqRun));

        auto load = [&](Share<FMT, G, S> &sh, int b) {
            const uint32_t n = 16 * b + r, none = b < nend ? 0u : kPast;  // (rows past N lie past the views)
#pragma unroll
            for (int s = 0; s < S; ++s)
                sh.c[s] = __builtin_amdgcn_raw_buffer_load_b128(
                    cr, (int)((n * row_bytes + ((k0 + 32 * s) >> 1)) | past[s] | none), 0, 0);
            const uint32_t gi = n * Gn + k0 / G, off = past[0] | none;
            // (a row's last share may end before its S steps do: what its scales
            // then hold belongs to the next row and meets codes and x of zero)
            if constexpr (ss == 4) {
                if constexpr (ng == 4) {
                    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(sr, (int)(4 * gi | off), 0, 0);
                    sh.s[0] = v[0], sh.s[1] = v[1], sh.s[2] = v[2], sh.s[3] = v[3];
                } else if constexpr (ng == 2) {
                    const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(sr, (int)(4 * gi | off), 0, 0);
                    sh.s[0] = v[0], sh.s[1] = v[1];
                } else {
                    sh.s[0] = __builtin_amdgcn_raw_buffer_load_b32(sr, (int)(4 * gi | off), 0, 0);
                }
            } else if constexpr (ss == 2 && ng > 1) {  // pairs, two to a word
#pragma unroll
                for (int e = 0; e < ng / 2; ++e)
                    sh.s[e] = __builtin_amdgcn_raw_buffer_load_b32(sr, (int)((2 * gi + 4 * e) | off), 0, 0);
            } else if constexpr (ss == 2) {
                sh.s[0] = __builtin_amdgcn_raw_buffer_load_b16(sr, (int)(2 * gi | off), 0, 0);
            } else if constexpr (ng == 4) {
                sh.s[0] = __builtin_amdgcn_raw_buffer_load_b32(sr, (int)(gi | off), 0, 0);
            } else if constexpr (ng == 2) {
                sh.s[0] = __builtin_amdgcn_raw_buffer_load_b16(sr, (int)(gi | off), 0, 0);
            } else {
                sh.s[0] = __builtin_amdgcn_raw_buffer_load_b8(sr, (int)(gi | off), 0, 0);
            }
            if constexpr (FMT == Q4_INT4_ASYM) {
                const uint32_t gz = (uint32_t)(g0 & 1) + gi;
                sh.first = (int)(gz & 1);
                sh.z[0] = __builtin_amdgcn_raw_buffer_load_b32(zr, (int)(gz >> 1 | off), 0, 0);
            } else if constexpr (FMT == Q4_NF4_DQ) {
                const uint32_t gr = (uint32_t)(g0 % kDqRun) + gi;
                sh.first = (int)(gr % kDqRun);
                const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(zr, (int)(4 * (gr / kDqRun) | off), 0, 0);
                sh.z[0] = v[0], sh.z[1] = v[1];
            }
        };

        Share<FMT, G, S> ring[kRing];
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // (in the blocks' order, or the first wait is for all)
            load(ring[i], nb + i);
        }
        __builtin_amdgcn_sched_barrier(0);
        for (int b0 = nb; b0 < nend; b0 += kRing) {
#pragma unroll
            for (int i = 0; i < kRing; ++i) {
                const int b = b0 + i;
                if (b >= nend)
                    break;
                Share<FMT, G, S> &sh = ring[i];
                f32x4 acc[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    acc[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    constexpr int per = G / 32 > S ? S : G / 32;  // steps of one group
                    const int e = s / per;
                    float sc, bias = 0.0f;
                    if constexpr (f32_absmax(FMT)) {
                        sc = std::bit_cast<float>(sh.s[e]);
                    } else if constexpr (FMT == Q4_NF4_DQ) {
                        sc = keep_f32((float)((sh.s[0] >> (8 * e)) & 0xffu) *
                                      std::bit_cast<float>(sh.first + e >= kDqRun ? sh.z[1] : sh.z[0]));
                    } else {
                        sc = h2f((ng > 1 ? sh.s[e / 2] >> (16 * (e & 1)) : sh.s[0]) & 0xffffu);
                        bias = FMT == Q4_INT4_SYM ? -8.0f * sc
                                                  : -(float)((sh.z[0] >> (4 * (sh.first + e))) & 0xfu) * sc;
                    }
                    const bool in = k0 + 32 * s < K;
                    sc = in ? sc : 0.0f;
                    bias = in ? bias : 0.0f;
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        float2 lp[4];
                        if constexpr (LF == Q4_NF4) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                lp[j] = ptbl[(sh.c[s][d] >> (8 * j)) & 0xffu];
                        }
                        const u32x4 wf = dequant8<FMT, ACT>(sh.c[s][d], sc, bias, lp);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            acc[mt] = mfma<ACT>(wf, xf[mt][s][d], acc[mt]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                load(sh, b + kRing);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    part[turn & 1][wave][slot * MT + mt][lane] = acc[mt];
                if (++slot < kBatch && b + 1 < nend)
                    continue;
                __syncthreads();
                // tile `wave` of the batch: block b + 1 - slot + wave / MT (buffer
                // turn & 1 is written again only behind the next barrier)
                if (wave < slot * MT) {
                    f32x4 v = part[turn & 1][0][wave][lane];
#pragma unroll
                    for (int w = 1; w < WAVES; ++w) {
                        const f32x4 u = part[turn & 1][w][wave][lane];
                        v = f32x4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
                    }
                    const int m = 16 * (wave % MT) + r, n = 16 * (b + 1 - slot + wave / MT) + 4 * q;
                    uint16_t *to = y + (int64_t)(p.lo + m) * N + n;
                    const uint32_t a0 = pack2<ACT>(v[0], v[1]), a1 = pack2<ACT>(v[2], v[3]);
                    if (m < M) {
                        if (vec_y && n < N) {
                            *(u32x2 *)to = u32x2{a0, a1};
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (n + e < N)
                                    to[e] = (uint16_t)((e < 2 ? a0 : a1) >> (16 * (e & 1)));
                        }
                    }
                }
                slot = 0;
                ++turn;
            }
        }
    }
}

template <int FMT, int G, int WAVES, int S, int MT>
hipError_t launch_est_s(q4_dtype act_t, const ExpertsArgs &a, hipStream_t s)
{
    // one workgroup a compute unit, and no more than there are blocks
    const int64_t blocks = most_pieces(a.rows, a.experts, 16 * MT) * ((a.N + 15) / 16);
    const int64_t cus = device_cu_count();
    const dim3 grid((unsigned)(blocks < cus ? blocks : cus)), block(64 * WAVES);
    const int vec_y = (a.N % 4 == 0 && ((uintptr_t)a.y & 7) == 0) ? 1 : 0;
    if (act_t == Q4_BF16)
        hipLaunchKernelGGL((experts_stream_kernel<FMT, Q4_BF16, G, WAVES, S, MT>), grid, block, 0, s,
                           (const uint16_t *)a.x, (int)a.xrows, a.index, a.offsets, (int)a.rows, a.experts, a.codes,
                           a.scales, a.zeros, (int)a.N, (int)a.K, vec_y, (uint16_t *)a.y);
    else
        hipLaunchKernelGGL((experts_stream_kernel<FMT, Q4_F16, G, WAVES, S, MT>), grid, block, 0, s,
                           (const uint16_t *)a.x, (int)a.xrows, a.index, a.offsets, (int)a.rows, a.experts, a.codes,
                           a.scales, a.zeros, (int)a.N, (int)a.K, vec_y, (uint16_t *)a.y);
    return hipGetLastError();
}

// Waves and steps so that the lanes' parts of K reach 2048 or 4096: 16 waves
// where their registers hold x's part (one block of 16 rows: 62 -> 58 us for
// 16 rows through 7 experts of 14336 x 4096), 8 for two blocks (with 16 the
// registers spill: 89 -> 100 us).
template <int FMT, int G>
hipError_t launch_est_g(q4_dtype act_t, const ExpertsArgs &a, int mt, hipStream_t s)
{
    if (mt == 1)
        return a.K <= 2048 ? launch_est_s<FMT, G, 16, 1, 1>(act_t, a, s) : launch_est_s<FMT, G, 16, 2, 1>(act_t, a, s);
    return a.K <= 2048 ? launch_est_s<FMT, G, 8, 2, 2>(act_t, a, s) : launch_est_s<FMT, G, 8, 4, 2>(act_t, a, s);
}

template <int FMT>
hipError_t launch_est(int g, q4_dtype act_t, const ExpertsArgs &a, int mt, hipStream_t s)
{
    switch (g) {
    case 32:
        return launch_est_g<FMT, 32>(act_t, a, mt, s);
    case 64:
        return launch_est_g<FMT, 64>(act_t, a, mt, s);
    default:
        return launch_est_g<FMT, 128>(act_t, a, mt, s);
    }
}

}  // namespace

hipError_t launch_experts_stream(q4_format f, int g, q4_dtype act_t, const ExpertsArgs &a, int mt, hipStream_t s)
{
    switch (f) {
    case Q4_NF4:
        return launch_est<Q4_NF4>(g, act_t, a, mt, s);
    case Q4_FP4:
        return launch_est<Q4_FP4>(g, act_t, a, mt, s);
    case Q4_NF4_DQ:
        return launch_est<Q4_NF4_DQ>(g, act_t, a, mt, s);
    case Q4_INT4_SYM:
        return launch_est<Q4_INT4_SYM>(g, act_t, a, mt, s);
    default:
        return launch_est<Q4_INT4_ASYM>(g, act_t, a, mt, s);
    }
}

}  // namespace q4
