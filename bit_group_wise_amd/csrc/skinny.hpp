// skinny.hpp -- skinny product y[M, N] = x[M, K] . What^T for small M on the
// matrix cores: one workgroup's blocks of weight rows.
//
// Method ("Loading a model in 4-bit", "Where the accuracy goes"; "INT4
// Quantization > Practical Implementation with bitsandbytes"): the weights
// are dequantized to the 16-bit compute dtype (each value as q4_dequantize
// writes it) and multiplied with fp32 accumulation.  With a few activation
// rows the product still streams every weight byte once ("What is 4-bit
// quantization and why does it matter?", "Why it matters for deployment"),
// but the per-weight work grows with M, so from 3 rows on it runs here on
// v_mfma_f32_16x16x32 instead of the vector ALUs.
//
// gfx950 mapping:
//  * A workgroup owns RB blocks of 16 weight rows (one MFMA operand each)
//    and MT blocks of 16 activation rows (MT = 1, 2 or 4: up to 64 rows per
//    launch; each dequantized weight fragment feeds MT products); more rows
//    run as consecutive launches over row slices.  Its 8 waves split K into steps of
//    128, interleaved (wave w takes steps w, w + 8, ...).  A step's x
//    fragment serves all RB blocks, so each workgroup reads x once for RB
//    blocks; RB (1, 2 or 4) is the largest that still gives every compute
//    unit a workgroup.  (Without x loads at all, a timing-only variant ran
//    twice as fast at M = 16; halving them gained only 6 %: what the x loads
//    cost is mostly their latency in a pipeline of few steps per wave.)
//  * Lane (r, q) = (lane % 16, lane / 16) loads 16 bytes of codes: 32
//    weights of row r at k = k0 + 32 q.  Dword d of them is the lane's share
//    of MFMA d of the step, which therefore contracts over k0 + 32 q + 8 d
//    ... + 7 for lane quad q; the activation operand uses the same order, so
//    lane (m, q) loads x[m][k0 + 32 q ... + 31] as four 16-byte pieces.
//    Every load is contiguous; x rows past M and k past K are sent out of
//    range and read zeros.
//  * A 2-deep ring of steps keeps the next step's loads in flight.
//  * The 8 partial 16 x 16 tiles of each (row block, activation block) meet
//    in LDS and are summed in wave order (a fixed order, so the result does
//    not depend on timing).
//  * Double-quantized NF4 absmax: the lane loads its group's 8-bit code and
//    its run's binary32 constant and recovers the absmax with one product.
#pragma once

#include "q4_common.hpp"
#include "q4_internal.hpp"
#include "q4_mfma.hpp"
#include "lora.hpp"

namespace q4 {
namespace {

constexpr int kSkWaves = 8;
constexpr int kSkBlock = 64 * kSkWaves;
constexpr int kSkStep = 128;  // k per step
#ifndef Q4_SK_RING
#define Q4_SK_RING 2
#endif
constexpr int kSkRing = Q4_SK_RING;
enum { kSkDense = 0, kSkGather = 1, kSkLora = 2 };

// One step's operands for a lane: for each of the RB row blocks, 32 codes
// and their group's scale (and asym zero-point, or NF4_DQ run constant);
// and 32 activations of one x row, shared by the blocks.
template <int FMT, int RB, int MT>
struct SkStep {
    u32x4 cw[RB];
    uint32_t sraw[RB];
    uint32_t zraw[RB];
    int zsh[RB];
    u32x4 xv[MT][4];
};

// What a workgroup works on: x rows 0 .. M - 1 (at most 16 MT) against W rows
// n0 .. N - 1 (at most 16 RB) of the weight that starts at row wrow0 of an
// array of wrows rows.  Gathered: row m is x's row index[m] (without an index
// m itself), of xrows; one outside them is zeros.
struct SkTask {
    int M, n0, N;
    int64_t wrow0, wrows;
    const int32_t *index;
    int xrows;
};

// EXTRA: waves beside the 8 that multiply, for the adapters' part (kSkLora),
// whose chain of latencies (ids, then h and B) then passes beside the stream of
// the weights; 0: the 8 waves do it themselves before that.
template <int FMT, int ACT, int RB, int MT, int KIND, int EXTRA = 0>
__device__ __forceinline__ void skinny_product(const SkTask &task, const uint16_t *__restrict__ x,
                                               const uint8_t *__restrict__ codes,
                                               const void *__restrict__ scales,
                                               const uint8_t *__restrict__ zeros, int K, int gshift,
                                               uint16_t *__restrict__ y, const LowRank *low = nullptr)
{
    constexpr int LF = level_fmt(FMT);
    __shared__ float2 ptbl[LF == Q4_NF4 ? 256 : 1];
    constexpr int kAll = kSkWaves + EXTRA;
    __shared__ f32x4 part[kAll][RB][MT][64];

    const int lane = threadIdx.x & 63;
    const int wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int M = task.M, n0 = task.n0, N = task.N;
    const int64_t r0 = task.wrow0 + n0;  // the first row of the weight array
    const int G = K >> gshift;
    const int row_bytes = K >> 1;
    constexpr int ss = f32_absmax(FMT) ? 4 : (FMT == Q4_NF4_DQ ? 1 : 2);

    if constexpr (LF == Q4_NF4) {
        if (threadIdx.x < 256)
            ptbl[threadIdx.x] = float2{level_entry<FMT>(threadIdx.x & 15), level_entry<FMT>(threadIdx.x >> 4)};
    }

    // views: this workgroup's 16 RB weight rows (rows past N read zeros) and
    // the M activation rows
    const int nrows = N - n0 < 16 * RB ? N - n0 : 16 * RB;
    const __amdgpu_buffer_rsrc_t cr = buffer_view(codes + r0 * row_bytes, (int64_t)nrows * row_bytes);
    const __amdgpu_buffer_rsrc_t sr =
        buffer_view((const char *)scales + r0 * G * ss, (int64_t)nrows * G * ss);
    const int64_t zg0 = r0 * G;  // flat group index of the first row's first group
    __amdgpu_buffer_rsrc_t zr = sr;
    if constexpr (FMT == Q4_INT4_ASYM)
        zr = buffer_view(zeros + (zg0 >> 1), (((int64_t)nrows * G + (zg0 & 1)) + 1) / 2);
    // double-quantized absmax: the runs' binary32 constants for the rows'
    // groups (zr then starts at the run holding the first group)
    if constexpr (FMT == Q4_NF4_DQ) {
        const float *s2 = (const float *)((const char *)scales + dq_s2_offset(task.wrows * G));
        const int64_t r0 = zg0 / kDqRun, r1 = (zg0 + (int64_t)nrows * G - 1) / kDqRun;
        zr = buffer_view(s2 + r0, 4 * (r1 - r0 + 1));
    }
    const bool gather = KIND == kSkGather && task.index;
    const __amdgpu_buffer_rsrc_t xr = buffer_view(x, (int64_t)(gather ? task.xrows : M) * K * 2);
    int xm[MT];  // gathered: the x row of the lane's row of each activation block (-1: none)
    if constexpr (KIND == kSkGather) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = 16 * mt + r;
            xm[mt] = m < M ? m : -1;
            if (gather && m < M) {
                xm[mt] = task.index[m];
                if ((uint32_t)xm[mt] >= (uint32_t)task.xrows)
                    xm[mt] = -1;
            }
        }
    }

    const int nsteps = (K + kSkStep - 1) / kSkStep;
    auto load = [&](SkStep<FMT, RB, MT> &st, int step) {
        const int k = step * kSkStep + 32 * q;  // the lane's first k
        const bool in = step < nsteps && k < K;
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const int rr = 16 * b + r;  // the lane's weight row in the workgroup
            st.cw[b] = __builtin_amdgcn_raw_buffer_load_b128(cr, in ? rr * row_bytes + (k >> 1) : -16,
                                                             0, 0);
            const int gi = rr * G + (k >> gshift);  // group within the workgroup's rows
            if constexpr (f32_absmax(FMT))
                st.sraw[b] = __builtin_amdgcn_raw_buffer_load_b32(sr, in ? 4 * gi : -16, 0, 0);
            else if constexpr (FMT == Q4_NF4_DQ)
                st.sraw[b] = __builtin_amdgcn_raw_buffer_load_b8(sr, in ? gi : -16, 0, 0);
            else
                st.sraw[b] = __builtin_amdgcn_raw_buffer_load_b16(sr, in ? 2 * gi : -16, 0, 0);
            if constexpr (FMT == Q4_INT4_ASYM) {
                // the byte as loaded (no arithmetic on a load in flight) and
                // the nibble's position
                const int gz = (int)(zg0 & 1) + gi;
                st.zraw[b] = __builtin_amdgcn_raw_buffer_load_b8(zr, in ? gz >> 1 : -16, 0, 0);
                st.zsh[b] = 4 * (gz & 1);
            } else if constexpr (FMT == Q4_NF4_DQ) {
                const int gr = (int)(zg0 % kDqRun) + gi;  // group index from the first run's start
                st.zraw[b] =
                    __builtin_amdgcn_raw_buffer_load_b32(zr, in ? 4 * (gr / kDqRun) : -16, 0, 0);
            } else {
                st.zraw[b] = 0;
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = KIND == kSkGather ? xm[mt] : 16 * mt + r;  // the lane's activation row
            const bool xin = in && (KIND == kSkGather ? m >= 0 : m < M);
#pragma unroll
            for (int d = 0; d < 4; ++d)
                st.xv[mt][d] = __builtin_amdgcn_raw_buffer_load_b128(
                    xr, xin ? 2 * (m * K + k + 8 * d) : -16, 0, 0);
        }
    };

    // the adapters' part, h B^T, left in the wave's tiles
    const auto adapters = [&]() {
        if constexpr (KIND == kSkLora) {
            f32x4 acc[RB][MT];
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    acc[b][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            AdapterSet<1> all;
            all.init(low->ids, low->adapters, 0, M);
            const __amdgpu_buffer_rsrc_t parts = buffer_view(low->part, 4 * low->parts * low->rows * low->rank);
            constexpr int kTurns = EXTRA ? EXTRA : kSkWaves;  // waves that share the adapters
            constexpr int kAhead = 3;                         // adapters whose B is in flight
            constexpr uint32_t kPast = 0x80000000u;           // past every view
            const int first = wave - (EXTRA ? kSkWaves : 0);
            for (int rs = 0; rs < low->rank; rs += 32) {
                const int r0 = rs + 8 * q;
                // this wave's adapters: every kTurns-th, another wave's turn with
                // the next 32 values
                AdapterSet<1> set = all;
                int turn = kTurns - first + (rs >> 5);
                struct Slot {
                    bool on;
                    uint64_t mask;
                    u32x4 b[RB];
                };
                const auto next = [&](Slot &sl) {
                    int ad;
                    uint64_t mask[1] = {};
                    do
                        sl.on = set.next(ad, mask);
                    while (sl.on && turn++ % kTurns != 0);
                    sl.mask = mask[0];
                    const __amdgpu_buffer_rsrc_t br =
                        buffer_view(low->w + (int64_t)(sl.on ? ad : 0) * N * low->rank, (int64_t)N * low->rank * 2);
                    const uint32_t none = sl.on && r0 < low->rank ? 0u : kPast;  // (rows past N lie past the view)
#pragma unroll
                    for (int b = 0; b < RB; ++b)
                        sl.b[b] = __builtin_amdgcn_raw_buffer_load_b128(
                            br, (int)((2u * (uint32_t)((n0 + 16 * b + r) * low->rank + r0)) | none), 0, 0);
                };
                Slot slots[kAhead];
                next(slots[0]);
                if (!slots[0].on)
                    continue;
#pragma unroll
                for (int i = 1; i < kAhead; ++i)
                    next(slots[i]);
                Low8 h[MT];  // of all rows, whatever their adapters
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float v[8];
                    sum_parts(parts, *low, 16 * mt + r, r0, 16 * mt + r < M && r0 < low->rank, v);
                    h[mt] = three_parts(v);
                }
                while (slots[0].on) {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        if (slots[i].on) {
#pragma unroll
                            for (int b = 0; b < RB; ++b) {
                                const Exact8 w = exact_parts<ACT>(slots[i].b[b]);
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt) {
                                    const uint32_t its = rows16(slots[i].mask, 16 * mt);
                                    if (its == 0)
                                        continue;
                                    const f32x4 t = mfma_exact_low<ACT>(w, h[mt], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                                    const bool mine = (its >> r) & 1;
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        acc[b][mt][e] = mine ? acc[b][mt][e] + t[e] : acc[b][mt][e];
                                }
                            }
                        }
                        next(slots[i]);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    part[wave][b][mt][lane] = acc[b][mt];
        }
    };

    if (EXTRA > 0 && wave >= kSkWaves) {
        __syncthreads();  // (with the others, at their level-pair table)
        adapters();
    } else {
        if constexpr (EXTRA == 0)
            adapters();
        // the wave's steps: wave, wave + 8, ...
        SkStep<FMT, RB, MT> ring[kSkRing];
#pragma unroll
        for (int i = 0; i < kSkRing; ++i)
            load(ring[i], wave + kSkWaves * i);
        __syncthreads();  // the level-pair table

        f32x4 acc[RB][MT];
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                acc[b][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int step = wave; step < nsteps; step += kSkWaves * kSkRing) {
#pragma unroll
            for (int i = 0; i < kSkRing; ++i) {
                SkStep<FMT, RB, MT> &st = ring[i];
                // a step past the end is not computed (its slot is still
                // refilled below, so the load waits stay partial)
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    if (step + kSkWaves * i >= nsteps)
                        break;
                    float s, bias;
                    if constexpr (f32_absmax(FMT)) {
                        s = std::bit_cast<float>(st.sraw[b]);
                        bias = 0.0f;
                    } else if constexpr (FMT == Q4_NF4_DQ) {  // c' = qc * s2, one product
                        s = keep_f32((float)st.sraw[b] * std::bit_cast<float>(st.zraw[b]));
                        bias = 0.0f;
                    } else {
                        s = h2f(st.sraw[b] & 0xffffu);
                        bias = FMT == Q4_INT4_SYM ? -8.0f * s
                                                  : -(float)((st.zraw[b] >> st.zsh[b]) & 0xfu) * s;
                    }
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        float2 lp[4];
                        if constexpr (LF == Q4_NF4) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                lp[e] = ptbl[(st.cw[b][d] >> (8 * e)) & 0xffu];
                        }
                        const u32x4 wf = dequant8<FMT, ACT>(st.cw[b][d], s, bias, lp);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            acc[b][mt] = mfma<ACT>(wf, st.xv[mt][d], acc[b][mt]);
                    }
                }
                load(st, step + kSkWaves * (i + kSkRing));
            }
        }

        // sum the waves' partial tiles of each (row block, activation block) in
        // wave order; lane l holds rows 4 q + v of the row block against
        // activation row 16 mt + r
#pragma unroll
        for (int b = 0; b < RB; ++b) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if constexpr (KIND == kSkLora && EXTRA == 0) {  // (beside the adapters' part)
                    const f32x4 u = part[wave][b][mt][lane];
                    acc[b][mt] = f32x4{acc[b][mt][0] + u[0], acc[b][mt][1] + u[1], acc[b][mt][2] + u[2],
                                       acc[b][mt][3] + u[3]};
                }
                part[wave][b][mt][lane] = acc[b][mt];
            }
        }
    }
    __syncthreads();
    for (int t = wave; t < RB * MT; t += kAll) {
        const int b = t / MT, mt = t % MT;
        f32x4 u0 = part[0][b][mt][lane];
#pragma unroll
        for (int w = 1; w < kAll; ++w) {
            const f32x4 u = part[w][b][mt][lane];
            u0 = f32x4{u0[0] + u[0], u0[1] + u[1], u0[2] + u[2], u0[3] + u[3]};
        }
        const int m = 16 * mt + r;
        const int n = n0 + 16 * b + 4 * q;
        if (m < M) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                if (n + v < N)
                    y[(int64_t)m * N + n + v] =
                        (uint16_t)(ACT == Q4_BF16 ? f2bf_bits(u0[v]) : f2h_bits(u0[v]));
            }
        }
    }
}

}  // namespace
}  // namespace q4
