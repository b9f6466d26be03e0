// kv_token.hip -- attention over the 4-bit cache for a few rows a head: single
// tokens and short drafts (q4_kv_attention).
//
// Mathematics: one pass over the cached tokens with the running reference m of
// the softmax.  With scores x_t (in powers of two: scale log2(e) is folded
// into the row's factor), weights w_t = 2^(x_t - m), row sum l = sum w_t and
// output sum w_t V_t / l; raising m scales both sums by 2^(m_old - m_new).
//
//  * Scores.  S = K Q^T on 16x16x32 products, 16 cached tokens by 16 columns.
//    K enters as levels (see kv_mfma.hpp) less zero-points, exactly; q is fp16
//    exactly (a row is scaled by a power of two that puts its largest value
//    just below 2^12; values 2^-22 below the largest would round).  Scales are
//    applied in binary32: a column is a row and a scale group (see kv_attn.hpp).
//  * Output.  O^T = V^T W^T, 16 values by 16 columns over 32 tokens.  S leaves
//    each lane with eight tokens of one row; contracting the tokens in that
//    order makes them the second product's column operand without moving.  A
//    V scale belongs to a token and a group, so it goes into the weight of the
//    group's column, w_t s_tj, rounded to fp16: 11 bits.  That is 2^-11 of each
//    weight, independently: a bf16 output, of 8 bits, is as far from binary64
//    as without it (1.7e-3).  An fp16 output would be 2.8e-4 to 3.5e-4 off
//    instead of the 2.1e-4 of its own rounding, so for those a second product
//    adds what the rounding left of the weights (TWO; kv_token_f16.hip): 66.9
//    instead of 60.8 us at 131071 tokens, 29.3 for 26.2 in 8 drafts of 4.  Of a
//    column's result only its group's values are used.
//  * Reference.  w_t s_tj must stay below 65504 and the largest should be well
//    inside fp16's normal range whatever the values' size, so m tracks
//    x_t + log2(s_t), not x_t: it moves only when a weight would pass 2^15.5
//    and is then set to put the largest at 2^13.5, so that a weight has fp16's
//    full 11 bits down to 2^-27 of the largest (in long caches most of the sum
//    is in weights far below it; with the largest at 2^6 the 131071-token case
//    was 2.5 times as far from binary64).  That it may have to move is seen from
//    a bound (the largest score and the largest scale of eight tokens); where
//    their scales differ by more than 2^4, it moves to the largest sum of a
//    token's own two, so large values of tokens that the row does not see, or
//    hardly weighs, take no more bits than that of the others'.
//
// Bound: HBM traffic of the packed rows in the limit; in practice the rate at
// which lanes receive their words (the texture path takes some 16 cycles an
// instruction, whatever its width, hence 16-byte loads of whole rows handed on
// through LDS) and vector-ALU issue, each busy for half to two thirds of the
// time.  Nothing is read twice.  One new token a sequence, dim 128:
//   2 x 131071 tokens, 8 heads, 4 rows, INT4-asym g32   61 us + 5 to join, 4.2 TB/s
//     (fp16, weights in two parts: 67 + 5)
//   32 x 4096, 8 heads, 4 rows, INT4-sym g64, scores kept   35 us + 4 to 6
//   16 x 2048, 32 heads, 1 row, NF4 g64                 35 us, 3.4 TB/s (level
//     lookups: LDS busy half the time, with conflicts; levels by v_perm 39 us)
//   333 tokens, 8 heads                                  8 us, of which a launch 2.5
//
// Split: a workgroup's four waves take 32-token steps of one range of one
// sequence and head in turn and join their sums in LDS; where sequences and
// heads alone would leave compute units idle the length is split over
// workgroups and a second launch joins the parts.
#include "kv_attn.hpp"

#ifndef Q4_KV_TOKEN_TWO
#define Q4_KV_TOKEN_TWO 0  // weights in two parts: kv_token_f16.hip
#endif

namespace q4 {
namespace {

constexpr int kWaves = 4;
constexpr int kBlock = 64 * kWaves;
constexpr int kStep = 32;  // tokens per wave and step
constexpr bool kTwo = Q4_KV_TOKEN_TWO;

// The values of a step's 32 tokens: as they are in memory, 16 bytes a lane in a
// row, and from LDS a lane's share of rows 4 kg .. + 3, the values (D/16) i ..
// of row part h.
template <int D>
struct ValueCodes {
    static constexpr int W = D < 128 ? D : 128, HV = D / W, RD = D / 8, NL = D / 64;  // 16-byte loads
    static constexpr int STRIDE = 4 * RD + (D == 64 ? 8 : 16);  // words of four rows: no two lanes on a bank
    struct Lds {
        __attribute__((aligned(16))) uint32_t v[2][4 * STRIDE];
    };
    u32x4 w[NL];

    // Place k of the lane: subtile u, row, 16-byte chunk.
    static __device__ __forceinline__ void place(int k, int lane, int &u, int &row, int &chunk)
    {
        const int e = 64 * k + lane, at = e % (16 * (D / 32));
        u = e / (16 * (D / 32));
        row = at / (D / 32);
        chunk = at % (D / 32);
    }
    __device__ __forceinline__ void load(const KvCache &c, int64_t row0, int64_t row1, int lane)
    {
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            int u, row, chunk;
            place(k, lane, u, row, chunk);
            const int64_t r = max(u ? row1 : row0, (int64_t)0);  // (page 0 is read and not used)
            w[k] = *(const u32x4 *)(c.v.codes + r * (D / 2) + (uint32_t)(row * (D / 2) + 16 * chunk));
        }
    }
    __device__ __forceinline__ void put(Lds &to, int lane) const
    {
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            int u, row, chunk;
            place(k, lane, u, row, chunk);
            *(u32x4 *)&to.v[u][(row >> 2) * STRIDE + (row & 3) * RD + 4 * chunk] = w[k];
        }
    }
    static __device__ __forceinline__ uint32_t get(const Lds &from, int u, int r, int h, int i, int kg)
    {
        return from.v[u][kg * STRIDE + r * RD + h * (W / 8) + value_dword<W>(i)];
    }
};

// Zero-points of tokens t and t + 1 in the group of the lane's values of part
// h, as the two halves of a word; z: those of four tokens from 4 kg.
template <int D, int GS, int ZB>
__device__ __forceinline__ uint32_t zero_pair(const uint32_t *z, int r, int h, int i)
{
    constexpr int W = D < 128 ? D : 128;
    const int sh = 4 * ((W * h + W / 16 * i) / GS);
    const uint32_t a = z[r * ZB / 4] >> (8 * (r * ZB % 4)) >> sh;
    const uint32_t b = z[(r + 1) * ZB / 4] >> (8 * ((r + 1) * ZB % 4)) >> sh;
    return (a & 15u) | (b & 15u) << 16;
}

template <int FMT, int D, int GS, int NT, bool KEEP, bool TWO>
__global__ __launch_bounds__(kBlock, (D == 256 ? 1 : NT == 1 ? 3 : 2)) void kv_token_kernel(
    KvCache c, KvBatch b, Rows rows, Split sp, float *__restrict__ part, float2 *__restrict__ part_ml)
{
    constexpr int NG = D / GS, W = D < 128 ? D : 128, HV = D / W, NP = W / 16;
    constexpr int NR = NT * 16 / NG;                         // rows
    constexpr int ZB = (NG + 1) / 2;
    using Codes = ValueCodes<D>;
    using M = Meta<FMT, NG, 64>;  // lanes 0..31: keys, 32..63: values
    struct Work {
        typename Codes::Lds v;
        typename M::Lds m;
    };
    union Share {  // a wave's: the step's, and its sums in the end
        Work work;
        float os[NR][D + 4];
    };
    __shared__ Share share[kWaves];
    __shared__ float2 ml[kWaves][NR];
    __shared__ uint32_t pairs[FMT == Q4_NF4 ? 256 : 1];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, kg = lane >> 4;
    const int seq = blockIdx.z, h = blockIdx.y, pt = blockIdx.x;
    const KvSeq s = kv_seq(b, seq);
    const int nrows = s.fresh * rows.group;
    if (nrows == 0)
        return;
    const int begin0 = range_begin(s, rows.window), begin = begin0 + pt * sp.span;
    float *kept = KEEP ? rows.kept + ((int64_t)seq * c.heads + h) * rows.kept_range * rows.kept_rows : nullptr;
    const int end = min(s.len, begin + sp.span);
    if (begin >= s.len && pt > 0)
        return;

    if constexpr (FMT == Q4_NF4) {
        pairs[tid] = nf4_pair(tid);
        __syncthreads();
    }

    ColQueries<FMT, D, GS, NT> q;
    q.load(s, rows, h, 0, lane);
    // tokens that every row sees need no mask
    const int all_to = s.len - s.fresh, all_from = rows.window > 0 ? s.len - rows.window : 0;

    const uint32_t sel = value_select<FMT, W>(i);
    f32x4 o[NT][HV][NP];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = kNone;
        l[n] = 0.0f;
#pragma unroll
        for (int v = 0; v < HV; ++v)
#pragma unroll
            for (int p = 0; p < NP; ++p)
                o[n][v][p] = f32x4{0, 0, 0, 0};
    }

    Pages pg{b.table + (int64_t)seq * b.table_width, c.page_shift, c.heads, h, c.pages, 1 << 30,
             (s.len - 1) >> c.page_shift, -1};
    // The registers of a step's codes take the next step's as soon as they are
    // unpacked or in LDS: loads are in flight most of the time without a
    // second set.
    Work &wk = share[wave].work;
    KeyCodes<FMT, D, GS> kt[2];
    Codes vt;
    M meta;
    int t0 = begin + wave * kStep;
    int64_t row0 = pg.row(t0, end, lane), row1 = pg.row(t0 + 16, end, lane);
    auto load_step = [&](int64_t r0, int64_t r1) {
        kt[0].load(c, r0, lane);
        kt[1].load(c, r1, lane);
        const int64_t r = max(lane & 16 ? r1 : r0, (int64_t)0) + (lane & 15);
        meta.load(lane < 32 ? c.k : c.v, r);
        vt.load(c, r0, r1, lane);
    };
    if (t0 < end)
        load_step(row0, row1);
    while (t0 < end) {
        const int tn = t0 + kWaves * kStep;
        wave_order();
        meta.put(wk.m, lane);
        vt.put(wk.v, lane);
        wave_order();
        f32x4 x[2][NT];
        Scales4<FMT> vs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            Scales4<FMT> ks;
            ks.get(wk.m.s[i % NG], 16 * u + 4 * kg);
            vs[u].get(wk.m.s[i % NG], 32 + 16 * u + 4 * kg);
            const uint32_t z = FMT == Q4_INT4_ASYM ? key_zeros<D, GS>(wk.m.z, 16 * u + i, kg) : 0u;
            col_scores<FMT, D, GS, NT>(kt[u], z, ks, q, pairs, x[u]);
        }
        const int64_t next0 = pg.row(tn, end, lane), next1 = pg.row(tn + 16, end, lane);
        if (tn < end)
            load_step(next0, next1);
        if (__builtin_expect(row0 < 0 || row1 < 0 || t0 + kStep - 1 > all_to || t0 < all_from, 0)) {
            const int ta = branch_only(t0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int have = (u ? row1 : row0) < 0 ? 0 : end - ta - 16 * u - 4 * kg;
                vs[u].keep(have);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = ta + 16 * u + 4 * kg + r;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        x[u][n][r] = r < have && at <= q.pos[n] && at > q.low[n] ? x[u][n][r] : -__builtin_inff();
                }
            }
        }
        if constexpr (KEEP) {
            // the scores, in powers of two, for the mass pass; a row's first
            // column writes them
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int row = ColQueries<FMT, D, GS, NT>::row(n, lane);
                if (i % NG == 0 && row < nrows) {
                    float *to = kept + (int64_t)(t0 - begin0 + 4 * kg) * rows.kept_rows + row;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (t0 + 16 * u + 4 * kg + r < end)
                                to[(16 * u + r) * rows.kept_rows] = x[u][n][r] * q.factor[n];
                }
            }
        }
        // (2^-40: rows of zeros do not pull the reference down)
        const float big = __builtin_amdgcn_logf(
            fmaxf(group_max<NG>(fmaxf(vs[0].largest(), vs[1].largest())), 0x1p-40f));
        float reach[NT];
        bool move = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float top = fmaxf(x[0][n][0], x[1][n][0]);
#pragma unroll
            for (int r = 1; r < 4; ++r)
                top = fmaxf(top, fmaxf(x[0][n][r], x[1][n][r]));
            reach[n] = __builtin_fmaf(top, q.factor[n], big);
            move = move || reach[n] > m[n] + 15.5f;
        }
        if (__builtin_expect(__any(move), 0)) {
            // (the bound does where the eight tokens' scales are within 2^4)
            const Scales4<FMT> s0 = vs[0].branch_only(), s1 = vs[1].branch_only();
            const float least = group_max<NG>(fminf(s0.smallest(), s1.smallest()));
            if (__any(!(__builtin_amdgcn_logf(least) >= big - 4.0f))) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    reach[n] = -__builtin_inff();
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const Scales4<FMT> here = (u ? s1 : s0).branch_only();
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float size = __builtin_amdgcn_logf(fmaxf(group_max<NG>(here[r]), 0x1p-40f));
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            reach[n] = fmaxf(reach[n], __builtin_fmaf(x[u][n][r], q.factor[n], size));
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float to = fmaxf(m[n], quad_max(reach[n]) - 13.5f);
                const float f = __builtin_amdgcn_exp2f(m[n] - to);
                m[n] = to;
                l[n] *= f;
#pragma unroll
                for (int v = 0; v < HV; ++v)
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        o[n][v][p] *= f;
            }
        }
        u32x4 wp[NT], wr[TWO ? NT : 1];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int u = e >> 1, r = 2 * (e & 1);
                const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][n][r], q.factor[n], -m[n]));
                const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][n][r + 1], q.factor[n], -m[n]));
                l[n] += w0 + w1;
                // (fma with 0: the scale's conversion is part of v_fma_mix)
                const float s0 = __builtin_fmaf(w0, vs[u][r], 0.0f), s1 = __builtin_fmaf(w1, vs[u][r + 1], 0.0f);
                wp[n][e] = pair_h2(s0, s1);
                if constexpr (TWO)
                    wr[n][e] = pair_h2(s0 - h2f(wp[n][e] & 0xffffu), s1 - h2f(wp[n][e] >> 16));
            }
#pragma unroll
        for (int v = 0; v < HV; ++v) {
            u32x4 va[NP];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int u = e >> 1, r = 2 * (e & 1);
                uint32_t p[NP];
                KeyZero z = zero_of_pair(0x00080008u);
                if constexpr (FMT == Q4_INT4_ASYM) {
                    uint32_t zw[ZB];
                    load_words(zw, wk.m.z + ZB * (32 + 16 * u + 4 * kg));
                    z = zero_of_pair(zero_pair<D, GS, ZB>(zw, r, v, i));
                }
                value_pairs<FMT, W>(Codes::get(wk.v, u, r, v, i, kg), Codes::get(wk.v, u, r + 1, v, i, kg), sel, z,
                                    pairs, p);
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    va[k][e] = p[k];
            }
#pragma unroll
            for (int k = 0; k < NP; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (TWO)
                        o[n][v][k] = mfma<Q4_F16>(va[k], wr[n], o[n][v][k]);
                    o[n][v][k] = mfma<Q4_F16>(va[k], wp[n], o[n][v][k]);
                }
        }
        t0 = tn;
        row0 = next0;
        row1 = next1;
    }

    // join the waves
    wave_order();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r0 = ColQueries<FMT, D, GS, NT>::row(n, lane);
        l[n] = quad_sum(l[n]);
        if (kg == 0 && i % NG == 0)
            ml[wave][r0] = float2{m[n], l[n]};
#pragma unroll
        for (int v = 0; v < HV; ++v) {
            // values (W/16) (4 kg + r) + k of part v, of use in their group's column
            if ((W * v + W / 4 * kg) / GS != i % NG)
                continue;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int k = 0; k < NP; k += 4) {
                    f32x4 y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float unit = value_unit<FMT>() * (kv_int<FMT>() && (e & 1) ? 0.0625f : 1.0f);
                        y[e] = o[n][v][k + e][r] * unit;
                    }
                    *(f32x4 *)&share[wave].os[r0][W * v + W / 16 * (4 * kg + r) + k] = y;
                }
        }
    }
    __syncthreads();
    for (int e = tid; e < NR * D / 4; e += kBlock) {
        const int row = e / (D / 4), d = 4 * (e % (D / 4));
        if (row >= nrows)
            break;
        float mm = kNone;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            mm = fmaxf(mm, ml[w][row].x);
        f32x4 sum = {0, 0, 0, 0};
        float ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(ml[w][row].x - mm);
            ll += ml[w][row].y * f;
            sum += *(const f32x4 *)&share[w].os[row][d] * f;
        }
        const int tk = row / rows.group;
        const int64_t to = (int64_t)(s.first + tk) * rows.q_heads + h * rows.group + row - tk * rows.group;
        if (sp.parts == 1) {
            const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
            sum *= inv;
            u32x2 pk;
            pk[0] = rows.act == Q4_F16 ? pair_h2(sum[0], sum[1]) : pack_bf2(sum[0], sum[1]);
            pk[1] = rows.act == Q4_F16 ? pair_h2(sum[2], sum[3]) : pack_bf2(sum[2], sum[3]);
            *(u32x2 *)(rows.out + to * D + d) = pk;
            if (d == 0) {
                const float v = ll > 0.0f ? row_stat(mm, ll) : -__builtin_inff();
                if (rows.lse)
                    rows.lse[to] = v * kLn2;
                if (rows.stat)
                    rows.stat[to] = v;
            }
        } else {
            const int64_t at = to * sp.parts + pt;
            *(f32x4 *)(part + at * D + d) = sum;
            if (d == 0)
                part_ml[at] = float2{mm, ll};
        }
    }
}

#if !Q4_KV_TOKEN_TWO
// Most parts that a length is split into: as many as leave every workgroup
// resident at once (three to each of the 256 compute units, two where rows
// fill more than one column tile; dim 256 takes the registers of one), none
// shorter than 256 tokens; up to 512 tokens one (a
// single launch of at most four steps a wave).  A second round of workgroups
// costs more than it balances: 32 x 4096 tokens in 3, 4, 8 parts 27.3, 31.0,
// 34.8 us; 512 sequences and heads of 2048 tokens in 1, 2, 4 parts 36.8, 40.1
// (+ 4.6 to join), 44.3 (+ 4.4) us; 8 heads of 4096 tokens in parts of 256 and
// 128 tokens 12.3 and 13.5; 333 and 500 tokens in one part 7.6 and 8.7 a call, in
// two 12.0 and 11.9.  (The parts are cut by max_len: a batch of ragged lengths
// leaves those past a sequence's end empty.)
int most_parts(const KvCache &c, const KvBatch &b, int group)
{
    if (b.max_len <= 512)
        return 1;
    const int64_t wgs = (int64_t)b.seqs * c.heads, cols = (int64_t)b.max_new * group * (c.dim / c.g);
    const int64_t room = c.dim == 256 ? 256 : cols <= 16 ? 768 : 512;
    return (int)std::max<int64_t>(1, std::min<int64_t>(room / wgs, (b.max_len + 255) / 256));
}

#endif

}  // namespace

#if !Q4_KV_TOKEN_TWO
Split token_split(const KvCache &c, const KvBatch &b, int group, int window)
{
    Split sp;
    sp.tiles = 1;
    const int64_t range = longest_range(b, window);
    const int64_t parts = range <= 512 ? 1 : most_parts(c, b, group);
    // whole rounds of the four waves' steps
    const int64_t span = std::max<int64_t>((range + parts - 1) / parts, parts > 1 ? 256 : 1);
    sp.span = (int)((span + kWaves * kStep - 1) / (kWaves * kStep) * (kWaves * kStep));
    sp.parts = (int)std::max<int64_t>((range + sp.span - 1) / sp.span, 1);
    return sp;
}

#endif

hipError_t launch_kv_token(int f, const KvCache &c, const KvBatch &b, const Rows &rows, const Split &sp,
                           float *part, float2 *part_ml, hipStream_t s)
{
    return kv_by_shape(f, c.dim, c.g, [&](auto fmt, auto dim, auto gs) {
        constexpr int F = decltype(fmt)::value, D = decltype(dim)::value, GS = decltype(gs)::value;
        const dim3 grid(sp.parts, c.heads, b.seqs);
        const int64_t cols = (int64_t)b.max_new * rows.group * (D / GS);
        auto go = [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            if (rows.kept)
                kv_token_kernel<F, D, GS, NT, true, kTwo><<<grid, kBlock, 0, s>>>(c, b, rows, sp, part, part_ml);
            else
                kv_token_kernel<F, D, GS, NT, false, kTwo><<<grid, kBlock, 0, s>>>(c, b, rows, sp, part, part_ml);
        };
        if (cols <= 16)
            go(KvInt<1>{});
        else if (cols <= 32)
            go(KvInt<2>{});
        else if constexpr (D == 64)
            go(KvInt<4>{});
        return hipGetLastError();
    });
}

}  // namespace q4
