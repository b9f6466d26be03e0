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
//    group's column, w_t s_tj, rounded to fp16 (11 bits against the output's 8
//    or 11: each weight is off by at most 2^-11 of itself, independently).  Of
//    a column's result only its group's values are used.  The zero-points'
//    share, sum_t w_t s_tj z_tj, is one more product of the same rounded
//    weights with the zero-points as rows, taken off at the end.
//  * Reference.  w_t s_tj must stay below 65504 and the largest should be well
//    inside fp16's normal range whatever the values' size, so m tracks
//    x_t + log2(s_t), not x_t: it moves only when a weight would pass 2^15 and
//    is then set to put the largest at 2^6.
//
// Bound: HBM traffic of the packed rows in the limit; in practice the rate at
// which lanes receive their words (texture path) and vector-ALU issue.
//
// Split: a workgroup's four waves take 32-token steps of one range of one
// sequence and head in turn and join their sums in LDS; where sequences and
// heads alone would leave compute units idle the length is split over
// workgroups and a second launch joins the parts.
#include "kv_attn.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 4;
constexpr int kBlock = 64 * kWaves;
constexpr int kStep = 32;  // tokens per wave and step

// Values of 16 tokens as they are in memory, a lane's share of rows 4 kg .. + 3:
// the values (D/16) i .. of row part h, the scales in the column's group, the
// zero-points of the values' groups.
template <int FMT, int D, int GS>
struct ValueTile {
    static constexpr int NG = D / GS, ZB = (NG + 1) / 2, W = D < 128 ? D : 128, HV = D / W;
    uint32_t w[4][HV], s[4], z[FMT == Q4_INT4_ASYM ? ZB : 1];

    __device__ __forceinline__ void load(const KvCache &c, int64_t row0, int lane)
    {
        const int i = lane & 15, kg = lane >> 4;
        const int64_t row = row0 >= 0 ? row0 : 0;  // (page 0 is read and not used)
        const uint8_t *p = c.v.codes + row * (D / 2) + (uint32_t)(4 * kg * (D / 2) + 4 * value_dword<W>(i));
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int h = 0; h < HV; ++h)
                w[r][h] = *(const uint32_t *)(p + r * (D / 2) + h * (W / 2));
        load_scales<FMT, NG>(s, c.v.scales, row, kg, i % NG);
        if constexpr (FMT == Q4_INT4_ASYM) {
            const uint32_t *zp = (const uint32_t *)(c.v.zeros + row * ZB + (uint32_t)(4 * kg * ZB));
#pragma unroll
            for (int k = 0; k < ZB; ++k)
                z[k] = zp[k];
        }
    }
    // The scales of the lane's rows from the n-th on become 0.
    __device__ __forceinline__ void keep(int n)
    {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            s[r] = r < n ? s[r] : 0u;
    }
    __device__ __forceinline__ float largest() const  // (no scale is negative)
    {
        return fmaxf(fmaxf(scale_of<FMT>(s[0]), scale_of<FMT>(s[1])), fmaxf(scale_of<FMT>(s[2]), scale_of<FMT>(s[3])));
    }
    // Zero-points of rows r and r + 1 in the group of the lane's values of
    // part h, as the two halves of a word.
    __device__ __forceinline__ uint32_t zero_pair(int r, int h, int i) const
    {
        const int sh = 4 * ((W * h + W / 16 * i) / GS);
        const uint32_t a = z[r * ZB / 4] >> (8 * (r * ZB % 4)) >> sh;
        const uint32_t b = z[(r + 1) * ZB / 4] >> (8 * ((r + 1) * ZB % 4)) >> sh;
        return (a & 15u) | (b & 15u) << 16;
    }
};

template <int FMT, int D, int GS, int NT>
__global__ __launch_bounds__(kBlock, (D == 256 ? 1 : NT == 1 ? 3 : 2)) void kv_token_kernel(
    KvCache c, KvBatch b, Rows rows, Split sp, float *__restrict__ part, float2 *__restrict__ part_ml)
{
    constexpr int NG = D / GS, W = D < 128 ? D : 128, HV = D / W, NP = W / 16;
    constexpr int NR = NT * 16 / NG;                         // rows
    constexpr int HZ = FMT == Q4_INT4_ASYM ? HV : 1;         // zero-point products
    __shared__ float os[kWaves][NR][D + 4];
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
    const int begin = range_begin(s, rows.window) + pt * sp.span;
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
    f32x4 o[NT][HV][NP], oz[NT][HZ];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = kNone;
        l[n] = 0.0f;
#pragma unroll
        for (int v = 0; v < HZ; ++v)
            oz[n][v] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < HV; ++v)
#pragma unroll
            for (int p = 0; p < NP; ++p)
                o[n][v][p] = f32x4{0, 0, 0, 0};
    }

    Pages pg{b.table + (int64_t)seq * b.table_width, c.page_shift, c.heads, h, c.pages, 1 << 30,
             (s.len - 1) >> c.page_shift, -1};
    // The registers of a step's keys take the next step's as soon as the scores
    // are formed, those of its values once they are summed: loads are always
    // in flight, without a second set.
    KeyTile<FMT, D, GS> kt[2];
    ValueTile<FMT, D, GS> vt[2];
    int t0 = begin + wave * kStep;
    int64_t row0 = pg.row(t0, end, lane), row1 = pg.row(t0 + 16, end, lane);
    if (t0 < end) {
        kt[0].load(c, row0, lane);
        kt[1].load(c, row1, lane);
        vt[0].load(c, row0, lane);
        vt[1].load(c, row1, lane);
    }
    while (t0 < end) {
        const int tn = t0 + kWaves * kStep;
        f32x4 x[2][NT];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            col_scores<FMT, D, GS, NT>(kt[u], q, kg, pairs, x[u]);
        const int64_t next0 = pg.row(tn, end, lane), next1 = pg.row(tn + 16, end, lane);
        if (tn < end) {
            kt[0].load(c, next0, lane);
            kt[1].load(c, next1, lane);
        }
        if (__builtin_expect(row0 < 0 || row1 < 0 || t0 + kStep - 1 > all_to || t0 < all_from, 0)) {
            const int ta = branch_only(t0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int have = (u ? row1 : row0) < 0 ? 0 : end - ta - 16 * u - 4 * kg;
                vt[u].keep(have);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = ta + 16 * u + 4 * kg + r;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        x[u][n][r] = r < have && at <= q.pos[n] && at > q.low[n] ? x[u][n][r] : -__builtin_inff();
                }
            }
        }
        // (2^-40: rows of zeros do not pull the reference down)
        const float big = __builtin_amdgcn_logf(
            fmaxf(group_max<NG>(fmaxf(vt[0].largest(), vt[1].largest())), 0x1p-40f));
        float reach[NT];
        bool move = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float top = fmaxf(x[0][n][0], x[1][n][0]);
#pragma unroll
            for (int r = 1; r < 4; ++r)
                top = fmaxf(top, fmaxf(x[0][n][r], x[1][n][r]));
            reach[n] = __builtin_fmaf(top, q.factor[n], big);
            move = move || reach[n] > m[n] + 15.0f;
        }
        if (__builtin_expect(__any(move), 0)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float to = fmaxf(m[n], quad_max(reach[n]) - 6.0f);
                const float f = __builtin_amdgcn_exp2f(m[n] - to);
                m[n] = to;
                l[n] *= f;
#pragma unroll
                for (int v = 0; v < HZ; ++v)
                    oz[n][v] *= f;
#pragma unroll
                for (int v = 0; v < HV; ++v)
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        o[n][v][p] *= f;
            }
        }
        u32x4 wp[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int u = e >> 1, r = 2 * (e & 1);
                const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][n][r], q.factor[n], -m[n]));
                const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][n][r + 1], q.factor[n], -m[n]));
                l[n] += w0 + w1;
                // (fma with 0: the scale's conversion is part of v_fma_mix)
                wp[n][e] = pair_h2(__builtin_fmaf(w0, scale_of<FMT>(vt[u].s[r]), 0.0f),
                                   __builtin_fmaf(w1, scale_of<FMT>(vt[u].s[r + 1]), 0.0f));
            }
#pragma unroll
        for (int v = 0; v < HV; ++v) {
            u32x4 va[NP];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int u = e >> 1, r = 2 * (e & 1);
                uint32_t p[NP];
                value_pairs<FMT, W>(vt[u].w[r][v], vt[u].w[r + 1][v], sel, pairs, p);
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    va[k][e] = p[k];
            }
#pragma unroll
            for (int k = 0; k < NP; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    o[n][v][k] = mfma<Q4_F16>(va[k], wp[n], o[n][v][k]);
        }
        if constexpr (kv_int<FMT>()) {
#pragma unroll
            for (int v = 0; v < HZ; ++v) {
                u32x4 z = {0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u};
                if constexpr (FMT == Q4_INT4_ASYM) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[e] = vt[e >> 1].zero_pair(2 * (e & 1), v, i);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    oz[n][v] = mfma<Q4_F16>(z, wp[n], oz[n][v]);
            }
        }
        if (tn < end) {
            vt[0].load(c, next0, lane);
            vt[1].load(c, next1, lane);
        }
        t0 = tn;
        row0 = next0;
        row1 = next1;
    }

    // join the waves
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
                        if constexpr (kv_int<FMT>())
                            y[e] -= oz[n][HZ == 1 ? 0 : v][r] * value_unit<FMT>();
                    }
                    *(f32x4 *)&os[wave][r0][W * v + W / 16 * (4 * kg + r) + k] = y;
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
            sum += *(const f32x4 *)&os[w][row][d] * f;
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
                const float v = ll > 0.0f ? mm + __builtin_amdgcn_logf(ll) : -__builtin_inff();
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

// Most parts that a length is split into: as many as give the 256 compute
// units about four workgroups each, none shorter than 256 tokens; up to 512
// tokens one (a single launch of at most four steps a wave).
int most_parts(const KvCache &c, const KvBatch &b)
{
    if (b.max_len <= 512)
        return 1;
    const int64_t wgs = (int64_t)b.seqs * c.heads;
    return (int)std::min<int64_t>((1024 + wgs - 1) / wgs, (b.max_len + 255) / 256);
}

}  // namespace

Split token_split(const KvCache &c, const KvBatch &b, int group, int window)
{
    Split sp;
    sp.tiles = 1;
    const int64_t range = longest_range(b, window);
    const int64_t parts = range <= 512 ? 1 : most_parts(c, b);
    // whole rounds of the four waves' steps
    const int64_t span = std::max<int64_t>((range + parts - 1) / parts, parts > 1 ? 256 : 1);
    sp.span = (int)((span + kWaves * kStep - 1) / (kWaves * kStep) * (kWaves * kStep));
    sp.parts = (int)std::max<int64_t>((range + sp.span - 1) / sp.span, 1);
    return sp;
}

hipError_t launch_kv_token(int f, const KvCache &c, const KvBatch &b, const Rows &rows, const Split &sp,
                           float *part, float2 *part_ml, hipStream_t s)
{
    return kv_by_shape(f, c.dim, c.g, [&](auto fmt, auto dim, auto gs) {
        constexpr int F = decltype(fmt)::value, D = decltype(dim)::value, GS = decltype(gs)::value;
        const dim3 grid(sp.parts, c.heads, b.seqs);
        const int64_t cols = (int64_t)b.max_new * rows.group * (D / GS);
        if (cols <= 16)
            kv_token_kernel<F, D, GS, 1><<<grid, kBlock, 0, s>>>(c, b, rows, sp, part, part_ml);
        else if (cols <= 32)
            kv_token_kernel<F, D, GS, 2><<<grid, kBlock, 0, s>>>(c, b, rows, sp, part, part_ml);
        else if constexpr (D == 64)
            kv_token_kernel<F, D, GS, 4><<<grid, kBlock, 0, s>>>(c, b, rows, sp, part, part_ml);
        return hipGetLastError();
    });
}

}  // namespace q4
