// kv_token.hip -- attention over the 4-bit cache for a few rows a head: single
// tokens and short drafts (q4_kv_attention).
//
// Mathematics: one pass over the cached tokens with the running reference m of
// the softmax.  With scores x_t (in powers of two: scale log2(e) is folded
// into the row's factor), weights w_t = 2^(x_t - m), row sum l = sum w_t and
// output sum w_t V_t / l; raising m scales both sums by 2^(m_old - m_new).
//
//  * Scores.  S = K Q^T on 16x16x32 products, 16 cached tokens by 16 rows (the
//    new tokens' query heads of one key head).  K enters as levels (see
//    kv_mfma.hpp) less zero-points, one accumulator per scale group, so x =
//    sum_j s_j acc_j holds exact products.  q is fp16 exactly: a row is scaled
//    by a power of two that puts its largest value just below 2^12 (values
//    2^-22 below the largest would round).
//  * Output.  O^T = V^T W^T, 16 values by 16 rows over 32 tokens.  S leaves
//    each lane with eight tokens of one row; contracting the tokens in that
//    order makes them the second product's column operand without moving.
//    A V scale belongs to a token, so it goes into the weight: w_t s_tj, one
//    set per group j, rounded to fp16 (11 bits against the output's 8 or 11:
//    each weight is off by at most 2^-12 of itself, independently).  The
//    zero-points' share, sum_t w_t s_tj z_tj, is one more product of the same
//    rounded weights with the zero-points as rows, taken off at the end.
//  * Reference.  w_t s_tj must stay below 65504 and the largest should be well
//    inside fp16's normal range whatever the values' size, so m tracks
//    x_t + log2(s_t), not x_t: it moves only when a weight would pass 2^15 and
//    is then set to put the largest at 2^6.
//
// Bound: HBM traffic of the packed rows in the limit, vector-ALU issue in
// practice (unpacking about 1.5 instructions a code word's nibble pair, and
// the softmax of a 16-column tile of which a head group may fill only some).
//
// Split: a workgroup's four waves take 32-token steps of one range of one
// sequence and head in turn and join their sums in LDS; where sequences and
// heads alone would leave compute units idle the length is split over
// workgroups and a second launch joins the parts (kv_token_split).
#include "kv_attn.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 4;
constexpr int kBlock = 64 * kWaves;
constexpr int kStep = 32;  // tokens per wave and step

template <int FMT, int D, int GS>
__global__ __launch_bounds__(kBlock, (D == 256 ? 1 : GS == 32 && D == 128 ? 2 : 3)) void kv_token_kernel(KvCache c, KvBatch b, Rows rows, Split sp,
                                                          float *__restrict__ part,
                                                          float2 *__restrict__ part_ml)
{
    constexpr int NG = D / GS, NP = GS / 16;
    __shared__ float os[kWaves][16][D + 4];
    __shared__ float2 ml[kWaves][16];
    __shared__ uint32_t pairs[FMT == Q4_NF4 ? 256 : 1];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, kg = lane >> 4;
    const int seq = blockIdx.z, h = blockIdx.y, ct = blockIdx.x / sp.parts, pt = blockIdx.x % sp.parts;
    const KvSeq s = kv_seq(b, seq);
    const int nrows = s.fresh * rows.group;
    if (ct * 16 >= nrows)
        return;
    const int begin = range_begin(s, rows.window) + pt * sp.span;
    const int end = min(s.len, begin + sp.span);
    if (begin >= s.len && pt > 0)
        return;

    if constexpr (FMT == Q4_NF4) {
        pairs[tid] = nf4_pair(tid);
        __syncthreads();
    }

    // the lane's column: a new token's query head
    const int r0 = ct * 16 + i;
    const bool live = r0 < nrows;
    const int tok = live ? r0 / rows.group : 0;
    const int head = h * rows.group + (live ? r0 - tok * rows.group : 0);
    Queries<FMT, D, GS> q;
    q.load(rows.q + (int64_t)(s.first + tok) * rows.qts + (int64_t)head * rows.qhs, live, rows.act,
           rows.scale2, kg);
    const int pos = live ? s.len - s.fresh + tok : -1;  // sees low < t <= pos
    const int low = rows.window > 0 ? pos - rows.window : -1;
    // tokens that every live row sees need no mask
    const int all_to = s.len - s.fresh + ct * 16 / rows.group;
    const int all_from = rows.window > 0
        ? s.len - s.fresh + (min(ct * 16 + 16, nrows) - 1) / rows.group - rows.window + 1 : 0;

    const uint32_t sel = value_select<FMT, GS>(i);
    f32x4 o[NG][NP], oz[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        oz[j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < NP; ++n)
            o[j][n] = f32x4{0, 0, 0, 0};
    }
    float m = kNone, l = 0.0f;

    Pages pg{b.table + (int64_t)seq * b.table_width, c.page_shift, c.heads, h, c.pages, 0, 0, -1};
    pg.last = (s.len - 1) >> c.page_shift;
    pg.first = -1000;
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
        float x[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const f32x4 a = scores<FMT, D, GS>(kt[u], q, pairs);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[4 * u + r] = a[r];
        }
        const int64_t next0 = pg.row(tn, end, lane), next1 = pg.row(tn + 16, end, lane);
        if (tn < end) {
            kt[0].load(c, next0, lane);
            kt[1].load(c, next1, lane);
        }
        if (__builtin_expect(row0 < 0 || row1 < 0 || t0 + kStep - 1 > all_to || t0 < all_from, 0)) {
            const int ta = branch_only(t0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = (u ? row1 : row0) < 0 ? 0 : end - ta - 16 * u - 4 * kg;
                vt[u].keep(n);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = ta + 16 * u + 4 * kg + r;
                    x[4 * u + r] = r < n && at <= pos && at > low ? x[4 * u + r] : -__builtin_inff();
                }
            }
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < 8; ++e)
            top = fmaxf(top, x[e]);
        // (2^-40: rows of zeros do not pull the reference down)
        const float big = fmaxf(fmaxf(vt[0].largest(), vt[1].largest()), 0x1p-40f);
        const float reach = __builtin_fmaf(top, q.factor, __builtin_amdgcn_logf(big));
        if (__builtin_expect(__any(reach > m + 15.0f), 0)) {
            const float to = fmaxf(m, quad_max(reach) - 6.0f);
            const float f = __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                oz[j] *= f;
#pragma unroll
                for (int n = 0; n < NP; ++n)
                    o[j][n] *= f;
            }
        }
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], q.factor, -m));
            l += w[e];
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            u32x4 wp, va[NP];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int u = e >> 1, r = 2 * (e & 1);
                // (fma with 0: the scale's conversion is part of v_fma_mix)
                wp[e] = pair_h2(__builtin_fmaf(w[2 * e], vt[u].scale(r, j), 0.0f),
                                __builtin_fmaf(w[2 * e + 1], vt[u].scale(r + 1, j), 0.0f));
                uint32_t p[NP];
                value_pairs<FMT, GS>(vt[u].w[r][j], vt[u].w[r + 1][j], sel, pairs, p);
#pragma unroll
                for (int n = 0; n < NP; ++n)
                    va[n][e] = p[n];
            }
#pragma unroll
            for (int n = 0; n < NP; ++n)
                o[j][n] = mfma<Q4_F16>(va[n], wp, o[j][n]);
            if constexpr (kv_int<FMT>()) {
                u32x4 z = {0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u};
                if constexpr (FMT == Q4_INT4_ASYM) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int u = e >> 1, r = 2 * (e & 1);
                        z[e] = vt[u].zero(r, j) | vt[u].zero(r + 1, j) << 16;
                    }
                }
                oz[j] = mfma<Q4_F16>(z, wp, oz[j]);
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
    l = quad_sum(l);
    if (kg == 0)
        ml[wave][i] = float2{m, l};
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float unit = value_unit<FMT>() * (kv_int<FMT>() && (n & 1) ? 0.0625f : 1.0f);
                float v = o[j][n][r] * unit;
                if constexpr (kv_int<FMT>())
                    v -= oz[j][r] * value_unit<FMT>();
                os[wave][i][j * GS + NP * (4 * kg + r) + n] = v;
            }
    __syncthreads();
    for (int e = tid; e < 16 * D / 4; e += kBlock) {
        const int col = e / (D / 4), d = 4 * (e % (D / 4));
        const int row = ct * 16 + col;
        if (row >= nrows)
            continue;
        float mm = kNone;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            mm = fmaxf(mm, ml[w][col].x);
        f32x4 sum = {0, 0, 0, 0};
        float ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(ml[w][col].x - mm);
            ll += ml[w][col].y * f;
            sum += *(const f32x4 *)&os[w][col][d] * f;
        }
        const int tk = row / rows.group;
        const int64_t to = (int64_t)(s.first + tk) * rows.q_heads + h * rows.group + row - tk * rows.group;
        if (sp.parts == 1) {
            const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
            sum *= inv;
            u32x2 pk;
            pk[0] = rows.act == Q4_F16 ? pack_h2(sum[0], sum[1]) : pack_bf2(sum[0], sum[1]);
            pk[1] = rows.act == Q4_F16 ? pack_h2(sum[2], sum[3]) : pack_bf2(sum[2], sum[3]);
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
int most_parts(const KvCache &c, const KvBatch &b, int64_t tiles)
{
    if (b.max_len <= 512)
        return 1;
    const int64_t wgs = b.seqs * c.heads * tiles;
    return (int)std::min<int64_t>((1024 + wgs - 1) / wgs, (b.max_len + 255) / 256);
}

}  // namespace

Split token_split(const KvCache &c, const KvBatch &b, int group, int window)
{
    Split sp;
    sp.tiles = (int)(((int64_t)b.max_new * group + 15) / 16);
    const int64_t range = longest_range(b, window);
    const int64_t parts = range <= 512 ? 1 : most_parts(c, b, sp.tiles);
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
        kv_token_kernel<decltype(fmt)::value, decltype(dim)::value, decltype(gs)::value>
            <<<dim3(sp.parts * sp.tiles, c.heads, b.seqs), kBlock, 0, s>>>(c, b, rows, sp, part, part_ml);
        return hipGetLastError();
    });
}

}  // namespace q4
