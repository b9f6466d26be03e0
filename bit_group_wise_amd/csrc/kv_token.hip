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
#include <algorithm>

#include "kv_mfma.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 4;
constexpr int kBlock = 64 * kWaves;
constexpr int kStep = 32;  // tokens per wave and step
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -1.0e30f;  // reference before any token

// Where a launch puts a row's result.
struct Rows {
    const uint16_t *q;
    int64_t qts, qhs;
    int q_heads, group, act, window;
    float scale2;  // scale * log2(e)
    uint16_t *out;
    float *lse;    // natural log, or null
    float *stat;   // base-2 log of the denominator for the mass pass, or null
};

// Work of a launch: `span` tokens per workgroup, col tiles per head.
struct Split {
    int span, parts, tiles;
};

// Sixteen tokens' rows as they are in memory, a lane's share.
template <int FMT, int D, int GS>
struct Tile {
    static constexpr int NG = D / GS;                       // groups a row
    static constexpr int SW = f32_absmax(FMT) ? NG : (NG + 1) / 2;  // scale words a row (rounded up)
    static constexpr int ZB = (NG + 1) / 2;                 // zero-point bytes a row
    uint32_t kw[D / 32];
    uint32_t vw[4][NG];
    uint32_t ks[4 * NG * (f32_absmax(FMT) ? 2 : 1) / 2];    // 4 tokens' scales, in order
    uint32_t vs[4 * NG * (f32_absmax(FMT) ? 2 : 1) / 2];
    uint32_t kz;                                            // row i's zero-points (ZB bytes)
    uint32_t vz[FMT == Q4_INT4_ASYM ? ZB : 1];              // 4 tokens' bytes
    bool there;                                             // the page exists

    __device__ __forceinline__ void load(const KvCache &c, int64_t row0, int lane)
    {
        const int i = lane & 15, kg = lane >> 4;
        there = row0 >= 0;
        const int64_t row = there ? row0 : 0;  // (page 0 is read and not used)
        const uint8_t *kc = c.k.codes + row * (D / 2), *vc = c.v.codes + row * (D / 2);
#pragma unroll
        for (int m = 0; m < D / 32; ++m)
            kw[m] = *(const uint32_t *)(kc + (uint32_t)(i * (D / 2) + 16 * m + 4 * kg));
        const uint32_t vo = 4 * kg * (D / 2) + 4 * value_dword<GS>(i);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < NG; ++j)
                vw[r][j] = *(const uint32_t *)(vc + vo + (uint32_t)(r * (D / 2) + j * (GS / 2)));
        constexpr int SB = f32_absmax(FMT) ? 4 : 2;  // bytes a scale
        load_words(ks, (const char *)c.k.scales + row * (NG * SB) + (uint32_t)(4 * kg * NG * SB));
        load_words(vs, (const char *)c.v.scales + row * (NG * SB) + (uint32_t)(4 * kg * NG * SB));
        if constexpr (FMT == Q4_INT4_ASYM) {
            const uint8_t *z = c.k.zeros + row * ZB + (uint32_t)(i * ZB);
            if constexpr (ZB == 1)
                kz = *z;
            else if constexpr (ZB == 2)
                kz = *(const uint16_t *)z;
            else
                kz = *(const uint32_t *)z;
            load_words(vz, (const char *)c.v.zeros + row * ZB + (uint32_t)(4 * kg * ZB));
        }
    }
    template <int N>
    static __device__ __forceinline__ void load_words(uint32_t (&to)[N], const char *from)
    {
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int j = 0; j < N / 4; ++j) {
                const u32x4 v = ((const u32x4 *)from)[j];
                to[4 * j] = v[0], to[4 * j + 1] = v[1], to[4 * j + 2] = v[2], to[4 * j + 3] = v[3];
            }
        } else if constexpr (N == 2) {
            const u32x2 v = *(const u32x2 *)from;
            to[0] = v[0], to[1] = v[1];
        } else {
            to[0] = *(const uint32_t *)from;
        }
    }
    // Scale and zero-point of the lane's token 4 kg + r, group j.
    static __device__ __forceinline__ float scale(const uint32_t *s, int r, int j)
    {
        const int e = r * NG + j;
        if constexpr (f32_absmax(FMT))
            return std::bit_cast<float>(s[e]);
        else
            return h2f((s[e >> 1] >> (16 * (e & 1))) & 0xffffu);
    }
    static __device__ __forceinline__ uint32_t zero(const uint32_t *z, int r, int j)
    {
        const int byte = r * ZB + (j >> 1);
        return (z[byte >> 2] >> (8 * (byte & 3) + 4 * (j & 1))) & 15u;
    }
};

// The page numbers of a range, 64 at a time in one register across the lanes.
struct Pages {
    const int32_t *table;
    int shift, heads, h, pages, first, last, mine;
    __device__ __forceinline__ void fetch(int p0, int lane)
    {
        first = p0;
        mine = p0 + lane <= last ? table[p0 + lane] : -1;
    }
    // First row of the 16 tokens from t, or -1.
    __device__ __forceinline__ int64_t row(int t, int end, int lane)
    {
        if (t >= end)
            return -1;
        const int p = t >> shift;
        if (p - first >= 64 || p < first)
            fetch(p, lane);
        const int id = __builtin_amdgcn_readlane(mine, p - first);
        if ((unsigned)id >= (unsigned)pages)
            return -1;
        return (((int64_t)id * heads + h) << shift) + (t & ((1 << shift) - 1));
    }
};

__device__ __forceinline__ float quad_max(float v)  // over the four lanes of a column
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float quad_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// The range of cached tokens that a sequence's rows can see.
__device__ __forceinline__ int range_begin(const KvSeq &s, int window)
{
    return window > 0 ? max(0, s.len - s.fresh - window + 1) & ~15 : 0;
}

// A column's queries as operands, and the factor from products to scores.
template <int FMT, int D, int GS>
struct Queries {
    u32x4 op[D / 32];
    float factor;

    __device__ __forceinline__ void load(const uint16_t *q, bool live, int act, float scale2, int kg)
    {
        u32x4 raw[D / 32];
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            raw[k] = live ? *(const u32x4 *)(q + 32 * k + 8 * kg) : u32x4{0, 0, 0, 0};
            m = fmaxf(m, query_max(raw[k], act));
        }
        m = quad_max(m);
        // 2^e >= the largest value > 2^(e-1); both powers are normal numbers
        int e = 0;
        if (m > 0.0f)
            e = min(max(__builtin_amdgcn_frexp_expf(m), -110), 128);
        const float f = __builtin_amdgcn_ldexpf(1.0f, 12 - e);
        // (never 0, which would make a masked score's -inf a NaN; scores of
        // such rows are 0 to any precision)
        factor = fmaxf(__builtin_amdgcn_ldexpf(scale2, e - 12) * key_unit<FMT>(), 0x1p-120f);
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
            op[k] = query_operand<FMT>(raw[k], act, f);
    }
};

// Scores of 16 tokens (rows 4 kg + r of the tile) by the lane's column, in
// units of the column's factor.
template <int FMT, int D, int GS>
__device__ __forceinline__ f32x4 scores(const Tile<FMT, D, GS> &t, const Queries<FMT, D, GS> &q,
                                        const uint32_t *pairs)
{
    constexpr int NG = D / GS;
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        const KeyZero z = key_zero(FMT == Q4_INT4_ASYM ? (t.kz >> (4 * j)) & 15u : 8u);
        f32x4 a = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < GS / 32; ++k)
            a = mfma<Q4_F16>(key_operand<FMT>(t.kw[j * (GS / 32) + k], z, pairs), q.op[j * (GS / 32) + k], a);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r] = __builtin_fmaf(a[r], t.scale(t.ks, r, j), x[r]);
    }
    return x;
}

template <int FMT, int D, int GS>
__global__ __launch_bounds__(kBlock) void kv_token_kernel(KvCache c, KvBatch b, Rows rows, Split sp,
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
    Tile<FMT, D, GS> t[2];
    for (int t0 = begin + wave * kStep; t0 < end; t0 += kWaves * kStep) {
        t[0].load(c, pg.row(t0, end, lane), lane);
        t[1].load(c, pg.row(t0 + 16, end, lane), lane);
        const bool whole = t[0].there && t[1].there && t0 + kStep - 1 <= all_to && t0 >= all_from;
        float x[8], vs[NG][8];
        float top = -__builtin_inff(), big = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const f32x4 a = scores<FMT, D, GS>(t[u], q, pairs);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[4 * u + r] = a[r];
#pragma unroll
                for (int j = 0; j < NG; ++j)
                    vs[j][4 * u + r] = t[u].scale(t[u].vs, r, j);
            }
        }
        if (!whole) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = t0 + 16 * (e >> 2) + 4 * kg + (e & 3);
                const bool in = t[e >> 2].there && at < end;
                x[e] = in && at <= pos && at > low ? x[e] : -__builtin_inff();
#pragma unroll
                for (int j = 0; j < NG; ++j)
                    vs[j][e] = in ? vs[j][e] : 0.0f;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            top = fmaxf(top, x[e]);
#pragma unroll
            for (int j = 0; j < NG; ++j)
                big = fmaxf(big, vs[j][e]);
        }
        // (2^-40: rows of zeros do not pull the reference down)
        const float reach = __builtin_fmaf(top, q.factor, __builtin_amdgcn_logf(fmaxf(big, 0x1p-40f)));
        if (__any(reach > m + 15.0f)) {
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
                wp[e] = pack_h2(w[2 * e] * vs[j][2 * e], w[2 * e + 1] * vs[j][2 * e + 1]);
                uint32_t p[NP];
                const int u = e >> 1, r = 2 * (e & 1);
                value_pairs<FMT, GS>(t[u].vw[r][j], t[u].vw[r + 1][j], sel, pairs, p);
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
                        z[e] = t[u].zero(t[u].vz, r, j) | t[u].zero(t[u].vz, r + 1, j) << 16;
                    }
                }
                oz[j] = mfma<Q4_F16>(z, wp, oz[j]);
            }
        }
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

// Joins the parts of a row: one workgroup per new token and query head.
template <int D>
__global__ __launch_bounds__(D) void kv_join_kernel(KvBatch b, Rows rows, Split sp, const float *__restrict__ part,
                                                    const float2 *__restrict__ part_ml)
{
    const int seq = blockIdx.z, head = blockIdx.y, tok = blockIdx.x, d = threadIdx.x;
    const KvSeq s = kv_seq(b, seq);
    if (tok >= s.fresh)
        return;
    const int64_t to = (int64_t)(s.first + tok) * rows.q_heads + head;
    const int n = max(1, (s.len - range_begin(s, rows.window) + sp.span - 1) / sp.span);
    const float2 *ml = part_ml + to * sp.parts;
    float m = kNone;
    for (int p = 0; p < n; ++p)
        m = fmaxf(m, ml[p].x);
    float sum = 0.0f, l = 0.0f;
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
        const float f = __builtin_amdgcn_exp2f(ml[p].x - m);
        l += ml[p].y * f;
        sum += part[(to * sp.parts + p) * D + d] * f;
    }
    const float v = l > 0.0f ? sum / l : 0.0f;
    rows.out[to * D + d] = (uint16_t)(rows.act == Q4_F16 ? f2h_bits(v) : f2bf_bits(v));
    if (d == 0) {
        const float e = l > 0.0f ? m + __builtin_amdgcn_logf(l) : -__builtin_inff();
        if (rows.lse)
            rows.lse[to] = e * kLn2;
        if (rows.stat)
            rows.stat[to] = e;
    }
}

// mass[b, h, t] += sum over rows of 2^(x - stat), one wave per 32 tokens, the
// rows 16 at a time.  A row that sees nothing has stat = -inf and is skipped.
template <int FMT, int D, int GS>
__global__ __launch_bounds__(kBlock) void kv_mass_kernel(KvCache c, KvBatch b, Rows rows,
                                                         float *__restrict__ mass, int64_t mass_width)
{
    __shared__ uint32_t pairs[FMT == Q4_NF4 ? 256 : 1];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int seq = blockIdx.z, h = blockIdx.y;
    const KvSeq s = kv_seq(b, seq);
    if constexpr (FMT == Q4_NF4) {
        pairs[tid] = nf4_pair(tid);
        __syncthreads();
    }
    const int t0 = range_begin(s, rows.window) + ((int)blockIdx.x * kWaves + wave) * kStep;
    if (t0 >= s.len)
        return;
    Pages pg{b.table + (int64_t)seq * b.table_width, c.page_shift, c.heads, h, c.pages, -1000,
             (s.len - 1) >> c.page_shift, -1};
    Tile<FMT, D, GS> t[2];
    t[0].load(c, pg.row(t0, s.len, lane), lane);
    t[1].load(c, pg.row(t0 + 16, s.len, lane), lane);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int nrows = s.fresh * rows.group;
    for (int r0 = 0; r0 < nrows; r0 += 16) {
        const int row = r0 + i;
        const bool live = row < nrows;
        const int tok = live ? row / rows.group : 0;
        const int head = h * rows.group + (live ? row - tok * rows.group : 0);
        const int pos = live ? s.len - s.fresh + tok : -1;
        const int low = rows.window > 0 ? pos - rows.window : -1;
        Queries<FMT, D, GS> q;
        q.load(rows.q + (int64_t)(s.first + tok) * rows.qts + (int64_t)head * rows.qhs, live, rows.act,
               rows.scale2, kg);
        const float st = live ? rows.stat[(int64_t)(s.first + tok) * rows.q_heads + head] : 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const f32x4 a = scores<FMT, D, GS>(t[u], q, pairs);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int at = t0 + 16 * u + 4 * kg + r;
                const bool see = t[u].there && at <= pos && at > low;
                sum[4 * u + r] += see ? __builtin_amdgcn_exp2f(__builtin_fmaf(a[r], q.factor, -st)) : 0.0f;
            }
        }
    }
    // over the 16 columns, in a fixed order
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int d = 1; d < 16; d <<= 1)
            sum[e] += __shfl_xor(sum[e], d);
    if (i < 8) {
        float v = sum[0];
#pragma unroll
        for (int e = 1; e < 8; ++e)
            v = i == e ? sum[e] : v;
        const int at = t0 + 16 * (i >> 2) + 4 * kg + (i & 3);
        if (at < s.len)
            mass[((int64_t)seq * c.heads + h) * mass_width + at] += v;
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

// Cached tokens that any row of a sequence sees, at most.
int64_t longest_range(const KvBatch &b, int window)
{
    const int64_t w = (int64_t)window + b.max_new + 15;  // (the range starts at a multiple of 16)
    return window > 0 && w < b.max_len ? w : b.max_len;
}

Split split_for(const KvCache &c, const KvBatch &b, int group, int window)
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

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

template <class F>
hipError_t by_shape(int f, int dim, int g, F &&fn)
{
    return kv_by_format(f, [&](auto fmt) {
        switch (dim * 1000 + g) {
        case 64032: return fn(fmt, KvInt<64>{}, KvInt<32>{});
        case 64064: return fn(fmt, KvInt<64>{}, KvInt<64>{});
        case 128032: return fn(fmt, KvInt<128>{}, KvInt<32>{});
        case 128064: return fn(fmt, KvInt<128>{}, KvInt<64>{});
        case 128128: return fn(fmt, KvInt<128>{}, KvInt<128>{});
        case 256032: return fn(fmt, KvInt<256>{}, KvInt<32>{});
        case 256064: return fn(fmt, KvInt<256>{}, KvInt<64>{});
        case 256128: return fn(fmt, KvInt<256>{}, KvInt<128>{});
        }
        return hipErrorInvalidValue;
    });
}

}  // namespace

size_t kv_attention_workspace(int f, const KvCache &c, const KvBatch &b, int q_heads, bool mass)
{
    const int parts = most_parts(c, b, ((int64_t)b.max_new * (q_heads / c.heads) + 15) / 16);
    const size_t rows = (size_t)b.tokens * q_heads;
    size_t n = mass ? round256(rows * 4) : 0;
    if (parts > 1)
        n += round256(rows * parts * sizeof(float2)) + round256(rows * parts * c.dim * 4);
    return n;
}

hipError_t launch_kv_attention(int f, const KvCache &c, const KvBatch &b, int act_t, const void *q,
                               int64_t qts, int64_t qhs, int q_heads, float scale, int window,
                               void *out, float *lse, float *mass, int64_t mass_width,
                               void *workspace, hipStream_t s)
{
    const int group = q_heads / c.heads;
    const Split sp = split_for(c, b, group, window);
    const size_t n = (size_t)b.tokens * q_heads;
    char *w = (char *)workspace;
    Rows rows{(const uint16_t *)q, qts, qhs, q_heads, group, act_t, window, scale * kLog2e,
              (uint16_t *)out, lse, nullptr};
    if (mass) {
        rows.stat = (float *)w;
        w += round256(n * 4);
    }
    float2 *part_ml = (float2 *)w;
    float *part = (float *)(w + round256(n * sp.parts * sizeof(float2)));
    return by_shape(f, c.dim, c.g, [&](auto fmt, auto dim, auto gs) {
        constexpr int F = decltype(fmt)::value, D = decltype(dim)::value, GS = decltype(gs)::value;
        kv_token_kernel<F, D, GS><<<dim3(sp.parts * sp.tiles, c.heads, b.seqs), kBlock, 0, s>>>(
            c, b, rows, sp, part, part_ml);
        if (sp.parts > 1)
            kv_join_kernel<D><<<dim3(b.max_new, q_heads, b.seqs), D, 0, s>>>(b, rows, sp, part, part_ml);
        if (mass) {
            const int per = kWaves * kStep;
            const int64_t range = longest_range(b, window);
            kv_mass_kernel<F, D, GS><<<dim3((unsigned)((range + per - 1) / per), c.heads, b.seqs), kBlock, 0, s>>>(
                c, b, rows, mass, mass_width);
        }
        return hipGetLastError();
    });
}

}  // namespace q4
