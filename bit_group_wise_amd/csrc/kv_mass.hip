// kv_mass.hip -- the attention weight that each cached token draws, added to
// its mass (q4_kv_attention with mass).
//
// A token's mass is a sum over rows of 2^(x_t - stat): it needs every row's
// final statistics, so it is a second pass over the keys.  Scores come as in
// the attention kernels (16 tokens by 16 rows a product, exact levels, scales
// in binary32), so they are the same numbers.  A lane adds up the weights of
// its tokens over the rows it meets; the 16 columns meet once at the end, in a
// fixed order.
//
//  * Up to 8 rows: the attention kept the scores, in binary32; this pass only
//    reads them (kv_mass_kept_kernel).
//  * Few rows (as kv_token.hip takes), else: the rows stay in registers and a
//    wave walks over 64-token blocks of a span.  Bound as kv_token.hip.
//  * Many rows: 64 tokens' keys stay in registers, unpacked once, and the rows
//    pass by as operands that a first launch laid out (kv_rows_kernel), with
//    their factors and statistics.  The four waves of a workgroup hold 256
//    tokens and read the same rows, from the L1.  Bound by vector-ALU issue:
//    a score costs its groups' scales, an fma, exp2 at a quarter rate, a sum:
//    at 8 issue slots with two groups, 220 us for the 1.05e9 visible scores of
//    1024 new tokens after 31744 (8 heads of 4 rows, dim 128, g 64), which take
//    285 to 305 us (72 % of the slots); 32 x 4096 tokens of kept scores take 6 us.
#include "kv_attn.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 4;
constexpr int kBlock = 64 * kWaves;
constexpr int kBlk = 64;  // tokens of a wave at a time
constexpr int kMaxKept = 8;  // rows whose scores are kept

// 16 TT tokens' keys as operands, with the scales of the lane's rows.
template <int FMT, int D, int GS, int TT>
struct Keys {
    static constexpr int NG = D / GS, ZB = (NG + 1) / 2;
    u32x4 op[TT][D / 32];
    f32x4 s[TT][NG];
    uint32_t there;  // bit tt: the tile's page exists

    __device__ __forceinline__ void load(const KvCache &c, Pages &pg, int t0, int end, int lane, const uint32_t *pairs)
    {
        const int i = lane & 15, kg = lane >> 4;
        uint32_t w[TT][D / 32], z[TT];
        there = 0;
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
            const int64_t row0 = pg.row(t0 + 16 * tt, end, lane);
            there |= (row0 >= 0 ? 1u : 0u) << tt;
            const int64_t row = row0 >= 0 ? row0 : 0;
            const uint8_t *kc = c.k.codes + row * (D / 2);
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                w[tt][k] = *(const uint32_t *)(kc + (uint32_t)(i * (D / 2) + 16 * k + 4 * kg));
#pragma unroll
            for (int j = 0; j < NG; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    s[tt][j][r] = kv_scale<FMT>(c.k, row + 4 * kg + r, NG, j);
            if constexpr (FMT == Q4_INT4_ASYM) {
                const uint8_t *zp = c.k.zeros + row * ZB + (uint32_t)(i * ZB);
                if constexpr (ZB == 1)
                    z[tt] = *zp;
                else if constexpr (ZB == 2)
                    z[tt] = *(const uint16_t *)zp;
                else
                    z[tt] = *(const uint32_t *)zp;
            }
        }
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                op[tt][k] = key_operand<FMT>(
                    w[tt][k], key_zero(FMT == Q4_INT4_ASYM ? (z[tt] >> (4 * (k * 32 / GS))) & 15u : 8u), pairs);
    }
};

// Scores of tile tt by the lane's column, in units of the column's factor.
template <int FMT, int D, int GS, int TT>
__device__ __forceinline__ f32x4 tile_scores(const Keys<FMT, D, GS, TT> &k, int tt, const u32x4 *q)
{
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < D / GS; ++j) {
        f32x4 a = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < GS / 32; ++e)
            a = mfma<Q4_F16>(k.op[tt][j * (GS / 32) + e], q[j * (GS / 32) + e], a);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r] = __builtin_fmaf(a[r], k.s[tt][j][r], x[r]);
    }
    return x;
}

// Sum over the 16 lanes of a column tile, every lane the same bits.
template <int ROT>
__device__ __forceinline__ float add_rotated(float v)
{
    return v + std::bit_cast<float>(__builtin_amdgcn_update_dpp(0, std::bit_cast<int>(v), 0x120 + ROT, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float v)
{
    return add_rotated<1>(add_rotated<2>(add_rotated<4>(add_rotated<8>(v))));
}

// Adds a wave's 4 N sums (lane's tokens 16 (e / 4) + 4 kg + e % 4) to the mass.
template <int N>
__device__ __forceinline__ void add_mass(float (&sum)[N], float *mass, int t0, int len, uint32_t there, int lane)
{
    const int i = lane & 15, kg = lane >> 4;
    float v = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float s = sum16(sum[e]);
        v = i == e ? s : v;
    }
    const int at = t0 + 16 * (i >> 2) + 4 * kg + (i & 3);
    if (i < N && at < len && (there >> (i >> 2) & 1))
        mass[at] += v;
}

template <int FMT, int D, int GS, int NT>
__global__ __launch_bounds__(kBlock) void kv_mass_few_kernel(KvCache c, KvBatch b, Rows rows, int span,
                                                             float *__restrict__ mass, int64_t mass_width)
{
    constexpr int NG = D / GS;
    using M = Meta<FMT, NG, 64>;
    __shared__ typename M::Lds share[kWaves];
    __shared__ uint32_t pairs[FMT == Q4_NF4 ? 256 : 1];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int seq = blockIdx.z, h = blockIdx.y;
    const KvSeq s = kv_seq(b, seq);
    const int nrows = s.fresh * rows.group;
    const int begin = range_begin(s, rows.window) + (int)blockIdx.x * span, end = min(s.len, begin + span);
    if (begin >= end || nrows == 0)
        return;
    if constexpr (FMT == Q4_NF4) {
        pairs[tid] = nf4_pair(tid);
        __syncthreads();
    }
    ColQueries<FMT, D, GS, NT> q;
    q.load(s, rows, h, 0, lane);
    float st[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = ColQueries<FMT, D, GS, NT>::row(n, lane);
        const bool live = row < nrows;
        const int tok = live ? row / rows.group : 0;
        const int head = h * rows.group + (live ? row - tok * rows.group : 0);
        const float v = rows.stat[(int64_t)(s.first + tok) * rows.q_heads + head];
        // a row counts once, in its first group's column; rows that see
        // nothing weigh nothing anywhere
        st[n] = live && i % NG == 0 && v != -__builtin_inff() ? v : __builtin_inff();
    }
    const int all_to = s.len - s.fresh, all_from = rows.window > 0 ? s.len - rows.window : 0;
    Pages pg{b.table + (int64_t)seq * b.table_width, c.page_shift, c.heads, h, c.pages, 1 << 30,
             (s.len - 1) >> c.page_shift, -1};
    KeyCodes<FMT, D, GS> k[4];
    M meta;
    uint32_t there = 0;
    auto load_block = [&](int t0) {
        int64_t mine = 0;
        there = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t row0 = pg.row(t0 + 16 * u, end, lane);
            there |= (row0 >= 0 ? 1u : 0u) << u;
            mine = kg == u ? max(row0, (int64_t)0) + i : mine;
            k[u].load(c, row0, lane);
        }
        meta.load(c.k, mine);
    };
    int t0 = begin + wave * kBlk;
    if (t0 < end)
        load_block(t0);
    for (; t0 < end; t0 += kWaves * kBlk) {
        typename M::Lds &mt = share[wave];
        const uint32_t here = there;
        float sum[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            sum[e] = 0.0f;
        wave_order();
        meta.put(mt, lane);
        wave_order();
        f32x4 x[4][NT];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            Scales4<FMT> ks;
            ks.get(mt.s[i % NG], 16 * u + 4 * kg);
            const uint32_t z = FMT == Q4_INT4_ASYM ? key_zeros<D, GS>(mt.z, 16 * u + i, kg) : 0u;
            col_scores<FMT, D, GS, NT>(k[u], z, ks, q, pairs, x[u]);
        }
        if (t0 + kWaves * kBlk < end)
            load_block(t0 + kWaves * kBlk);
        if (__builtin_expect(t0 + kBlk - 1 > all_to || t0 < all_from, 0)) {
            const int ta = branch_only(t0);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = ta + 16 * u + 4 * kg + r;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        x[u][n][r] = at <= q.pos[n] && at > q.low[n] ? x[u][n][r] : -__builtin_inff();
                }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                sum[e] += __builtin_amdgcn_exp2f(__builtin_fmaf(x[e >> 2][n][e & 3], q.factor[n], -st[n]));
        add_mass(sum, mass + ((int64_t)seq * c.heads + h) * mass_width, t0, end, here, lane);
    }
}

constexpr int kKeptTokens = 4 * kBlock;

// The same from the scores that the attention kept: four tokens a thread.
// W: rows read at a time (4 where their number is a multiple of four).
template <int W>
__global__ __launch_bounds__(kBlock) void kv_mass_kept_kernel(KvBatch b, Rows rows, int heads, float *__restrict__ mass,
                                                              int64_t mass_width)
{
    __shared__ float st[kMaxKept];
    const int seq = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
    const KvSeq s = kv_seq(b, seq);
    const int nrows = s.fresh * rows.group, begin = range_begin(s, rows.window);
    const int n = s.len - begin, t0 = (int)blockIdx.x * kKeptTokens + tid;
    if ((int)blockIdx.x * kKeptTokens >= n || nrows == 0)
        return;
    if (tid < nrows) {
        const int tok = tid / rows.group;
        const float v = rows.stat[(int64_t)(s.first + tok) * rows.q_heads + h * rows.group + tid - tok * rows.group];
        st[tid] = v == -__builtin_inff() ? __builtin_inff() : v;  // rows that see nothing weigh nothing
    }
    __syncthreads();
    const float *x = rows.kept + ((int64_t)seq * heads + h) * rows.kept_range * rows.kept_rows;
    float *m = mass + ((int64_t)seq * heads + h) * mass_width + begin;
    float sum[4] = {0, 0, 0, 0}, old[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int t = min(t0 + k * kBlock, n - 1);  // (past the end: read and not used)
        old[k] = m[t];
        for (int r = 0; r < nrows; r += W) {
            float v[W];
            if constexpr (W == 4) {
                const f32x4 y = *(const f32x4 *)(x + (int64_t)t * rows.kept_rows + r);
                v[0] = y[0], v[1] = y[1], v[2] = y[2], v[3] = y[3];
            } else {
                v[0] = x[(int64_t)t * rows.kept_rows + r];
            }
#pragma unroll
            for (int e = 0; e < W; ++e)  // (rows past a sequence's own are not)
                sum[k] += r + e < nrows ? __builtin_amdgcn_exp2f(v[e] - st[r + e]) : 0.0f;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (t0 + k * kBlock < n)
            m[t0 + k * kBlock] = old[k] + sum[k];
}

// Rows as operands: tile t of head h holds 16 rows of a sequence, the
// sequence's first tile being floor(first * group / 16) + seq (so sequences
// never share one).
struct RowTiles {
    u32x4 *op;     // [tiles][heads][D / 32][64]
    float2 *fs;    // [tiles][heads][16]: factor, statistics
};
__device__ __forceinline__ int64_t first_tile(const KvSeq &s, int group, int seq)
{
    return ((int64_t)s.first * group >> 4) + seq;
}

template <int FMT, int D, int GS>
__global__ __launch_bounds__(64) void kv_rows_kernel(KvCache c, KvBatch b, Rows rows, RowTiles to)
{
    const int seq = blockIdx.z, h = blockIdx.y, t = blockIdx.x, lane = threadIdx.x, i = lane & 15;
    const KvSeq s = kv_seq(b, seq);
    const int nrows = s.fresh * rows.group;
    if (16 * t >= nrows)
        return;
    const int row = 16 * t + i;
    const bool live = row < nrows;
    const int tok = live ? row / rows.group : 0;
    const int head = h * rows.group + (live ? row - tok * rows.group : 0);
    Queries<FMT, D, GS> q;
    q.load(rows.q + (int64_t)(s.first + tok) * rows.qts + (int64_t)head * rows.qhs, live, rows.act, rows.scale2,
           lane >> 4);
    const int64_t at = (first_tile(s, rows.group, seq) + t) * c.heads + h;
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
        to.op[(at * (D / 32) + k) * 64 + lane] = q.op[k];
    if (lane < 16) {
        // rows that see nothing, and none at all, weigh nothing anywhere
        const float st = live ? rows.stat[(int64_t)(s.first + tok) * rows.q_heads + head] : -__builtin_inff();
        to.fs[at * 16 + i] = float2{q.factor, st == -__builtin_inff() ? __builtin_inff() : st};
    }
}

template <int FMT, int D, int GS, int TT>
__global__ __launch_bounds__(kBlock, 2) void kv_mass_many_kernel(KvCache c, KvBatch b, int group, int window, RowTiles from,
                                                              float *__restrict__ mass, int64_t mass_width)
{
    __shared__ uint32_t pairs[FMT == Q4_NF4 ? 256 : 1];
    constexpr int BLK = 16 * TT;  // tokens of a wave
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.x, seq = blockIdx.z;
    const KvSeq s = kv_seq(b, seq);
    if constexpr (FMT == Q4_NF4) {
        for (int e = tid; e < 256; e += blockDim.x)
            pairs[e] = nf4_pair(e);
        __syncthreads();
    }
    const int t0 = range_begin(s, window) + ((int)blockIdx.y * (int)(blockDim.x >> 6) + wave) * BLK;
    if (t0 >= s.len)
        return;
    Pages pg{b.table + (int64_t)seq * b.table_width, c.page_shift, c.heads, h, c.pages, 1 << 30,
             (s.len - 1) >> c.page_shift, -1};
    Keys<FMT, D, GS, TT> k;
    k.load(c, pg, t0, s.len, lane, pairs);
    float sum[4 * TT];
#pragma unroll
    for (int e = 0; e < 4 * TT; ++e)
        sum[e] = 0.0f;
    // the row tiles that see any of the tokens: new tokens from t0 - base on,
    // and with a window those less than `window` past the last
    const int base = s.len - s.fresh, nrows = s.fresh * group;
    int rt = max(t0 - base, 0) * group >> 4, rt_end = (nrows + 15) >> 4;
    if (window > 0) {
        const int64_t past = (int64_t)t0 + BLK - 1 + window - base;  // first new token past every window
        if (past * group < nrows)
            rt_end = min(rt_end, (int)((max(past, (int64_t)0) * group + 15) >> 4));
    }
    // rows that see all the tokens: from the last one's on, and inside every window
    const int from_row = max(t0 + BLK - 1 - base, 0) * group;
    const int64_t past = window > 0 ? ((int64_t)t0 + window - base) * group : INT32_MAX;
    const int to_row = (int)min(max(past, (int64_t)0), (int64_t)INT32_MAX);
    const int64_t at0 = first_tile(s, group, seq);
    const u32x4 *op = from.op + ((at0 + rt) * c.heads + h) * (D / 32) * 64 + lane;
    const float2 *fs = from.fs + ((at0 + rt) * c.heads + h) * 16 + i;
    const int64_t op_step = (int64_t)c.heads * (D / 32) * 64, fs_step = (int64_t)c.heads * 16;
    u32x4 q[D / 32];
    float2 next;
    if (rt < rt_end) {
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            q[e] = op[64 * e];
        next = *fs;
    }
    for (; rt < rt_end; ++rt) {
        float x[4 * TT];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
            const f32x4 y = tile_scores<FMT, D, GS>(k, tt, q);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[4 * tt + r] = y[r];
        }
        // the next tile's rows come while this one's weights are formed
        const float2 f = next;
        if (rt + 1 < rt_end) {
            op += op_step;
            fs += fs_step;
        }
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            q[e] = op[64 * e];
        next = *fs;
        if (__builtin_expect(16 * rt < from_row || 16 * rt + 15 >= to_row, 0)) {
            const int pos = branch_only(base) + (16 * rt + i) / group, low = window > 0 ? pos - window : -1;
#pragma unroll
            for (int e = 0; e < 4 * TT; ++e) {
                const int at = t0 + 16 * (e >> 2) + 4 * kg + (e & 3);
                x[e] = at <= pos && at > low ? x[e] : -__builtin_inff();
            }
        }
#pragma unroll
        for (int e = 0; e < 4 * TT; ++e)
            sum[e] += __builtin_amdgcn_exp2f(__builtin_fmaf(x[e], f.x, -f.y));
    }
    add_mass(sum, mass + ((int64_t)seq * c.heads + h) * mass_width, t0, s.len, k.there, lane);
}

bool is_few(const KvCache &c, const KvBatch &b, int group) { return (int64_t)b.max_new * group <= few_rows(c); }

int64_t row_tiles(const KvBatch &b, int group) { return (b.tokens * group >> 4) + b.seqs; }

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

// Scores of up to 8 rows a head are kept between the passes where they take at
// most 1 GiB: 4 bytes a row and token, written and read once, against half a
// cached row to read and unpack again.  (32 x 4096 tokens, 8 heads, g 64, whole
// calls, kept and formed anew: 8 rows of dim 128 46 and 54 us, 16 rows 69 and 77;
// 8 rows of dim 64 38 and 42, 16 rows 48 and 43, 32 rows 93 and 56.  One bound
// for all widths; the workspace grows with the rows.)
size_t kv_kept_bytes(const KvCache &c, const KvBatch &b, int group, int window)
{
    const int64_t rows = (int64_t)b.max_new * group;
    const double n = 4.0 * rows * b.seqs * c.heads * longest_range(b, window);
    return rows <= kMaxKept && rows <= few_rows(c) && n <= 0x1p30 ? (size_t)n : 0;
}

size_t kv_mass_workspace(const KvCache &c, const KvBatch &b, int group)
{
    if (is_few(c, b, group))
        return 0;
    const size_t n = (size_t)row_tiles(b, group) * c.heads;
    return round256(n * 16 * sizeof(float2)) + n * c.dim * 32;
}

hipError_t launch_kv_mass(int f, const KvCache &c, const KvBatch &b, const Rows &rows, float *mass,
                          int64_t mass_width, void *workspace, hipStream_t s)
{
    const int64_t range = longest_range(b, rows.window);
    if (range == 0)
        return hipSuccess;
    if (rows.kept) {
        const dim3 grid((unsigned)((range + kKeptTokens - 1) / kKeptTokens), c.heads, b.seqs);
        if (rows.kept_rows % 4 == 0)
            kv_mass_kept_kernel<4><<<grid, kBlock, 0, s>>>(b, rows, c.heads, mass, mass_width);
        else
            kv_mass_kept_kernel<1><<<grid, kBlock, 0, s>>>(b, rows, c.heads, mass, mass_width);
        return hipGetLastError();
    }
    return kv_by_shape(f, c.dim, c.g, [&](auto fmt, auto dim, auto gs) {
        constexpr int F = decltype(fmt)::value, D = decltype(dim)::value, GS = decltype(gs)::value;
        const int per = kWaves * kBlk;
        if (is_few(c, b, rows.group)) {
            // spans of whole rounds, at most four workgroups a compute unit
            // (32 x 4096 tokens: 512 workgroups 28.6 us, 1024 24.1, 2048 27.6)
            const int64_t wgs = (int64_t)b.seqs * c.heads;
            const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(1024 / wgs, (range + per - 1) / per));
            const int64_t span = ((range + parts - 1) / parts + per - 1) / per * per;
            const dim3 grid((unsigned)((range + span - 1) / span), c.heads, b.seqs);
            const int64_t cols = (int64_t)b.max_new * rows.group * (D / GS);
            if (cols <= 16)
                kv_mass_few_kernel<F, D, GS, 1><<<grid, kBlock, 0, s>>>(c, b, rows, (int)span, mass, mass_width);
            else if (cols <= 32)
                kv_mass_few_kernel<F, D, GS, 2><<<grid, kBlock, 0, s>>>(c, b, rows, (int)span, mass, mass_width);
            else if constexpr (D == 64)
                kv_mass_few_kernel<F, D, GS, 4><<<grid, kBlock, 0, s>>>(c, b, rows, (int)span, mass, mass_width);
            return hipGetLastError();
        }
        const size_t n = (size_t)row_tiles(b, rows.group) * c.heads;
        const RowTiles t{(u32x4 *)((char *)workspace + round256(n * 16 * sizeof(float2))), (float2 *)workspace};
        kv_rows_kernel<F, D, GS><<<dim3((unsigned)(((int64_t)b.max_new * rows.group + 15) / 16), c.heads, b.seqs), 64, 0, s>>>(
            c, b, rows, t);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        // 64 tokens a wave (dim 256: 32, by registers); four waves share the
        // rows they read, unless that leaves compute units without one (whole
        // calls of 256 rows, single waves and fours: 256 waves 41.5 and 48.3 us,
        // 1024 61.2 and 62.2, 2048 75.1 and 73.0, 4096 116 and 109.5)
        constexpr int TT = D == 256 ? 2 : 4;
        const int64_t waves = (range + 16 * TT - 1) / (16 * TT);
        const int w = waves * c.heads * b.seqs >= 2048 ? kWaves : 1;
        kv_mass_many_kernel<F, D, GS, TT><<<dim3(c.heads, (unsigned)((waves + w - 1) / w), b.seqs), 64 * w, 0, s>>>(
            c, b, rows.group, rows.window, t, mass, mass_width);
        return hipGetLastError();
    });
}

}  // namespace q4
