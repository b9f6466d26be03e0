// kv_prompt.hip -- attention over the 4-bit cache for many rows a head: prompts
// and chunks of them (q4_kv_attention).
//
// Mathematics: as in kv_token.hip (one pass, running reference, scores in
// powers of two, K as exact levels with one accumulator per scale group).
// With many rows the unpacking is shared: a workgroup turns a tile of cached
// tokens into matrix operands in LDS once, for all its rows.
//
//  * Keys lie there as exact fp16 levels less zero-points, their scales beside
//    them in binary32; a score is sum_j s_j acc_j as before.
//  * Values lie there as fp16(level * s_tj 2^-E_t), at most one rounding of the
//    cached value.  2^E_t is the token's size: E_t is added to its score, which
//    puts it into the weight, and taken off the row sum again.  Table formats
//    and single groups take the largest scale itself, so that its group's levels
//    are exact (of an NF4 cache in groups of 64, half of them); several groups of
//    INT4 the power of two that puts it just below 2^12, by which fp16 scales
//    stay exact and small levels round to themselves.  So a row meets a token's size only in what it sees of it (a
//    size shared by several tokens would let one that a row does not see take
//    the others' bits), and neither weights (at most 2^15.5) nor values (at
//    most 61440) leave fp16: groups down to 2^-21 of their token's largest
//    keep all their bits.  (The reference puts the largest weight at 2^11: it
//    moves rarely, and weights down to 2^-25 of the largest are exact to fp16's
//    11 bits.)
//  * For fp16 outputs a second product adds what rounding the weights left
//    (TWO): 2.1e-4 to 2.8e-4 from binary64, 2.1e-4 of it the output's own
//    rounding, where 3.0e-4 to 3.4e-4 were; it costs a fifth (137 us for 113
//    below).  A bf16 output is 1.7e-3 off either way.
//  * LDS holds operands as the lanes read them, 16 bytes a lane in a row, in
//    two buffers: the next tile is fetched while one is worked on, one barrier
//    a tile.  Rows of V operands are values d = 8 i + j of the dword i that a
//    staging lane unpacked, so both its writes and a result's stores are
//    contiguous.
//
// Bound: vector-ALU issue.  A score costs about eleven issue slots (its groups'
// scales, the exponent's fma, maximum, reference, exp2 at a quarter rate, sum,
// rounding; one size a wave's tokens would save one: 110 us where this takes 113)
// against 4 D / 1024 of matrix time; tiles are 64 tokens (dim 128) by 16 NT
// rows a wave, eight waves, so that a row pays little of the unpacking.  Of the
// chunk below the vector ALUs are busy 60 % of the time, the matrix cores 32 %
// (of the prompts, whose workgroups end unevenly, 50 and 23 %); the rest is the
// barrier a tile and the staging waves' wait for their loads.  dim 128, g 64:
//   2 x 2048 new tokens, 32 heads, causal, INT4-sym       113 us, 595 TFLOP/s
//   1024 after 31744, 8 heads of 4 rows, INT4-asym        662 us, 817 TFLOP/s
#include "kv_attn.hpp"

namespace q4 {
namespace {

constexpr int kWaves = 8;
constexpr int kBlock = 64 * kWaves;
constexpr int kStagers = 256;  // lanes that stage keys; as many stage values

// 16-row column tiles a wave: two where rows are many (one for dim 256, whose
// sums take the registers); one, with room for a second workgroup on the unit,
// where they are few.
template <int D>
constexpr int most_nt() { return D == 256 ? 1 : 2; }
constexpr int block_rows(int nt) { return 16 * nt * kWaves; }
// Tokens a tile: one staging item of 32 keys or 32 values a lane.
template <int D>
constexpr int prompt_tile() { return 32 * kStagers / D; }

// Value d of an output operand's row rho in product n (the rows are the
// nibbles j of dwords i, d = 8 i + j).
template <int D>
__device__ __forceinline__ int out_value(int n, int rho)
{
    if constexpr (D == 64)
        return 8 * (rho >> 1) + 2 * n + (rho & 1);
    else if constexpr (D == 128)
        return 8 * rho + n;
    else
        return 8 * (rho + 16 * (n >> 3)) + (n & 7);
}
// And the operand and row of nibble j of dword i.
template <int D>
__device__ __forceinline__ int operand_slot(int i, int j)  // (n * 64 + rho)
{
    if constexpr (D == 64)
        return (j >> 1) * 64 + 2 * i + (j & 1);
    else if constexpr (D == 128)
        return j * 64 + i;
    else
        return (j + 8 * (i >> 4)) * 64 + (i & 15);
}

// The largest scale of a token, its D / 8 staging lanes holding their group's
// (those of a group alike; none is negative, so as integers they compare the
// same): mirrored in 8 lanes, rotated by 8 in 16, and across 16.
template <int D, int GS>
__device__ __forceinline__ float token_max(float v)
{
    int u = std::bit_cast<int>(v);
    if constexpr (GS == 32)
        u = max(u, __builtin_amdgcn_update_dpp(0, u, 0x141, 0xf, 0xf, true));
    if constexpr (GS <= 64 && D >= 128)
        u = max(u, __builtin_amdgcn_update_dpp(0, u, 0x128, 0xf, 0xf, true));
    if constexpr (D == 256) {  // (the even rows of 16 twice, and the odd ones)
        const auto rows = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        u = max((int)rows[0], (int)rows[1]);
    }
    return std::bit_cast<float>(u);
}

// A staging lane's share of a tile as it is in memory: 32 keys of a token (the
// first four waves), or a dword of values of four tokens (the others).
template <int FMT, int D, int GS>
struct Fetch {
    static constexpr int NG = D / GS, ZB = (NG + 1) / 2, TT = prompt_tile<D>(), ND = D / 8;
    uint32_t w[4], s[4], z[4];  // as stored
    uint32_t ok;                // keys: the token is there; values: bit e, token e is

    // Keys: token u % TT, 32 values u / TT.  Values: dword u % ND of the four
    // tokens of quad u / ND, whose place tt in a 32-token step moves fastest.
    static __device__ __forceinline__ int k_token(int u) { return u % TT; }
    static __device__ __forceinline__ int k_chunk(int u) { return u / TT; }
    static __device__ __forceinline__ int v_dword(int u) { return u % ND; }
    static __device__ __forceinline__ int v_quad(int u)
    {
        const int p = u / ND;  // tt | kg << 1 | tb << 3
        return (p >> 3) * 8 + (p & 1) * 4 + ((p >> 1) & 3);
    }

    int64_t r;    // the row of the tile to load next
    bool in;      // which is there
    int t;        // and its token

    // Looks up where the tile from t0 lies.
    __device__ __forceinline__ void locate(const KvCache &c, Pages &pg, int t0, int end, int wave, int u)
    {
        const int lane = u & 63;
        const int p0 = min(t0, end - 1) >> c.page_shift, p1 = (min(t0 + TT, end) - 1) >> c.page_shift;
        if (p0 < pg.first || p1 - pg.first >= 64)
            pg.fetch(p0, lane);
        t = t0 + (wave < 4 ? k_token(u) : 4 * v_quad(u));
        const int id = __shfl(pg.mine, (min(t, end - 1) >> c.page_shift) - pg.first);
        in = t < end && (unsigned)id < (unsigned)c.pages;
        r = in ? (((int64_t)id * c.heads + pg.h) << c.page_shift) + (t & ((1 << c.page_shift) - 1)) : 0;
    }
    // One straight run of loads for both roles and every tile (past the end from
    // row 0): where branches met after their loads, the merged registers would
    // be copied, and so waited for, at once.
    __device__ __forceinline__ void load(const KvCache &c, int end, int wave, int u)
    {
        const bool keys = wave < 4;
        // keys: four dwords of a row, one scale; values: a dword and its scale
        // of four rows (which share a page; those past the end are not used)
        const int first = keys ? 4 * k_chunk(u) : v_dword(u);
        const int j = keys ? min(k_chunk(u), NG - 1) : 8 * first / GS;
        const int step = keys ? 4 : D / 2, rows = keys ? 0 : 1;
        const KvHalf &x = keys ? c.k : c.v;
        const uint8_t *p = x.codes + r * (D / 2) + 4 * first;
        const int zj = 8 * first / GS;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = *(const uint32_t *)(p + e * step);
            s[e] = scale_bits<FMT>(x, (r + e * rows) * NG + j);
            if constexpr (FMT == Q4_INT4_ASYM)
                z[e] = x.zeros[(r + e * rows) * ZB + (zj >> 1)];
        }
        const int left = in ? min(end - t, 4) : 0;
        ok = (1u << left) - 1;
    }
};

// Whether a token's size is its largest scale itself, or the power of two above.
template <int FMT, int D, int GS>
constexpr bool whole_scale() { return !kv_int<FMT>() || D == GS; }

template <int FMT, int D, int GS>
struct Stage {
    static constexpr int NG = D / GS, TT = prompt_tile<D>();
    u32x4 k[TT * D / 8];        // [16 tokens][D / 32] operands of 64 lanes
    u32x2 v[TT * D / 4];        // [32 tokens][D / 16] operands, halves of lanes
    float ks[NG][TT];           // (four at a time, as the next two: 16 bytes aligned)
    float e[TT], down[TT];      // E_t, and 2^-E_t
    uint32_t valid[TT / 32];
};

template <int FMT, int D, int GS>
__device__ __forceinline__ void stage(Stage<FMT, D, GS> &st, const Fetch<FMT, D, GS> &f, int wave, int u,
                                      const uint32_t *pairs)
{
    using F = Fetch<FMT, D, GS>;
    constexpr int TT = F::TT;
    const int lane = u & 63;
    if (wave < 4) {
        const int t = F::k_token(u), ch = F::k_chunk(u);
        if (ch < F::NG)
            st.ks[ch][t] = f.ok & 1 ? scale_of<FMT>(f.s[0]) : 0.0f;
        const uint64_t in = __ballot(f.ok & 1);
        const int word = 2 * wave + lane;
        if (lane < 2 && word < TT / 32)
            st.valid[word] = (uint32_t)(in >> (32 * lane));
        const KeyZero z = key_zero(FMT == Q4_INT4_ASYM ? (f.z[0] >> (4 * (32 * ch / GS & 1))) & 15u : 8u);
        u32x4 *to = st.k + ((t >> 4) * (D / 32) + ch) * 64 + (t & 15);
#pragma unroll
        for (int kg = 0; kg < 4; ++kg)
            to[16 * kg] = key_operand<FMT>(f.w[kg], z, pairs);
        return;
    }
    // values: four tokens' eight, scaled by 2^-E, then by value
    const int i = F::v_dword(u), qd = F::v_quad(u), j = 8 * i / GS;
    float s[4];
    [[maybe_unused]] float size = 0.0f;  // of token i % 4
    [[maybe_unused]] f32x4 e, down;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        s[t] = f.ok >> t & 1 ? scale_of<FMT>(f.s[t]) : 0.0f;
        // (2^-40: a token of zeros has a weight in the row sum all the same,
        // which must not vanish beside large ones)
        const float top = fmaxf(token_max<D, GS>(s[t]), 0x1p-40f);
        if constexpr (whole_scale<FMT, D, GS>()) {
            constexpr float up = FMT == Q4_NF4 ? 4.0f : FMT == Q4_FP4 ? 1024.0f : 4096.0f;
            s[t] *= __builtin_amdgcn_rcpf(top) * up;
            size = (i & 3) == t ? top * (key_unit<FMT>() / up) : size;
        } else {
            const int e2 = min(__builtin_amdgcn_frexp_expf(top), 100) - 12;
            e[t] = (float)e2;
            down[t] = __builtin_amdgcn_ldexpf(1.0f, -e2);
            s[t] *= down[t];
        }
    }
    if constexpr (whole_scale<FMT, D, GS>()) {
        // (a token a lane: transcendentals take four slots; 56 rows of dim 256 on
        // 4 x 110266 FP4 g32 tokens 186 us, 198 with all four in every lane)
        if (i < 4) {
            const float log_size = __builtin_amdgcn_logf(size);
            st.e[4 * qd + i] = log_size;
            st.down[4 * qd + i] = __builtin_amdgcn_exp2f(-log_size);
        }
    } else if (i == 0) {
        *(f32x4 *)&st.e[4 * qd] = e;
        *(f32x4 *)&st.down[4 * qd] = down;
    }
    uint32_t x[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const u32x4 a = key_operand<FMT>(
            f.w[t], key_zero(FMT == Q4_INT4_ASYM ? (f.z[t] >> (4 * (j & 1))) & 15u : 8u), pairs);
        if constexpr (kv_int<FMT>()) {
            const uint32_t h = pair_h2(s[t], s[t]), q = pair_h2(s[t] * 0.0625f, s[t] * 0.0625f);
#pragma unroll
            for (int p = 0; p < 4; ++p)
                x[t][p] = std::bit_cast<uint32_t>(std::bit_cast<f16x2>(a[p]) * std::bit_cast<f16x2>(p & 1 ? q : h));
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p)
                x[t][p] = pair_h2(h2f(a[p] & 0xffffu) * s[t], h2f(a[p] >> 16) * s[t]);
        }
    }
    // quad qd = 8 tb + 4 tt + kg: half tt of lane (kg, row)
    u32x2 *to = st.v + (((qd >> 3) * (D / 16)) * 64 + 16 * (qd & 3)) * 2 + ((qd >> 2) & 1);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t lo = 0x05040100u, hi = 0x07060302u;
        // pair p holds values (p, p + 4) for INT4, (2p, 2p + 1) otherwise
        const int j0 = kv_int<FMT>() ? p : 2 * p, j1 = kv_int<FMT>() ? p + 4 : 2 * p + 1;
        to[2 * operand_slot<D>(i, j0)] = u32x2{__builtin_amdgcn_perm(x[1][p], x[0][p], lo),
                                               __builtin_amdgcn_perm(x[3][p], x[2][p], lo)};
        to[2 * operand_slot<D>(i, j1)] = u32x2{__builtin_amdgcn_perm(x[1][p], x[0][p], hi),
                                               __builtin_amdgcn_perm(x[3][p], x[2][p], hi)};
    }
}

template <int FMT, int D, int GS, int NT, bool TWO>
__global__ __launch_bounds__(kBlock, (NT < most_nt<D>() ? 4 : 2)) void kv_prompt_kernel(KvCache c, KvBatch b, Rows rows, Split sp,
                                                              float *__restrict__ part,
                                                              float2 *__restrict__ part_ml)
{
    constexpr int NG = D / GS, R = block_rows(NT), TT = prompt_tile<D>(), NV = D / 16;
    constexpr int TB = TT >= 64 && NT == most_nt<D>() ? 2 : 1;   // 32-token steps worked on together
    constexpr int VF = NV < 8 || NT < most_nt<D>() ? 4 : 8;  // value operands fetched together
    constexpr int KT = D == 256 || NT < most_nt<D>() ? 1 : 2;  // 16-token halves of a step whose keys are fetched together
    __shared__ Stage<FMT, D, GS> st[2];
    __shared__ uint32_t pairs[FMT == Q4_NF4 ? 256 : 1];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, kg = lane >> 4;
    // heads fastest (a head's blocks share an XCD's L2 where heads fill all
    // eight), the blocks with most to see first
    int id = blockIdx.x;
    const int h = id % c.heads;
    id /= c.heads;
    const int seq = id % b.seqs;
    id /= b.seqs;
    const int pt = id % sp.parts, blk = sp.tiles - 1 - id / sp.parts;
    const KvSeq s = kv_seq(b, seq);
    const int nrows = s.fresh * rows.group, base = s.len - s.fresh;
    if (blk * R >= nrows)
        return;
    const int pos_min = base + blk * R / rows.group, pos_max = base + (min(blk * R + R, nrows) - 1) / rows.group;
    int begin = rows.window > 0 ? max(0, pos_min - rows.window + 1) & ~15 : 0;
    int end = pos_max + 1;
    if (sp.parts > 1) {
        const int p0 = range_begin(s, rows.window) + pt * sp.span;
        begin = max(begin, p0);
        end = min(end, p0 + sp.span);
    }
    if constexpr (FMT == Q4_NF4) {
        if (tid < 256)
            pairs[tid] = nf4_pair(tid);
        __syncthreads();
    }

    const int w0 = blk * R + wave * 16 * NT;  // the wave's first row
    Queries<FMT, D, GS> q[NT];
    int pos[NT], low[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = w0 + 16 * n + i;
        const bool live = r < nrows;
        const int tok = live ? r / rows.group : 0;
        const int head = h * rows.group + (live ? r - tok * rows.group : 0);
        q[n].load(rows.q + (int64_t)(s.first + tok) * rows.qts + (int64_t)head * rows.qhs, live, rows.act,
                  rows.scale2, kg);
        pos[n] = live ? base + tok : -1;
        low[n] = rows.window > 0 ? pos[n] - rows.window : -1;
    }
    // tokens that all the wave's live rows see, and that any sees
    const int last = min(w0 + 16 * NT, nrows) - 1;
    const int all_to = base + w0 / rows.group, any_to = last < w0 ? -1 : base + last / rows.group;
    const int all_from = rows.window > 0 ? any_to - rows.window + 1 : 0;
    const int any_from = rows.window > 0 ? all_to - rows.window + 1 : 0;

    f32x4 o[NV][NT];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = kNone;
        l[n] = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            o[v][n] = f32x4{0, 0, 0, 0};
    }

    Pages pg{b.table + (int64_t)seq * b.table_width, c.page_shift, c.heads, h, c.pages, 1 << 30, 0, -1};
    pg.last = (end - 1) >> c.page_shift;
    Fetch<FMT, D, GS> f;
    if (begin < end) {
        f.locate(c, pg, begin, end, wave, tid & 255);
        f.load(c, end, wave, tid & 255);
    }
    int buf = 0;
    for (int t0 = begin; t0 < end; t0 += TT, buf ^= 1) {
        f.locate(c, pg, t0 + TT, end, wave, tid & 255);
        stage<FMT, D, GS>(st[buf], f, wave, tid & 255, pairs);
        f.load(c, end, wave, tid & 255);
        __syncthreads();
        const Stage<FMT, D, GS> &S = st[buf];
#pragma unroll 1
        for (int tb = 0; tb < TT / 32; tb += TB) {
            const int t1 = t0 + 32 * tb;
            if (t1 > any_to || t1 + 32 * TB - 1 < any_from)
                continue;
            uint32_t valid[TB];
            float x[TB][NT][8];
            bool whole = t1 + 32 * TB - 1 <= all_to && t1 >= all_from;
#pragma unroll
            for (int b2 = 0; b2 < TB; ++b2) {
                valid[b2] = __builtin_amdgcn_readfirstlane(S.valid[tb + b2]);
                whole = whole && valid[b2] == ~0u;
            }
            // An LDS read takes about as long as ten products: operands are
            // asked for well before their use, those of a step's keys (KT of
            // its two halves) together, those of its values before the softmax
            // (the scheduler would fetch them one by one to save registers).
#pragma unroll
            for (int b2 = 0; b2 < TB; ++b2)
#pragma unroll
                for (int t2 = 0; t2 < 2; t2 += KT) {
                    u32x4 ka[KT][D / 32];
                    f32x4 ks[KT][NG];
#pragma unroll
                    for (int u = 0; u < KT; ++u) {
                        const int tt = t2 + u;
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            ka[u][k] = S.k[((2 * (tb + b2) + tt) * (D / 32) + k) * 64 + lane];
#pragma unroll
                        for (int j = 0; j < NG; ++j)
                            ks[u][j] = *(const f32x4 *)&S.ks[j][32 * (tb + b2) + 16 * tt + 4 * kg];
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int u = 0; u < KT; ++u)
#pragma unroll
                        for (int j = 0; j < NG; ++j)
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                f32x4 a = {0, 0, 0, 0};
#pragma unroll
                                for (int k = 0; k < GS / 32; ++k)
                                    a = mfma<Q4_F16>(ka[u][j * (GS / 32) + k], q[n].op[j * (GS / 32) + k], a);
                                float *y = x[b2][n] + 4 * (t2 + u);
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    y[r] = j == 0 ? a[r] * ks[u][j][r] : __builtin_fmaf(a[r], ks[u][j][r], y[r]);
                            }
                }
            u32x4 va[VF];
            auto fetch_values = [&](int b2, int v0) {
#pragma unroll
                for (int v = 0; v < VF; ++v)
                    va[v] = *(const u32x4 *)&S.v[(((tb + b2) * NV + v0 + v) * 64 + lane) * 2];
                __builtin_amdgcn_sched_barrier(0);
            };
            fetch_values(0, 0);
            if (__builtin_expect(!whole, 0)) {
                const int ta = branch_only(t1), k4 = 4 * (int)opaque_word(kg);
#pragma unroll
                for (int b2 = 0; b2 < TB; ++b2) {
                    const uint32_t here = valid[b2] >> k4;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int at = 16 * (k >> 2) + (k & 3), t = ta + 32 * b2 + k4 + at;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            x[b2][n][k] = (here >> at & 1) && t <= pos[n] && t > low[n] ? x[b2][n][k] : -__builtin_inff();
                    }
                }
            }
            float reach[NT];
            bool move = false;
#pragma unroll
            for (int b2 = 0; b2 < TB; ++b2) {
                const f32x4 e[2] = {*(const f32x4 *)&S.e[32 * (tb + b2) + 4 * kg],
                                    *(const f32x4 *)&S.e[32 * (tb + b2) + 16 + 4 * kg]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float top = b2 ? reach[n] : -__builtin_inff();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        x[b2][n][k] = __builtin_fmaf(x[b2][n][k], q[n].factor, e[k >> 2][k & 3]);
                        top = fmaxf(top, x[b2][n][k]);
                    }
                    reach[n] = top;
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
                move = move || reach[n] > m[n] + 15.5f;
            if (__builtin_expect(__any(move), 0)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float to = fmaxf(m[n], quad_max(reach[n]) - 11.0f);
                    const float g = __builtin_amdgcn_exp2f(m[n] - to);
                    m[n] = to;
                    l[n] *= g;
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        o[v][n] *= g;
                }
            }
#pragma unroll
            for (int b2 = 0; b2 < TB; ++b2) {
                const f32x4 down[2] = {*(const f32x4 *)&S.down[32 * (tb + b2) + 4 * kg],
                                       *(const f32x4 *)&S.down[32 * (tb + b2) + 16 + 4 * kg]};
                u32x4 w[NT], left[TWO ? NT : 1];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float sum = 0.0f, p[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        p[k] = __builtin_amdgcn_exp2f(x[b2][n][k] - m[n]);
                        sum = __builtin_fmaf(p[k], down[k >> 2][k & 3], sum);
                    }
                    l[n] += sum;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        w[n][k] = pair_h2(p[2 * k], p[2 * k + 1]);
                        if constexpr (TWO)
                            left[n][k] = pair_h2(p[2 * k] - h2f(w[n][k] & 0xffffu), p[2 * k + 1] - h2f(w[n][k] >> 16));
                    }
                }
#pragma unroll
                for (int v0 = 0; v0 < NV; v0 += VF) {
                    if (v0)
                        fetch_values(b2, v0);
#pragma unroll
                    for (int v = 0; v < VF; ++v)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if constexpr (TWO)
                                o[v0 + v][n] = mfma<Q4_F16>(va[v], left[n], o[v0 + v][n]);
                            o[v0 + v][n] = mfma<Q4_F16>(va[v], w[n], o[v0 + v][n]);
                        }
                }
                if (b2 + 1 < TB)
#pragma unroll
                    for (int v = 0; v < VF; ++v)
                        va[v] = *(const u32x4 *)&S.v[(((tb + b2 + 1) * NV + v) * 64 + lane) * 2];
            }
        }
    }

#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float ll = quad_sum(l[n]);
        const int r0 = w0 + 16 * n + i;
        if (r0 >= nrows)
            continue;
        const int tok = r0 / rows.group;
        const int64_t to = (int64_t)(s.first + tok) * rows.q_heads + h * rows.group + r0 - tok * rows.group;
        const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
        // a lane's rows 4 kg .. + 3 of all products are runs of 8 values
        constexpr int RUNS = D / 32;
#pragma unroll
        for (int run = 0; run < RUNS; ++run) {
            float v[8];
            int d = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                int nv, r;
                if constexpr (D == 64)
                    nv = k >> 1, r = 2 * run + (k & 1);
                else if constexpr (D == 128)
                    nv = k, r = run;
                else
                    nv = k + 8 * (run >> 2), r = run & 3;
                v[k] = o[nv][n][r];
                if (k == 0)
                    d = out_value<D>(nv, 4 * kg + r);
            }
            if (sp.parts == 1) {
                u32x4 pk;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    pk[k] = rows.act == Q4_F16 ? pack_h2(v[2 * k] * inv, v[2 * k + 1] * inv)
                                               : pack_bf2(v[2 * k] * inv, v[2 * k + 1] * inv);
                *(u32x4 *)(rows.out + to * D + d) = pk;
            } else {
                float *p = part + (to * sp.parts + pt) * D + d;
                *(f32x4 *)p = f32x4{v[0], v[1], v[2], v[3]};
                *(f32x4 *)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
            }
        }
        if (kg == 0) {
            if (sp.parts > 1) {
                part_ml[to * sp.parts + pt] = float2{m[n], ll};
            } else {
                const float v = ll > 0.0f ? row_stat(m[n], ll) : -__builtin_inff();
                if (rows.lse)
                    rows.lse[to] = v * kLn2;
                if (rows.stat)
                    rows.stat[to] = v;
            }
        }
    }
}

}  // namespace

// Row tiles of 256 (dim 256: 128) rows fill the 256 compute units, one
// workgroup each, or are split into as many parts as do, none shorter than 256
// tokens.  Where even that leaves units idle or rows empty, tiles of 128 rows,
// two workgroups a unit.  Calls in large and in small tiles (8 heads of dim 128,
// INT4-sym g 64): rows that a large tile would half fill, 4 x 100 on 2048 28.3 and
// 27.6 us; units idle, 1024 on 1024 31.2 and 25.5, 6 x 1024 on 2048 91.7 and 85.1;
// units filled, 1024 x 4 rows on 32768 680 and 797, 3 x 4096 x 4 on 4096 639 and
// 852, 8 x 1024 on 2048 93 and 91.  (Whole prompts that just fill the units are
// faster in small tiles all the same, their last rows having twice the mean to
// see: 32 heads of 2048 on 2048 92 and 77; not told apart.)  Parts of at least
// 128, 256 and 512 tokens: 64 on 4096 21.7, 18.2 and 23.0, on 1024 14.1, 15.9, 22.2.
Split prompt_split(const KvCache &c, const KvBatch &b, int group, int window)
{
    const int64_t range = longest_range(b, window), rows = (int64_t)b.max_new * group;
    auto with = [&](int nt, int64_t room) {
        Split sp;
        sp.rows = block_rows(nt);
        sp.tiles = (int)((rows + sp.rows - 1) / sp.rows);
        const int64_t wgs = (int64_t)b.seqs * c.heads * sp.tiles;
        const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(room / wgs, range / 256));
        sp.span = (int)std::max<int64_t>(((range + parts - 1) / parts + 127) / 128 * 128, 128);
        sp.parts = (int)std::max<int64_t>((range + sp.span - 1) / sp.span, 1);
        return sp;
    };
    if (c.dim == 256)
        return with(1, 256);
    const Split big = with(2, 256);
    return rows <= 128 || (int64_t)b.seqs * c.heads * big.tiles * big.parts < 224 ? with(1, 512) : big;
}

hipError_t launch_kv_prompt(int f, const KvCache &c, const KvBatch &b, const Rows &rows, const Split &sp,
                            float *part, float2 *part_ml, hipStream_t s)
{
    return kv_by_shape(f, c.dim, c.g, [&](auto fmt, auto dim, auto gs) {
        const int64_t grid = (int64_t)sp.parts * sp.tiles * b.seqs * c.heads;
        constexpr int F = decltype(fmt)::value, D = decltype(dim)::value, GS = decltype(gs)::value;
        auto go = [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            if (rows.act == Q4_F16)
                kv_prompt_kernel<F, D, GS, NT, true><<<dim3((unsigned)grid), kBlock, 0, s>>>(c, b, rows, sp, part, part_ml);
            else
                kv_prompt_kernel<F, D, GS, NT, false><<<dim3((unsigned)grid), kBlock, 0, s>>>(c, b, rows, sp, part, part_ml);
        };
        if (sp.rows == block_rows(most_nt<D>()))
            go(KvInt<most_nt<D>()>{});
        else
            go(KvInt<1>{});
        return hipGetLastError();
    });
}

}  // namespace q4
