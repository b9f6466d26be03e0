// kv_attn.hpp -- what the attention kernels over the 4-bit cache share: the
// launch's description, page numbers, queries and rows as operands.
#pragma once

#include <algorithm>

#include "kv_mfma.hpp"

namespace q4 {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -1.0e30f;  // reference before any token

// A wave-uniform value that is only known inside the branch that asks for it:
// what is computed from it stays in there, where the optimizer would otherwise
// compute the masks of the few tiles that need them for all.
__device__ __forceinline__ int branch_only(int v)
{
    asm volatile("" : "+s"(v));
    return v;
}
__device__ __forceinline__ uint32_t branch_only_lane(uint32_t v)  // the same, a value a lane
{
    asm volatile("" : "+v"(v));
    return v;
}

// Where a launch puts a row's result.
struct Rows {
    const uint16_t *q;
    int64_t qts, qhs;
    int q_heads, group, act, window;
    float scale2;  // scale * log2(e)
    uint16_t *out;
    float *lse;    // natural log, or null
    float *stat;   // base-2 log of the denominator for the mass pass, or null
    float *kept;   // the scores themselves for it, or null: [seqs][heads]
                   // [kept_range tokens from range_begin][kept_rows]
    int64_t kept_range;
    int kept_rows;
};

// How a launch divides a sequence's range of cached tokens and its rows.
struct Split {
    int span;   // tokens a part
    int parts;
    int tiles;  // row tiles a head
    int rows;   // rows a tile (prompts)
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

// m + log2(l), the base-2 log of a row's denominator, l > 0.  The hardware's
// logarithm is up to a last place low, so it is asked for a number in [-1, 0): of
// l itself, some 2^25 here, it left all of a row's weights 5e-7 to 1e-6 too large.
__device__ __forceinline__ float row_stat(float m, float l)
{
    return (m + (float)__builtin_amdgcn_frexp_expf(l)) + __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(l));
}

// The range of cached tokens that a sequence's rows can see.
__device__ __forceinline__ int range_begin(const KvSeq &s, int window)
{
    return window > 0 ? max(0, s.len - s.fresh - window + 1) & ~15 : 0;
}

// The power of two that puts a row's largest query just below 2^12, and the
// factor from products with rows of levels to scores in powers of two.
__device__ __forceinline__ float query_factor(float largest, float scale2, float unit, float &factor)
{
    // 2^e > the largest value >= 2^(e-1); both powers are normal numbers
    int e = 0;
    if (largest > 0.0f)
        e = min(max(__builtin_amdgcn_frexp_expf(largest), -110), 128);
    // (never 0, which would make a masked score's -inf a NaN; scores of such
    // rows are 0 to any precision)
    factor = fmaxf(__builtin_amdgcn_ldexpf(scale2, e - 12) * unit, 0x1p-120f);
    return __builtin_amdgcn_ldexpf(1.0f, 12 - e);
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
        const float f = query_factor(quad_max(m), scale2, key_unit<FMT>(), factor);
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
            op[k] = query_operand<FMT>(raw[k], act, f);
    }
};

// Columns of the few-row kernels.  A column is a row (a new token's query head)
// and a scale group: col = row * NG + group.  Its queries are zero outside the
// group, so a product over all of d leaves the group's share of the score, the
// lane scales it, and the shares of a row meet in neighbouring lanes.  So a
// head's rows fill the columns a tile has anyway, and the order of d within
// the product is free: lane kg takes d = D/4 kg .. + D/4 - 1 of a key row, one
// contiguous load.
template <int NG>
__device__ __forceinline__ float group_sum(float v)  // the same bits in all lanes of a row
{
    if constexpr (NG >= 2)
        v += std::bit_cast<float>(__builtin_amdgcn_update_dpp(0, std::bit_cast<int>(v), 0xb1, 0xf, 0xf, true));
    if constexpr (NG >= 4)
        v += std::bit_cast<float>(__builtin_amdgcn_update_dpp(0, std::bit_cast<int>(v), 0x4e, 0xf, 0xf, true));
    if constexpr (NG >= 8)  // (half mirror: the four lanes of a quad agree by now)
        v += std::bit_cast<float>(__builtin_amdgcn_update_dpp(0, std::bit_cast<int>(v), 0x141, 0xf, 0xf, true));
    return v;
}
template <int NG>
__device__ __forceinline__ float group_max(float v)
{
    if constexpr (NG >= 2)
        v = fmaxf(v, std::bit_cast<float>(__builtin_amdgcn_update_dpp(0, std::bit_cast<int>(v), 0xb1, 0xf, 0xf, true)));
    if constexpr (NG >= 4)
        v = fmaxf(v, std::bit_cast<float>(__builtin_amdgcn_update_dpp(0, std::bit_cast<int>(v), 0x4e, 0xf, 0xf, true)));
    if constexpr (NG >= 8)
        v = fmaxf(v, std::bit_cast<float>(__builtin_amdgcn_update_dpp(0, std::bit_cast<int>(v), 0x141, 0xf, 0xf, true)));
    return v;
}

// A scale as it is stored, and its value.  (A load's result is left alone until
// it is used: whatever touches it earlier waits for it.)
template <int FMT>
__device__ __forceinline__ uint32_t scale_bits(const KvHalf &x, int64_t i)
{
    return f32_absmax(FMT) ? ((const uint32_t *)x.scales)[i] : ((const uint16_t *)x.scales)[i];
}
template <int FMT>
__device__ __forceinline__ float scale_of(uint32_t s)
{
    return f32_absmax(FMT) ? std::bit_cast<float>(s) : h2f(s);
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&to)[N], const void *from)
{
    if constexpr (N == 4) {
        const u32x4 v = *(const u32x4 *)from;
        to[0] = v[0], to[1] = v[1], to[2] = v[2], to[3] = v[3];
    } else if constexpr (N == 2) {
        const u32x2 v = *(const u32x2 *)from;
        to[0] = v[0], to[1] = v[1];
    } else {
        to[0] = *(const uint32_t *)from;
    }
}

// What a wave keeps in LDS of the tokens it works on.  Every lane needs scales
// and values of four tokens that other lanes are next to in memory, and a
// load costs the texture path about 16 cycles however little it fetches
// (measured: 26-30 narrow loads a step kept it busy two thirds of the time).
// So memory is read in few wide loads and handed round through LDS, each wave
// in its own part (its LDS operations stay in order: no barrier).

// Orders a wave's LDS accesses for the compiler (a wave's lanes read what its
// other lanes wrote; the hardware keeps them in order by itself).
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Scales and zero-points, a token a lane, all its groups (32 tokens' keys and
// values, or 64 tokens' keys).
template <int FMT, int NG, int LANES>
struct Meta {
    static constexpr int SB = f32_absmax(FMT) ? 4 : 2, ZB = (NG + 1) / 2, SW = (NG * SB + 3) / 4;
    struct Lds {
        __attribute__((aligned(16))) uint8_t s[NG][LANES * SB];
        __attribute__((aligned(16))) uint8_t z[FMT == Q4_INT4_ASYM ? LANES * ZB : 16];
    };
    uint32_t s[SW], z;

    __device__ __forceinline__ void load(const KvHalf &x, int64_t row)
    {
        const char *p = (const char *)x.scales + row * (NG * SB);
        if constexpr (NG * SB == 2)
            s[0] = *(const uint16_t *)p;
        else if constexpr (SW == 1)
            s[0] = *(const uint32_t *)p;
        else if constexpr (SW == 2) {
            const u32x2 v = *(const u32x2 *)p;
            s[0] = v[0], s[1] = v[1];
        } else {
#pragma unroll
            for (int k = 0; k < SW / 4; ++k) {
                const u32x4 v = ((const u32x4 *)p)[k];
                s[4 * k] = v[0], s[4 * k + 1] = v[1], s[4 * k + 2] = v[2], s[4 * k + 3] = v[3];
            }
        }
        if constexpr (FMT == Q4_INT4_ASYM) {
            const uint8_t *zp = x.zeros + row * ZB;
            if constexpr (ZB == 1)
                z = *zp;
            else if constexpr (ZB == 2)
                z = *(const uint16_t *)zp;
            else
                z = *(const uint32_t *)zp;
        }
    }
    __device__ __forceinline__ void put(Lds &to, int lane) const
    {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            if constexpr (SB == 4)
                ((uint32_t *)to.s[j])[lane] = s[j];
            else
                ((uint16_t *)to.s[j])[lane] = (uint16_t)(s[j >> 1] >> (16 * (j & 1)));
        }
        if constexpr (FMT == Q4_INT4_ASYM) {
            if constexpr (ZB == 1)
                to.z[lane] = (uint8_t)z;
            else if constexpr (ZB == 2)
                ((uint16_t *)to.z)[lane] = (uint16_t)z;
            else
                ((uint32_t *)to.z)[lane] = z;
        }
    }
};
// The scales of tokens t .. t + 3 in a group.
template <int FMT>
struct Scales4 {
    uint32_t w[f32_absmax(FMT) ? 4 : 2];
    __device__ __forceinline__ void get(const uint8_t *row, int t)
    {
        if constexpr (f32_absmax(FMT)) {
            const u32x4 v = *(const u32x4 *)(row + 4 * t);
            w[0] = v[0], w[1] = v[1], w[2] = v[2], w[3] = v[3];
        } else {
            const u32x2 v = *(const u32x2 *)(row + 2 * t);
            w[0] = v[0], w[1] = v[1];
        }
    }
    __device__ __forceinline__ float operator[](int r) const
    {
        if constexpr (f32_absmax(FMT))
            return std::bit_cast<float>(w[r]);
        else
            return h2f((w[r >> 1] >> (16 * (r & 1))) & 0xffffu);
    }
    // Those from the n-th on become 0.
    __device__ __forceinline__ void keep(int n)
    {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (f32_absmax(FMT))
                w[r] = r < n ? w[r] : 0u;
            else
                w[r >> 1] = r < n ? w[r >> 1] : w[r >> 1] & (r & 1 ? 0x0000ffffu : 0xffff0000u);
        }
    }
    // The same, converted to binary32 in the branch that asks for them.
    __device__ __forceinline__ Scales4 branch_only() const
    {
        Scales4 s;
#pragma unroll
        for (int i = 0; i < (f32_absmax(FMT) ? 4 : 2); ++i)
            s.w[i] = branch_only_lane(w[i]);
        return s;
    }
    __device__ __forceinline__ float smallest() const
    {
        return fminf(fminf((*this)[0], (*this)[1]), fminf((*this)[2], (*this)[3]));
    }
    __device__ __forceinline__ float largest() const  // (no scale is negative)
    {
        return fmaxf(fmaxf((*this)[0], (*this)[1]), fmaxf((*this)[2], (*this)[3]));
    }
};

// The codes of 16 keys as they are in memory, a lane's share: values D/4 kg ..
// of row i.
template <int FMT, int D, int GS>
struct KeyCodes {
    static constexpr int NG = D / GS, ZB = (NG + 1) / 2, NW = D / 32;
    uint32_t w[NW];

    __device__ __forceinline__ void load(const KvCache &c, int64_t row0, int lane)
    {
        const int i = lane & 15, kg = lane >> 4;
        const int64_t row = row0 >= 0 ? row0 : 0;  // (page 0 is read and not used)
        const uint8_t *p = c.k.codes + row * (D / 2) + (uint32_t)(i * (D / 2) + kg * (D / 8));
        if constexpr (NW == 2) {
            const u32x2 v = *(const u32x2 *)p;
            w[0] = v[0], w[1] = v[1];
        } else {
#pragma unroll
            for (int m = 0; m < NW / 4; ++m) {
                const u32x4 v = ((const u32x4 *)p)[m];
                w[4 * m] = v[0], w[4 * m + 1] = v[1], w[4 * m + 2] = v[2], w[4 * m + 3] = v[3];
            }
        }
    }
    // Operand m of the row: values D/4 kg + 8 m .. + 7; z: the row's
    // zero-points, shifted to the group of value D/4 kg.
    __device__ __forceinline__ u32x4 operand(int m, uint32_t z, const uint32_t *pairs) const
    {
        uint32_t zp = 8;
        if constexpr (FMT == Q4_INT4_ASYM)
            zp = (z >> (4 * (8 * m / GS))) & 15u;
        return key_operand<FMT>(w[m], key_zero(zp), pairs);
    }
};
// Zero-points of the token `t` from LDS, for KeyCodes::operand.
template <int D, int GS>
__device__ __forceinline__ uint32_t key_zeros(const uint8_t *z, int t, int kg)
{
    constexpr int ZB = (D / GS + 1) / 2;
    const uint32_t v = ZB == 1 ? z[t] : ZB == 2 ? ((const uint16_t *)z)[t] : ((const uint32_t *)z)[t];
    return v >> (4 * (D / 4 * kg / GS));
}

// NT column tiles' queries as operands, and the factor from products to
// scores.
template <int FMT, int D, int GS, int NT>
struct ColQueries {
    static constexpr int NG = D / GS, NW = D / 32, ROWS = NT * 16 / NG;
    u32x4 op[NT][NW];
    float factor[NT];
    int pos[NT], low[NT];  // the row sees low < t <= pos

    // Row of the lane in column tile n, counted from the first.
    static __device__ __forceinline__ int row(int n, int lane) { return (16 * n + (lane & 15)) / NG; }

    __device__ __forceinline__ void load(const KvSeq &s, const Rows &rows, int h, int row0, int lane)
    {
        const int nrows = s.fresh * rows.group, kg = lane >> 4, g = lane % NG;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + row(n, lane);
            const bool live = r < nrows;
            const int tok = live ? r / rows.group : 0;
            const int head = h * rows.group + (live ? r - tok * rows.group : 0);
            const uint16_t *q = rows.q + (int64_t)(s.first + tok) * rows.qts + (int64_t)head * rows.qhs;
            pos[n] = live ? s.len - s.fresh + tok : -1;
            low[n] = rows.window > 0 ? pos[n] - rows.window : -1;
            u32x4 raw[NW];
            float m = 0.0f;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                raw[k] = live ? *(const u32x4 *)(q + (D / 4) * kg + 8 * k) : u32x4{0, 0, 0, 0};
                m = fmaxf(m, query_max(raw[k], rows.act));
            }
            const float f = query_factor(quad_max(m), rows.scale2, key_unit<FMT>(), factor[n]);
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const bool mine = ((D / 4) * kg + 8 * k) / GS == g;
                op[n][k] = query_operand<FMT>(mine ? raw[k] : u32x4{0, 0, 0, 0}, rows.act, f);
            }
        }
    }
};

// Scores of 16 tokens (4 kg + r of the tile) by the lane's row, in units of
// its factor.
template <int FMT, int D, int GS, int NT>
__device__ __forceinline__ void col_scores(const KeyCodes<FMT, D, GS> &t, uint32_t z, const Scales4<FMT> &s,
                                           const ColQueries<FMT, D, GS, NT> &q, const uint32_t *pairs,
                                           f32x4 (&x)[NT])
{
    f32x4 a[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        a[n] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < D / 32; ++m) {
        const u32x4 k = t.operand(m, z, pairs);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            a[n] = mfma<Q4_F16>(k, q.op[n][m], a[n]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)  // (fma with 0: the conversion is part of v_fma_mix)
            x[n][r] = group_sum<D / GS>(__builtin_fmaf(a[n][r], s[r], 0.0f));
}

// Rows that the few-row kernels take: four column tiles (dim 64) or two; the
// sums of more do not fit the registers.  At as many rows (INT4-sym, 8 heads, 1
// and 32 sequences of 4096 tokens; a call's time) against the prompt kernel:
// 16 rows of dim 128, g 64 12.9 and 42.5 us (14.9 and 70.2 there); 8 of dim 256,
// g 64 17.6 and 75 (18.8 and 158); 64 of dim 64, g 64 15.0 and 47.4 (13.5 and
// 54.8); at half as many no form is slower here.
inline int few_rows(const KvCache &c) { return (c.dim == 64 ? 64 : 32) / (c.dim / c.g); }

template <class F>
hipError_t kv_by_shape(int f, int dim, int g, F &&fn)
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

// Cached tokens that any row of a sequence sees, at most.
inline int64_t longest_range(const KvBatch &b, int window)
{
    const int64_t w = (int64_t)window + b.max_new + 15;  // (the range starts at a multiple of 16)
    return window > 0 && w < b.max_len ? w : b.max_len;
}

// The kernels' launchers; part and part_ml hold `parts` partial sums a row.
Split token_split(const KvCache &c, const KvBatch &b, int group, int window);
Split prompt_split(const KvCache &c, const KvBatch &b, int group, int window);
hipError_t launch_kv_token(int f, const KvCache &c, const KvBatch &b, const Rows &rows, const Split &sp,
                           float *part, float2 *part_ml, hipStream_t s);
hipError_t launch_kv_token_f16(int f, const KvCache &c, const KvBatch &b, const Rows &rows, const Split &sp,
                               float *part, float2 *part_ml, hipStream_t s);
hipError_t launch_kv_prompt(int f, const KvCache &c, const KvBatch &b, const Rows &rows, const Split &sp,
                            float *part, float2 *part_ml, hipStream_t s);
size_t kv_mass_workspace(const KvCache &c, const KvBatch &b, int group);
// Bytes of scores that few rows keep for the mass pass; 0: it forms them anew.
size_t kv_kept_bytes(const KvCache &c, const KvBatch &b, int group, int window);
hipError_t launch_kv_mass(int f, const KvCache &c, const KvBatch &b, const Rows &rows, float *mass,
                          int64_t mass_width, void *workspace, hipStream_t s);

}  // namespace q4
