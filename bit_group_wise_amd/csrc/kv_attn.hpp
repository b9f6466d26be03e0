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

// How a launch divides a sequence's range of cached tokens and its rows.
struct Split {
    int span;   // tokens a part
    int parts;
    int tiles;  // row tiles a head
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

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&to)[N], const void *from)
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

// Sixteen tokens' keys as they are in memory, a lane's share: row i's dwords
// 4 m + kg, the scales of rows 4 kg .. + 3, row i's zero-points.
template <int FMT, int D, int GS>
struct KeyTile {
    static constexpr int NG = D / GS, ZB = (NG + 1) / 2, SB = f32_absmax(FMT) ? 4 : 2;
    uint32_t w[D / 32], s[NG * SB], z;

    __device__ __forceinline__ void load(const KvCache &c, int64_t row0, int lane)
    {
        const int i = lane & 15, kg = lane >> 4;
        const int64_t row = row0 >= 0 ? row0 : 0;  // (page 0 is read and not used)
        const uint8_t *kc = c.k.codes + row * (D / 2);
#pragma unroll
        for (int m = 0; m < D / 32; ++m)
            w[m] = *(const uint32_t *)(kc + (uint32_t)(i * (D / 2) + 16 * m + 4 * kg));
        load_words(s, (const char *)c.k.scales + row * (NG * SB) + (uint32_t)(4 * kg * NG * SB));
        if constexpr (FMT == Q4_INT4_ASYM) {
            const uint8_t *zp = c.k.zeros + row * ZB + (uint32_t)(i * ZB);
            if constexpr (ZB == 1)
                z = *zp;
            else if constexpr (ZB == 2)
                z = *(const uint16_t *)zp;
            else
                z = *(const uint32_t *)zp;
        }
    }
    __device__ __forceinline__ float scale(int r, int j) const
    {
        const int e = r * NG + j;
        if constexpr (f32_absmax(FMT))
            return std::bit_cast<float>(s[e]);
        else
            return h2f((s[e >> 1] >> (16 * (e & 1))) & 0xffffu);
    }
    __device__ __forceinline__ KeyZero zero(int j) const
    {
        return key_zero(FMT == Q4_INT4_ASYM ? (z >> (4 * j)) & 15u : 8u);
    }
};

// Sixteen tokens' values, a lane's share of rows 4 kg .. + 3: one dword a
// group, the scales, the zero-points.
template <int FMT, int D, int GS>
struct ValueTile {
    static constexpr int NG = D / GS, ZB = (NG + 1) / 2, SB = f32_absmax(FMT) ? 4 : 2;
    uint32_t w[4][NG], s[NG * SB], z[FMT == Q4_INT4_ASYM ? ZB : 1];

    __device__ __forceinline__ void load(const KvCache &c, int64_t row0, int lane)
    {
        const int i = lane & 15, kg = lane >> 4;
        const int64_t row = row0 >= 0 ? row0 : 0;
        const uint8_t *vc = c.v.codes + row * (D / 2);
        const uint32_t vo = 4 * kg * (D / 2) + 4 * value_dword<GS>(i);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < NG; ++j)
                w[r][j] = *(const uint32_t *)(vc + vo + (uint32_t)(r * (D / 2) + j * (GS / 2)));
        load_words(s, (const char *)c.v.scales + row * (NG * SB) + (uint32_t)(4 * kg * NG * SB));
        if constexpr (FMT == Q4_INT4_ASYM)
            load_words(z, c.v.zeros + row * ZB + (uint32_t)(4 * kg * ZB));
    }
    __device__ __forceinline__ float scale(int r, int j) const
    {
        const int e = r * NG + j;
        if constexpr (f32_absmax(FMT))
            return std::bit_cast<float>(s[e]);
        else
            return h2f((s[e >> 1] >> (16 * (e & 1))) & 0xffffu);
    }
    // The scales of rows at and past `n` become 0 (rows of the lane count from
    // 4 kg).
    __device__ __forceinline__ void keep(int n)
    {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const int e = r * NG + j;
                if constexpr (f32_absmax(FMT))
                    s[e] = r < n ? s[e] : 0u;
                else
                    s[e >> 1] = r < n ? s[e >> 1] : s[e >> 1] & (e & 1 ? 0x0000ffffu : 0xffff0000u);
            }
    }
    // The largest scale (none is negative).
    __device__ __forceinline__ float largest() const
    {
        if constexpr (f32_absmax(FMT)) {
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 4 * NG; ++e)
                m = fmaxf(m, std::bit_cast<float>(s[e]));
            return m;
        } else {
            f16x2 m = std::bit_cast<f16x2>(s[0]);
#pragma unroll
            for (int e = 1; e < 2 * NG; ++e)
                m = __builtin_elementwise_max(m, std::bit_cast<f16x2>(s[e]));
            return fmaxf((float)m[0], (float)m[1]);
        }
    }
    __device__ __forceinline__ uint32_t zero(int r, int j) const
    {
        const int byte = r * ZB + (j >> 1);
        return (z[byte >> 2] >> (8 * (byte & 3) + 4 * (j & 1))) & 15u;
    }
};

// Scores of 16 tokens (rows 4 kg + r of the tile) by the lane's column, in
// units of the column's factor.
template <int FMT, int D, int GS>
__device__ __forceinline__ f32x4 scores(const KeyTile<FMT, D, GS> &t, const Queries<FMT, D, GS> &q,
                                        const uint32_t *pairs)
{
    f32x4 x = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < D / GS; ++j) {
        const KeyZero z = t.zero(j);
        f32x4 a = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < GS / 32; ++k)
            a = mfma<Q4_F16>(key_operand<FMT>(t.w[j * (GS / 32) + k], z, pairs), q.op[j * (GS / 32) + k], a);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r] = __builtin_fmaf(a[r], t.scale(r, j), x[r]);
    }
    return x;
}

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
hipError_t launch_kv_prompt(int f, const KvCache &c, const KvBatch &b, const Rows &rows, const Split &sp,
                            float *part, float2 *part_ml, hipStream_t s);
size_t kv_mass_workspace(const KvCache &c, const KvBatch &b, int group);
hipError_t launch_kv_mass(int f, const KvCache &c, const KvBatch &b, const Rows &rows, float *mass,
                          int64_t mass_width, void *workspace, hipStream_t s);

}  // namespace q4
