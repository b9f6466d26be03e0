// lora.hpp -- shared by the kernels of low-rank adapters beside a 4-bit
// weight (q4_lora_*).
//
// An adapter adds s (x A^T) B^T to a row's product.  The rows' h = s x A^T
// (and for gradients u = s dy B) are formed first, summed in binary32, and left
// in the workspace; the product's own kernel then adds h B^T (or u A) to its
// binary32 accumulators, so the sum is rounded once and y is written once.
//
// Operands: the matrix cores take 16 bits, so h and u enter as three bfloat16
// numbers, each the first 8 bits of what the ones before it left: all 24 bits of
// binary32 (and its range: nothing is lost of a gradient below fp16's).  What
// they meet is bfloat16 as it is, or for fp16 activations two such numbers (11
// bits = 8 + 3), of which the second and the third of h are not multiplied: below
// 2^-21 of the product, 2^-24 in the mean.  (With two numbers, 16 bits, one in 400
// bfloat16 gradients of a long batch rounded otherwise than its exact value; now
// one in 2700, of the plain binary32 form one in 1200.)
#pragma once

#include "plan.hpp"
#include "q4_common.hpp"
#include "q4_mfma.hpp"

namespace q4 {

// h[m][r] (or u) and what they go through.  For few rows h is left as binary32
// partial sums, part[i * rows * rank + m * rank + r] for i < parts; else as its
// operands, split[(3 m + i) * rank + r] for i < 3.
struct LowRank {
    const float *part;
    int parts;
    const uint16_t *split;
    int rank, adapters;
    int64_t rows;
    const int32_t *ids;  // adapter of each row, or NULL: all 0
    const uint16_t *w;   // B [adapters, N, rank] or A [adapters, rank, K]
};

// Adapter of row m (-1: none).
__device__ __forceinline__ int adapter_of(const int32_t *__restrict__ ids, int adapters, int64_t m)
{
    const int a = ids ? ids[m] : 0;
    return (uint32_t)a < (uint32_t)adapters ? a : -1;
}

// 16 rows of a mask, from a wave-uniform one; a lane's own is looked up in these 32
// bits.  A 64-bit shift reads its amount as a pair of registers, and on gfx950,
// if the second of the pair lies past the wave's, may take it from register 0.
// (The compiler keeps that from happening for gfx90a only.)
__device__ __forceinline__ uint32_t rows16(uint64_t mask, int from)
{
    return (uint32_t)(mask >> from) & 0xffffu;
}

// Two 16-bit numbers of a pair as binary32.
template <int ACT>
__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b)
{
    if constexpr (ACT == Q4_F16) {
        a = h2f(w & 0xffffu);
        b = h2f(w >> 16);
    } else {
        a = std::bit_cast<float>(w << 16);
        b = std::bit_cast<float>(w & 0xffff0000u);
    }
}

// The first 8 bits of a binary32 value (a bfloat16 number).
__device__ __forceinline__ float first8(float v)
{
    return std::bit_cast<float>(std::bit_cast<uint32_t>(v) & 0xffff0000u);
}
// What they leave of a number (nothing of an infinite one).
__device__ __forceinline__ float rest8(float v)
{
    return __builtin_fabsf(v) < __builtin_inff() ? v - first8(v) : 0.0f;
}
// Two values' first 8 bits as a pair of bfloat16 numbers.
__device__ __forceinline__ uint32_t pack_first8(float a, float b)
{
    return __builtin_amdgcn_perm(std::bit_cast<uint32_t>(b), std::bit_cast<uint32_t>(a), 0x07060302u);
}
// A pair of binary32 values as three pairs of bfloat16 numbers.
struct Split3 {
    uint32_t p[3];
};
// One value's parts, in their upper halves.  Their sum is the value exactly, and
// each has its sign and is zero only if it is (a part that would leave nothing
// is the number below, by 8 bits): beside an infinite operand every product is
// infinite of one sign.  An infinite (or NaN) value is in the last part, which
// alone meets nothing but operands' first parts, beside ones.
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3])
{
    const bool number = __builtin_fabsf(v) < __builtin_inff();
    const float n = number ? v : __builtin_copysignf(1.0f, v);
    const uint32_t below = n != 0.0f ? 1u : 0u;
    p[0] = (std::bit_cast<uint32_t>(n) - below) & 0xffff0000u;
    const float r = n - std::bit_cast<float>(p[0]);
    p[1] = (std::bit_cast<uint32_t>(r) - below) & 0xffff0000u;
    p[2] = std::bit_cast<uint32_t>(number ? r - std::bit_cast<float>(p[1]) : v);
}
__device__ __forceinline__ Split3 split3(float a, float b)
{
    uint32_t pa[3], pb[3];
    split3(a, pa);
    split3(b, pb);
    Split3 s;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        s.p[i] = __builtin_amdgcn_perm(pb[i], pa[i], 0x07060302u);
    return s;
}

// 8 values of h (or u) as operands.
struct Low8 {
    u32x4 p[3];
};
__device__ __forceinline__ Low8 three_parts(const float (&v)[8])
{
    Low8 l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Split3 s = split3(v[2 * i], v[2 * i + 1]);
        l.p[0][i] = s.p[0];
        l.p[1][i] = s.p[1];
        l.p[2][i] = s.p[2];
    }
    return l;
}
// 8 activations (or adapter weights) as operands: bfloat16 ones are their own
// first part and have no second.
struct Exact8 {
    u32x4 hi, lo;
};
template <int ACT>
__device__ __forceinline__ Exact8 exact_parts(const u32x4 &w)
{
    Exact8 e{w, u32x4{0, 0, 0, 0}};
    if constexpr (ACT == Q4_F16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack2<ACT>(w[i], a, b);
            e.hi[i] = pack_first8(a, b);
            e.lo[i] = pack_first8(rest8(a), rest8(b));
        }
    }
    return e;
}

// Products of such operands, small ones first.
template <int ACT>
__device__ __forceinline__ f32x4 mfma_exact_low(const Exact8 &x, const Low8 &l, f32x4 c)
{
    c = mfma<Q4_BF16>(x.hi, l.p[2], c);
    if constexpr (ACT == Q4_F16)
        c = mfma<Q4_BF16>(x.lo, l.p[1], c);
    c = mfma<Q4_BF16>(x.hi, l.p[1], c);
    if constexpr (ACT == Q4_F16)
        c = mfma<Q4_BF16>(x.lo, l.p[0], c);
    return mfma<Q4_BF16>(x.hi, l.p[0], c);
}
template <int ACT>
__device__ __forceinline__ f32x4 mfma_low_exact(const Low8 &l, const Exact8 &x, f32x4 c)
{
    c = mfma<Q4_BF16>(l.p[2], x.hi, c);
    if constexpr (ACT == Q4_F16)
        c = mfma<Q4_BF16>(l.p[1], x.lo, c);
    c = mfma<Q4_BF16>(l.p[1], x.hi, c);
    if constexpr (ACT == Q4_F16)
        c = mfma<Q4_BF16>(l.p[0], x.lo, c);
    return mfma<Q4_BF16>(l.p[0], x.hi, c);
}

// The sum of h's partial sums at row m, r0 .. r0 + 7 (in order of the parts),
// or zeros where not `there`; the parts by a view of them all.  All loads are
// issued before the first sum.
__device__ __forceinline__ void sum_parts(__amdgpu_buffer_rsrc_t view, const LowRank &l, int m, int r0, bool there,
                                          float (&v)[8])
{
    u32x4 a[kMostParts], b[kMostParts];
    const uint32_t at = 4u * (uint32_t)(m * l.rank + r0), none = there ? 0u : 0x80000000u;
#pragma unroll
    for (int i = 0; i < kMostParts; ++i) {
        const uint32_t off = (at + 4u * (uint32_t)i * (uint32_t)(l.rows * l.rank)) | none | (i < l.parts ? 0u : 0x80000000u);
        a[i] = __builtin_amdgcn_raw_buffer_load_b128(view, (int)off, 0, 0);
        b[i] = __builtin_amdgcn_raw_buffer_load_b128(view, (int)off, 16, 0);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = std::bit_cast<float>(a[0][e]);
        v[4 + e] = std::bit_cast<float>(b[0][e]);
    }
#pragma unroll
    for (int i = 1; i < kMostParts; ++i) {
        if (i < l.parts) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] += std::bit_cast<float>(a[i][e]);
                v[4 + e] += std::bit_cast<float>(b[i][e]);
            }
        }
    }
}

// The adapters of up to 64 C rows, one after another: which one, and in a mask
// of 64 rows each who has it.  (Every row has at most one, and each adapter's
// weights meet its own rows alone: what another adapter holds, NaN as well,
// never reaches a row.)
template <int C>
struct AdapterSet {
    int id[C];         // the lane's rows 64 c + lane
    uint64_t left[C];  // rows not yet taken

    __device__ __forceinline__ void init(const int32_t *__restrict__ ids, int adapters, int64_t m0, int rows)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int m = 64 * c + lane;
            id[c] = m < rows ? adapter_of(ids, adapters, m0 + m) : -1;
            left[c] = __ballot(id[c] >= 0);
        }
    }
    __device__ __forceinline__ bool next(int &a, uint64_t (&mask)[C])
    {
        a = -1;
#pragma unroll
        for (int c = C - 1; c >= 0; --c)
            if (left[c])
                a = __builtin_amdgcn_readlane(id[c], (int)__builtin_ctzll(left[c]));
        if (a < 0)
            return false;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            mask[c] = __ballot(id[c] == a);
            left[c] &= ~mask[c];
        }
        return true;
    }
};

}  // namespace q4
