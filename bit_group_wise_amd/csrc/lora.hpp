// lora.hpp -- shared by the kernels of low-rank adapters beside a 4-bit
// weight (q4_lora_*).
//
// An adapter adds s (x A^T) B^T to a row's product.  The rows' h = s x A^T
// (and for gradients u = s dy B) are formed first, summed in binary32, and left
// in the workspace; the product's own kernel then adds h B^T (or u A) to its
// binary32 accumulators, so the sum is rounded once and y is written once.
//
// Operands: the matrix cores take 16 bits, so h and u enter as two bfloat16
// numbers, the value's rounding and the rounding of what that left: 16 bits
// and binary32's range (a relative 2^-17, 1/64 of the half step of an fp16
// output, and nothing lost of a gradient below fp16's range).  What they meet
// is bfloat16 as it is, or for fp16 activations also two bfloat16 numbers (11
// bits = 8 + 3: exact); the product of the two second parts, a relative 2^-18,
// is left out.
#pragma once

#include "plan.hpp"
#include "q4_common.hpp"
#include "q4_mfma.hpp"

namespace q4 {

// h[m][r] (or u) and what they go through.  For few rows h is left as binary32
// partial sums, part[i * rows * rank + m * rank + r] for i < parts; else as its
// operands' two parts, two[m * rank + r] and two[(rows + m) * rank + r].
struct LowRank {
    const float *part;
    int parts;
    const uint16_t *two;
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

// 8 binary32 values as bfloat16 operands: their roundings, and the roundings
// of the rest.
struct Parts8 {
    u32x4 hi, lo;
};
__device__ __forceinline__ Parts8 two_parts(const float (&v)[8])
{
    Parts8 p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = pack_bf2(v[2 * i], v[2 * i + 1]);
        p.hi[i] = h;
        p.lo[i] = pack_bf2(v[2 * i] - std::bit_cast<float>(h << 16),
                           v[2 * i + 1] - std::bit_cast<float>(h & 0xffff0000u));
    }
    return p;
}
// 8 activations (or adapter weights) as such operands: bfloat16 ones are their
// own first part and have no second.
template <int ACT>
__device__ __forceinline__ Parts8 two_parts16(const u32x4 &w)
{
    if constexpr (ACT == Q4_BF16) {
        return Parts8{w, u32x4{0, 0, 0, 0}};
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            unpack2<ACT>(w[i], v[2 * i], v[2 * i + 1]);
        return two_parts(v);
    }
}

// Products of such operands: `exact` has a second part for fp16 alone.
template <int ACT>
__device__ __forceinline__ f32x4 mfma_parts_a(const Parts8 &exact, const Parts8 &b, f32x4 c)
{
    c = mfma<Q4_BF16>(exact.hi, b.lo, c);
    if constexpr (ACT == Q4_F16)
        c = mfma<Q4_BF16>(exact.lo, b.hi, c);
    return mfma<Q4_BF16>(exact.hi, b.hi, c);
}
template <int ACT>
__device__ __forceinline__ f32x4 mfma_parts_b(const Parts8 &a, const Parts8 &exact, f32x4 c)
{
    c = mfma<Q4_BF16>(a.lo, exact.hi, c);
    if constexpr (ACT == Q4_F16)
        c = mfma<Q4_BF16>(a.hi, exact.lo, c);
    return mfma<Q4_BF16>(a.hi, exact.hi, c);
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
