// kv_mfma.hpp -- 4-bit cache rows as operands of the 16x16x32 fp16 product.
//
// Rows enter the matrix cores as their levels, small exact numbers, and the
// scales (and zero-points) are applied in binary32 outside the product: to the
// scores of a group for keys, to the softmax weights for values.  So no value
// is rounded on the way in, and unpacking costs five to seven instructions
// per eight codes.
//
// INT4 keys: OR-ing a nibble into 0x6400 makes the fp16 number 1024 + c (bits
// 0-3) or 1024 + 16 c (bits 4-7); a packed add takes 1024 and the zero-point
// off again, exactly.  INT4 values do the same, a pair of tokens to a
// word.  (A nibble left in place is an fp16 subnormal, c 2^-24 or c 2^-20, for
// one mask a pair and no add.  But the matrix cores align subnormals' products
// by the exponent field and lose their low bits beside larger terms: scores of
// fp16 queries were off by up to 1e-4, and the output over 131071 tokens was
// 4.2e-4 from binary64 where rounding the weights and the output gives 2.9e-4.)
// NF4: the
// table's three-decimal entries times 1000 are integers of at most 10 bits,
// exact in fp16; a 256-entry LDS table gives the two levels of a byte.  FP4:
// E2M1 elements, converted by v_cvt_scalef32_pk_f16_fp4.
#pragma once

#include "kv_common.hpp"
#include "q4_mfma.hpp"

namespace q4 {

// What a level in the product's units is to be multiplied by.  INT4's odd
// nibbles count sixteenfold (values; for keys the queries make up for it).
template <int FMT>
constexpr float key_unit()
{
    return FMT == Q4_NF4 ? 1.0f / 1000.0f : FMT == Q4_FP4 ? 1.0f / 6.0f : 1.0f;
}
template <int FMT>
constexpr float value_unit()
{
    return FMT == Q4_NF4 ? 1.0f / 1000.0f : FMT == Q4_FP4 ? 1.0f / 6.0f : 1.0f;
}
template <int FMT>
constexpr bool kv_int() { return FMT == Q4_INT4_SYM || FMT == Q4_INT4_ASYM; }

// NF4's levels times 1000 as fp16, two of a byte to a dword.
__device__ __forceinline__ uint32_t nf4_pair(int byte)
{
    const float a = rintf(kNF4[byte & 15] * 1000.0f), b = rintf(kNF4[byte >> 4] * 1000.0f);
    return pack_h2(a, b);
}

// Two binary32 numbers as an fp16 pair, each rounded to nearest even
// (v_cvt_pk_f16_f32).
__device__ __forceinline__ uint32_t pair_h2(float a, float b)
{
    const f16x2 v = {(_Float16)a, (_Float16)b};
    return std::bit_cast<uint32_t>(v);
}

// Eight codes of one row (a dword) as the row operand of a product over d.
// The order of the eight within the operand is that of q_pair_order: INT4
// (0,4)(1,5)(2,6)(3,7) with the second and fourth pair sixteenfold, otherwise
// (0,1)(2,3)(4,5)(6,7).
constexpr uint32_t kNib0 = 0x000f000fu, kNib1 = 0x00f000f0u;
template <int SEL>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t w)
{
    return std::bit_cast<uint32_t>(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL));
}
// What takes the offset off: -(1024 + z) and -(1024 + 16 z), twice each.
struct KeyZero {
    uint32_t even, odd;
};
__device__ __forceinline__ KeyZero zero_of_pair(uint32_t z)  // a zero-point 0..15 in each half
{
    return KeyZero{0xe400e400u + z, 0xe400e400u + 16 * z};
}
__device__ __forceinline__ KeyZero key_zero(uint32_t z)  // z in 0..15
{
    return KeyZero{0xe400e400u + z * 0x00010001u, 0xe400e400u + z * 0x00100010u};
}
__device__ __forceinline__ uint32_t add_h2(uint32_t a, uint32_t b)
{
    return std::bit_cast<uint32_t>(std::bit_cast<f16x2>(a) + std::bit_cast<f16x2>(b));
}
template <int FMT>
__device__ __forceinline__ u32x4 key_operand(uint32_t w, const KeyZero &z, const uint32_t *pairs)
{
    if constexpr (kv_int<FMT>()) {
        // (masks in vector registers, the offset in a scalar one: mask and OR
        // are one v_and_or_b32)
        const uint32_t m0 = opaque_word(kNib0), m1 = opaque_word(kNib1);
        const uint32_t one = opaque_sword(0x64006400u), h = w >> 8;
        return u32x4{add_h2((w & m0) | one, z.even), add_h2((w & m1) | one, z.odd),
                     add_h2((h & m0) | one, z.even), add_h2((h & m1) | one, z.odd)};
    } else if constexpr (FMT == Q4_NF4) {
        return u32x4{pairs[w & 255], pairs[(w >> 8) & 255], pairs[(w >> 16) & 255], pairs[w >> 24]};
    } else {
        return u32x4{fp4_pair<0>(w), fp4_pair<1>(w), fp4_pair<2>(w), fp4_pair<3>(w)};
    }
}

// Which dword of a group lane i reads of a value row, and what it takes of it:
// lane i of 16 supplies values d = (g / 16) i + n of the group for the products
// n = 0 .. g/16 - 1, that is a dword (g = 128), a half (64) or a byte (32).
template <int GS>
__device__ __forceinline__ int value_dword(int i) { return i / (128 / GS); }
// The lane's selector for INT4 (v_perm_b32), or its shift (NF4, FP4).
template <int FMT, int GS>
__device__ __forceinline__ uint32_t value_select(int i)
{
    if constexpr (kv_int<FMT>()) {
        if constexpr (GS == 128)
            return 0x05040100u;  // low halves of two tokens' dwords
        else if constexpr (GS == 64)
            return i & 1 ? 0x07060302u : 0x05040100u;
        else
            return (uint32_t)(i & 3) * 0x00010001u + 0x0c040c00u;  // one byte each, zeros above
    } else {
        return GS == 128 ? 0u : GS == 64 ? 16u * (i & 1) : 8u * (i & 3);
    }
}
// Pairs (token a, token b) of the lane's g/16 values from the two tokens'
// dwords; o[n] is the pair of product n (INT4: odd n sixteenfold).  z: the two
// tokens' zero-points.
template <int FMT, int GS>
__device__ __forceinline__ void value_pairs(uint32_t a, uint32_t b, uint32_t sel, const KeyZero &z,
                                            const uint32_t *pairs, uint32_t (&o)[GS / 16])
{
    if constexpr (kv_int<FMT>()) {
        const uint32_t m0 = opaque_word(kNib0), m1 = opaque_word(kNib1);
        const uint32_t one = opaque_sword(0x64006400u);
        const uint32_t x = __builtin_amdgcn_perm(b, a, sel);
        o[0] = add_h2((x & m0) | one, z.even);
        o[1] = add_h2((x & m1) | one, z.odd);
        if constexpr (GS >= 64) {
            const uint32_t y = x >> 8;
            o[2] = add_h2((y & m0) | one, z.even);
            o[3] = add_h2((y & m1) | one, z.odd);
        }
        if constexpr (GS == 128) {
            const uint32_t u = __builtin_amdgcn_perm(b, a, 0x07060302u), v = u >> 8;
            o[4] = add_h2((u & m0) | one, z.even);
            o[5] = add_h2((u & m1) | one, z.odd);
            o[6] = add_h2((v & m0) | one, z.even);
            o[7] = add_h2((v & m1) | one, z.odd);
        }
    } else {
        if constexpr (GS != 128) {
            a >>= sel;
            b >>= sel;
        }
#pragma unroll
        for (int j = 0; j < GS / 32; ++j) {
            uint32_t la, lb;
            if constexpr (FMT == Q4_NF4) {
                la = pairs[(a >> (8 * j)) & 255];
                lb = pairs[(b >> (8 * j)) & 255];
            } else {
                la = j == 0 ? fp4_pair<0>(a) : j == 1 ? fp4_pair<1>(a) : j == 2 ? fp4_pair<2>(a) : fp4_pair<3>(a);
                lb = j == 0 ? fp4_pair<0>(b) : j == 1 ? fp4_pair<1>(b) : j == 2 ? fp4_pair<2>(b) : fp4_pair<3>(b);
            }
            o[2 * j] = __builtin_amdgcn_perm(lb, la, 0x05040100u);
            o[2 * j + 1] = __builtin_amdgcn_perm(lb, la, 0x07060302u);
        }
    }
}

// Eight query values (16-bit, d ascending, in four dwords) times f, in the
// order of key_operand.
template <int FMT>
__device__ __forceinline__ u32x4 query_operand(const u32x4 &raw, int act, float f)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = (act == Q4_F16 ? h2f(raw[i] & 0xffffu) : bf2f(raw[i] & 0xffffu)) * f;
        x[2 * i + 1] = (act == Q4_F16 ? h2f(raw[i] >> 16) : bf2f(raw[i] >> 16)) * f;
    }
    if constexpr (kv_int<FMT>())
        return u32x4{pair_h2(x[0], x[4]), pair_h2(x[1] * 0.0625f, x[5] * 0.0625f), pair_h2(x[2], x[6]),
                     pair_h2(x[3] * 0.0625f, x[7] * 0.0625f)};
    else
        return u32x4{pair_h2(x[0], x[1]), pair_h2(x[2], x[3]), pair_h2(x[4], x[5]), pair_h2(x[6], x[7])};
}
__device__ __forceinline__ float query_max(const u32x4 &raw, int act)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = fmaxf(m, act == Q4_F16 ? fmaxf(fabsf(h2f(raw[i] & 0xffffu)), fabsf(h2f(raw[i] >> 16)))
                                   : fmaxf(fabsf(bf2f(raw[i] & 0xffffu)), fabsf(bf2f(raw[i] >> 16))));
    return m;
}

}  // namespace q4
