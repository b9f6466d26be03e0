// q4_code.hpp -- the coding rules' arithmetic, shared by the weight quantizer
// and the key/value cache: correctly rounded quotients by a group's scale,
// nearest levels, packing, and reductions over a group's lanes.
#pragma once

#include "q4_common.hpp"

namespace q4 {

// Correctly rounded a / b given r = RN(1 / b) (Markstein).
__device__ __forceinline__ float div_mk(float a, float b, float r)
{
    float q0 = a * r;
    float e = __builtin_fmaf(-q0, b, a);
    return __builtin_fmaf(e, r, q0);
}

// The scale quotients a / 7 (INT4-sym, a the absmax) and (hi - lo) / 15
// (INT4-asym) with the constant reciprocals RN(1/7) and RN(1/15): three
// instructions instead of a general division.  Equal to the IEEE quotient
// for every operand these can meet (a any non-negative fp16 value; hi - lo
// rounded to binary32 for any non-negative fp16 hi and non-positive fp16 lo),
// checked exhaustively.
constexpr float kInv7 = 1.0f / 7.0f;
constexpr float kInv15 = 1.0f / 15.0f;

// RN(1 / s) for s > 0 an fp16 value (the stored scale, or the absmax): the
// hardware reciprocal (accurate to 1 ulp) and one Newton step,
// r = r0 + r0 * (1 - s * r0) with both steps fused.  The step leaves a
// relative error of order 2^-46, while 1 / s, whose divisor has at most 11
// significant bits, lies at least 2^-35 (relative) away from any rounding
// midpoint, so the result is the correctly rounded reciprocal; checked
// exhaustively for every positive fp16 s and every start within 2 ulps.
__device__ __forceinline__ float rcp_rn(float s)
{
    const float r0 = __builtin_amdgcn_rcpf(s);
    const float e = __builtin_fmaf(-r0, s, 1.0f);
    return __builtin_fmaf(e, r0, r0);
}

// INT4 codes q = clamp(rint(x) + z, 0, 15) for any finite x (here x = w / s).
// For |x| < 2^22, adding 1.5 * 2^23 rounds x to an integer exactly as rint
// does (to nearest, ties to even: the sum's unit is 1) and leaves it in the
// low bits of the sum's bit pattern, kRintBias + rint(x); a larger |x| puts
// the sum beyond the clamp below, on the side the clamp of rint(x) + z takes
// too (and |w / s| <= 23 for finite fp16 inputs anyway).  Clamping the sum to
// [1.5 * 2^23 - z, 1.5 * 2^23 + 15 - z] (v_med3; integers there are exact)
// leaves kRintBias - z + q in the bits, so the instructions per weight are
// one add, one clamp and the packing; the offset kRintBias - z comes off
// once per dword (pack8).
constexpr float kRint = 12582912.0f;         // 1.5 * 2^23
constexpr uint32_t kRintBias = 0x4B400000u;  // its bit pattern
__device__ __forceinline__ uint32_t code_bits(float x, float lo, float hi)
{
    return std::bit_cast<uint32_t>(__builtin_amdgcn_fmed3f(x + kRint, lo, hi));
}
// 8 codes as one dword, low nibble first, from code_bits values c = off + q:
// shifted and added (codes below 16 never carry into the next nibble), then
// the offsets' shifted sum, off * 0x11111111 mod 2^32, taken off.
__device__ __forceinline__ uint32_t pack8(const uint32_t (&c)[8], uint32_t off)
{
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        word += c[i] << (4 * i);
    return word - off * 0x11111111u;
}

template <int LPG>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int d = 1; d < LPG; d <<= 1)
        v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
template <int LPG>
__device__ __forceinline__ float group_min(float v)
{
#pragma unroll
    for (int d = 1; d < LPG; d <<= 1)
        v = fminf(v, __shfl_xor(v, d));
    return v;
}

// NF4 codes of 8 weights of a group with absmax c > 0, as one dword (low
// nibble first).
__device__ __forceinline__ uint32_t nf4_word(const float (&v)[8], float c, const NF4Bucket *lut)
{
    const float r = rcp_rn(c);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = div_mk(v[i], c, r);
        // bucket floor((x + 1) * 16), the product formed as one fma (16 (x + 1)
        // rounds as x + 1 does, scaled exactly); |x| <= 1, so b <= 32; the min
        // only guards inputs that break the finite-input precondition
        const uint32_t b = min((uint32_t)__builtin_fmaf(x, 16.0f, 16.0f), 32u);
        const NF4Bucket e = lut[b];
        const uint32_t code = e.base + (x >= e.thr ? 1u : 0u);
        word |= code << (4 * i);
    }
    return word;
}

// FP4 codes of 8 weights of a group with absmax c > 0: the magnitude index
// j = number of thresholds at or below |x| (seven compares), then the sign
// (code j + 8 for x < 0 and j > 0; the tie of +0 and -0 keeps code 0).
__device__ __forceinline__ uint32_t fp4_word(const float (&v)[8], float c)
{
    const float r = rcp_rn(c);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = div_mk(v[i], c, r);
        const float a = fabsf(x);
        uint32_t j = 0;
#pragma unroll
        for (int t = 0; t < 7; ++t)
            j += a >= kFP4Thr[t] ? 1u : 0u;
        const uint32_t code = (x < 0.0f && j != 0) ? j + 8 : j;
        word |= code << (4 * i);
    }
    return word;
}

}  // namespace q4
