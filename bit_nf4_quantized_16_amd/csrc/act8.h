// 8-bit activation checkpoints (gfx950): the codec shared by the kernels that
// write and read them.
//
// Blocks of 32 consecutive values of a row share one power-of-two scale 2^k,
// held as the byte k + 127 (E8M0); the values are OCP FP8 E4M3FN codes. With
// a = max |x| over the block's finite values, k is the least integer with
// a 2^-k <= 448 (E4M3's largest value), at least -124. A power of two makes
// x 2^-k exact, so the code is the correctly rounded one (nearest, ties to
// even) whatever the arithmetic, and a code times 2^k has four significant
// bits and a last place of at least 2^-9 2^-124 = 2^-133, the smallest bf16
// value: restoring to bf16 is exact (2^128, where magnitudes from
// 1.9375 2^127 on round to, becomes infinity). A NaN or infinite x becomes NaN (E4M3FN
// has no infinity) and leaves its block's scale to the finite values.
//
// The conversions are CDNA4's scaled ones (v_cvt_scalef32_pk_fp8_bf16 and
// v_cvt_scalef32_pk_bf16_fp8, two values an instruction at the rate of a
// multiply-add); their rounding was checked against the definition for every
// bf16 value and every code at scales from 2^-124 to 2^120.
#pragma once

#include "common.h"

namespace qlnf4 {

constexpr int kAct8Block = QL_ACT8_BLOCK;
static_assert(kAct8Block == 32, "a block is four lanes of eight values");

typedef __bf16 bf16x2_act __attribute__((ext_vector_type(2)));
typedef short i16x2_act __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2_act __attribute__((ext_vector_type(2)));

// Largest of the eight magnitudes in v as bf16 bits (sign cleared); with
// finite_only a NaN or infinity counts as zero.
__device__ __forceinline__ uint32_t act8_max8(uint4 v, bool finite_only) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    u16x2_act m = {0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t a = w[q] & 0x7FFF7FFFu;
        if (finite_only) {
            // a half of 0x7F80 or more carries into its sign bit, which then fills the half
            const u16x2_act c = __builtin_bit_cast(u16x2_act, a) + u16x2_act{0x80, 0x80};
            a &= ~__builtin_bit_cast(uint32_t, __builtin_bit_cast(i16x2_act, c) >> i16x2_act{15, 15});
        }
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_act, a));
    }
    return umax_(m[0], m[1]);
}

// Scale byte of the block whose eight-value pieces sit in four consecutive
// lanes (an aligned quad), piece v in this lane: every lane gets it.
__device__ __forceinline__ uint32_t act8_scale_byte(uint4 v) {
    uint32_t a = act8_max8(v, false);
    if (__builtin_expect(__any(a >= 0x7F80u), 0)) a = act8_max8(v, true);
    a = umax_(a, dpp_u<0xB1>(a));  // quad_perm [1,0,3,2]
    a = umax_(a, dpp_u<0x4E>(a));  // quad_perm [2,3,0,1]
    // bf16 exponent field, one more when the significand is over 1.75 (0x60);
    // 448 = 1.75 2^8; the floor 11 - 8 = 3 is k = -124
    return umax_((a + 0x1Fu) >> 7, 11u) - 8u;
}

// Eight bf16 values -> eight codes, value 0 in the lowest byte.
__device__ __forceinline__ uint2 act8_encode8(uint4 v, uint32_t scale_byte) {
    const float s = __uint_as_float(scale_byte << 23);
    i16x2_act lo = {0, 0}, hi = {0, 0};
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(bf16x2_act, v.x), s, false);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(bf16x2_act, v.y), s, true);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2_act, v.z), s, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2_act, v.w), s, true);
    return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

// Eight codes -> eight bf16 values (exact).
__device__ __forceinline__ uint4 act8_decode8(uint2 c, uint32_t scale_byte) {
    const float s = __uint_as_float(scale_byte << 23);
    uint4 r;
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, true));
    return r;
}

}  // namespace qlnf4
