// Codes in 8-bit integers: S = fp32(max|v| / 127) of a row or column and q =
// the integer nearest to v / S, ties to even.
#pragma once
#include "device_common.h"

namespace fp8bs {

constexpr float kI8Max = 127.0f;
// 1.5 * 2^23: adding it rounds to an integer, ties to even, and leaves that
// integer's two's complement in the sum's low bits.
constexpr float kI8Round = 12582912.0f;
// From this scale on 1 / S and the remainders below are normal numbers.
constexpr float kI8MinScale = 0x1p-100f;

// What a code needs of its scale: y = 1 / S and S / 2, or y = 0 where 1 / S does not
// serve (S = 0, where all values are 0; S tiny, infinite or NaN).
struct I8Scale {
    float s, y, half;
};
__device__ __forceinline__ I8Scale i8_scale(float s) {
    const bool fast = s >= kI8MinScale && s < INFINITY;
    return {s, fast ? 1.0f / s : 0.0f, fast ? 0.5f * s : INFINITY};
}
__device__ __forceinline__ bool i8_special(const I8Scale& c) { return c.y == 0.0f && c.s != 0.0f; }

// The code of one value under such a scale: in 64 bits, or 0 under an infinite or NaN
// scale (a row that holds an infinity or a NaN), so that the products with it are NaN.
__device__ __forceinline__ uint32_t i8_code_special(float v, float s) {
    return s < kI8MinScale ? (uint32_t)(int)rint((double)v / (double)s) & 0xffu : 0u;
}

// The codes of v[0..8) as two words, each value with its own scale (sc[i * STEP]:
// STEP 0 for one scale).  v y is within 127 * 2^-23 of v / S, so the rounded product
// is the code or its neighbour, and the remainder v - q S tells which: v is a bf16
// value (8 bits) and |q| <= 127, so the remainder is a multiple of S's last place below
// 2^24 of them, hence exact in the FMA, and beyond S / 2 where the neighbour is nearer.
// Such values are common (v / S is within 2^-24 of a half where max|v| has a short odd
// part), so nothing branches on them.  A remainder of exactly S / 2 needs (2 q + 1) S
// to be a bf16 value: S has to be a power of two (127 S = max|v|), whose product and
// rounding are exact, so the even code is there already.  |v / S| is at most
// 127 (1 + 2^-9) for subnormal S and 127 (1 + 2^-23) else: codes stay within +-127.
template <int STEP>
__device__ __forceinline__ uint2 i8_codes8(const float v[8], const I8Scale* sc) {
    uint32_t b[8];
    bool special = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const I8Scale& c = sc[i * STEP];
        const float m = __builtin_fmaf(v[i], c.y, kI8Round);
        const float r = __builtin_fmaf(kI8Round - m, c.s, v[i]);
        b[i] = __float_as_uint(m + (fabsf(r) > c.half ? __builtin_copysignf(1.0f, r) : 0.0f));
        if (STEP || i == 0) special |= i8_special(c);
    }
    if (__builtin_expect(special, 0)) {
        // one copy of the rare code, whatever the caller unrolls
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            float x = v[0];
            I8Scale c = sc[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                x = k == i ? v[i] : x;
                if (STEP && k == i) c = sc[i * STEP];
            }
            const uint32_t q = i8_code_special(x, c.s);
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = k == i && i8_special(c) ? q : b[i];
        }
    }
    // byte 0 of each word: v_perm_b32 takes bytes 0-3 from its second operand,
    // 4-7 from its first, and 0 for selector 0x0c
    return make_uint2(__builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u) | __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu),
                      __builtin_amdgcn_perm(b[5], b[4], 0x0c0c0400u) | __builtin_amdgcn_perm(b[7], b[6], 0x04000c0cu));
}

// max of the two halves' magnitudes over four words of bf16 pairs, as 16-bit
// patterns (infinities above every finite value, NaN above those).
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 absmax_bits(u16x2 m, uint4 w) {
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w.x & 0x7fff7fffu));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w.y & 0x7fff7fffu));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w.z & 0x7fff7fffu));
    return __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w.w & 0x7fff7fffu));
}
// The scale of a maximum given as a bf16 magnitude pattern.
__device__ __forceinline__ float i8_scale_of(uint32_t bits) { return __uint_as_float(bits << 16) / kI8Max; }

}  // namespace fp8bs
