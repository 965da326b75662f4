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

// What a code needs of its scale.  `half` is never reached by a remainder where
// y = 1 / S serves; 0 sends every nonzero value to i8_code_slow.
struct I8Scale {
    float s, y, half;
};
__device__ __forceinline__ I8Scale i8_scale(float s) {
    if (s == 0.0f) return {0.0f, 0.0f, 1.0f};       // only zeros have this scale
    const bool fast = s >= kI8MinScale && s < INFINITY;
    return {s, fast ? 1.0f / s : 0.0f, fast ? 0.5f * s : 0.0f};
}

// The code of one value by the definition: for scales without a normal
// reciprocal in 64 bits; 0 under an infinite or NaN scale (a row that holds an
// infinity or a NaN), so that the products with it are NaN.
__device__ __forceinline__ uint32_t i8_code_slow(float v, const I8Scale& c) {
    if (!(c.s < INFINITY)) return 0u;
    if (c.s < kI8MinScale) return c.s > 0.0f ? (uint32_t)(int)rint((double)v / (double)c.s) & 0xffu : 0u;
    float q = __builtin_fmaf(v, c.y, kI8Round) - kI8Round;
    const float r = __builtin_fmaf(-q, c.s, v);
    if (fabsf(r) > c.half || (fabsf(r) == c.half && ((int)q & 1))) q += __builtin_copysignf(1.0f, r);
    return (uint32_t)(int)q & 0xffu;
}

// The codes of v[0..8) as two words, each value with its own scale (sc[i * STEP]:
// STEP 0 for one scale).  v y is within 127 * 2^-23 of v / S, so the rounded
// product is the code or its neighbour, and the remainder v - q S tells which:
// v is a bf16 value (8 bits) and |q| <= 127, so the remainder is a multiple of
// S's last place below 2^24 of them, hence exact in the FMA.  Only where it
// reaches S / 2 (about one value in 10^5, and exact ties) can the code be
// another.  |v / S| is at most 127 (1 + 2^-9) for subnormal S and 127 (1 + 2^-23)
// else: codes stay within +-127.
template <int STEP>
__device__ __forceinline__ uint2 i8_codes8(const float v[8], const I8Scale* sc) {
    float m[8];
    bool slow = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const I8Scale& c = sc[i * STEP];
        m[i] = __builtin_fmaf(v[i], c.y, kI8Round);
        const float r = __builtin_fmaf(kI8Round - m[i], c.s, v[i]);
        slow |= !(fabsf(r) < c.half);
    }
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(m[i]);
    if (__builtin_expect(slow, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = i8_code_slow(v[i], sc[i * STEP]);
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
