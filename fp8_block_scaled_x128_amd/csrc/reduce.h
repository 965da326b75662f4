// Lane reductions shared by the norm and router kernels (64-wide waves).
// Inside the 16-lane rows the steps are DPP moves, which cost a VALU
// instruction each or none; between the rows they are row swaps or reads into
// scalar registers, so nothing goes through the LDS crossbar.  Sums have a
// fixed order: results do not depend on scheduling.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {

// Source lane of each DPP step inside a 16-lane row: xor 1, xor 2 (quad
// permutes), 7 - i within 8 lanes, 15 - i within 16.  After each step the
// lanes it has joined hold the same value, so the four make an all-reduce.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_mov(uint32_t v) {
    // every source lane exists, so the bound control never matters; with it
    // set the compiler folds the move into the operation that follows
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp_movf(float v) {
    return __uint_as_float(dpp_mov<CTRL>(__float_as_uint(v)));
}

__device__ __forceinline__ float row16_sum(float v) {
    v += dpp_movf<kDppXor1>(v);
    v += dpp_movf<kDppXor2>(v);
    v += dpp_movf<kDppHalfMirror>(v);
    v += dpp_movf<kDppMirror>(v);
    return v;
}
__device__ __forceinline__ float row16_max(float v) {
    v = fmaxf(v, dpp_movf<kDppXor1>(v));
    v = fmaxf(v, dpp_movf<kDppXor2>(v));
    v = fmaxf(v, dpp_movf<kDppHalfMirror>(v));
    v = fmaxf(v, dpp_movf<kDppMirror>(v));
    return v;
}
__device__ __forceinline__ uint32_t row16_umax(uint32_t v) {
    v = max(v, dpp_mov<kDppXor1>(v));
    v = max(v, dpp_mov<kDppXor2>(v));
    v = max(v, dpp_mov<kDppHalfMirror>(v));
    v = max(v, dpp_mov<kDppMirror>(v));
    return v;
}
__device__ __forceinline__ uint32_t row16_umin(uint32_t v) {
    v = min(v, dpp_mov<kDppXor1>(v));
    v = min(v, dpp_mov<kDppXor2>(v));
    v = min(v, dpp_mov<kDppHalfMirror>(v));
    v = min(v, dpp_mov<kDppMirror>(v));
    return v;
}

// v + v of the lane 32 lanes away.
__device__ __forceinline__ float halves_sum(float v) {
    const uint32_t b = __float_as_uint(v);
    const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// v + v of the lane 16, then 32 lanes away.  The swaps exchange the odd rows
// (of 16 or 32 lanes) of their first operand with the even rows of the second;
// given v twice they return the even rows' and the odd rows' values in every
// row.
__device__ __forceinline__ float rows_sum(float v) {
    const uint32_t a = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    return halves_sum(__uint_as_float(p[0]) + __uint_as_float(p[1]));
}

// Sums over the lanes with the same index modulo n (a power of two, uniform).
template <int K>
__device__ __forceinline__ void lanes_sum_mod(uint32_t (&v)[K], int n) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
        if (n <= 8) v[i] += dpp_mov<0x128>(v[i]);        // rotate the 16-lane rows by 8, 4, 2, 1
        if (n <= 4) v[i] += dpp_mov<0x124>(v[i]);
        if (n <= 2) v[i] += dpp_mov<0x122>(v[i]);
        if (n <= 1) v[i] += dpp_mov<0x121>(v[i]);
        if (n <= 16) {
            const auto p = __builtin_amdgcn_permlane16_swap(v[i], v[i], false, false);
            v[i] = p[0] + p[1];
        }
        if (n <= 32) {
            const auto p = __builtin_amdgcn_permlane32_swap(v[i], v[i], false, false);
            v[i] = p[0] + p[1];
        }
    }
}

// Inclusive prefix sum over the wave: shifts inside the 16-lane rows, then the
// last lane of a row to the rows behind it.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int wave_scan(int v) {
    v = dpp_add<0x111, 0xf>(v);                          // row_shr 1, 2, 4, 8
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);                          // lane 15 of rows 0, 2 to rows 1, 3
    return dpp_add<0x143, 0xc>(v);                       // lane 31 to rows 2, 3
}

// All-reduce over LANES lanes (16: a DPP row; 32: two of them, sums only; 64:
// the wave, whose rows meet in scalar registers, so the result is uniform).
// Every lane of the wave must be active.
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    v = row16_sum(v);
    if (LANES == 32) {
        const uint32_t a = __float_as_uint(v);
        const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if (LANES == 64) {
        const uint32_t u = __float_as_uint(v);
        v = (__uint_as_float(lane_value(u, 0)) + __uint_as_float(lane_value(u, 16))) +
            (__uint_as_float(lane_value(u, 32)) + __uint_as_float(lane_value(u, 48)));
    }
    return v;
}
// Sum of a wave's 64 integers.
__device__ __forceinline__ uint32_t lanes_usum(uint32_t v) {
    v += dpp_mov<kDppXor1>(v);
    v += dpp_mov<kDppXor2>(v);
    v += dpp_mov<kDppHalfMirror>(v);
    v += dpp_mov<kDppMirror>(v);
    return lane_value(v, 0) + lane_value(v, 16) + lane_value(v, 32) + lane_value(v, 48);
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_umax(uint32_t v) {
    v = row16_umax(v);
    if (LANES == 64) v = max(max(lane_value(v, 0), lane_value(v, 16)), max(lane_value(v, 32), lane_value(v, 48)));
    return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_umin(uint32_t v) {
    v = row16_umin(v);
    if (LANES == 64) v = min(min(lane_value(v, 0), lane_value(v, 16)), min(lane_value(v, 32), lane_value(v, 48)));
    return v;
}

}  // namespace fp8bs
