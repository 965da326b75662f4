// What the forward and backward block-norm kernels share: element access, the
// row layout over lanes, and a row's reduction and factor.
//
// Layout: a row belongs to `wpr` waves of a workgroup; lane l of them holds
// the 8-column chunks l, l + 64 wpr, ..., NV of them.  All but the last chunk
// of a lane are inside the row, so only the last is guarded.
#pragma once
#include "device_common.h"
#include "internal.h"
#include "reduce.h"

namespace fp8bs {

// Eight elements as loaded.  They stay packed until they are used, so that a
// row's loads are all in flight before the first conversion waits for one.
template <bool F32>
struct Raw8 {
    uint4 r[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        if (F32) {
            const float* f = static_cast<const float*>(p) + i;
            r[0] = load_nt16(f);
            r[F32 ? 1 : 0] = load_nt16(f + 4);
        } else {
            r[0] = load_nt16(static_cast<const uint16_t*>(p) + i);
        }
    }
    __device__ __forceinline__ void load_shared(const void* p, int64_t i) {     // bf16, cached policy
        r[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
        r[0] = make_uint4(0, 0, 0, 0);
        r[F32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float v[8]) const {
        if (F32) {
            const uint4 a = r[0], b = r[F32 ? 1 : 0];
            v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
            v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
            v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
            v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
        } else {
            unpack8(r[0], v);
        }
    }
};

// Norm weights and gates: rows share them, so they keep the cached policy.
__device__ __forceinline__ void load8_shared(const void* p, int64_t i, bool f32, float v[8]) {
    if (f32) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = f[0], b = f[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), v);
    }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float v[8]) {
    if (F32) {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        f[0] = make_float4(v[0], v[1], v[2], v[3]);
        f[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
    }
}

constexpr int kMaxRowWaves = 8;      // waves that share a row
constexpr int kMaxNv = 8;            // chunks per lane: 8 * 8 * 64 chunks of 8 = 32768 columns
// Chunks that are inside the row for every lane: the host launches NV <= 4
// only for rows that need the last chunk, and NV 8 for 5 to 8.
template <int NV>
constexpr int kSure = NV <= 4 ? NV - 1 : 4;

// Sum of squares of eight values, as a tree: three roundings deep.
__device__ __forceinline__ float sumsq8(const float v[8]) {
    const float a = __builtin_fmaf(v[0], v[0], v[1] * v[1]), b = __builtin_fmaf(v[2], v[2], v[3] * v[3]);
    const float c = __builtin_fmaf(v[4], v[4], v[5] * v[5]), d = __builtin_fmaf(v[6], v[6], v[7] * v[7]);
    return (a + b) + (c + d);
}
__device__ __forceinline__ float dot8(const float u[8], const float v[8]) {
    const float a = __builtin_fmaf(u[0], v[0], u[1] * v[1]), b = __builtin_fmaf(u[2], v[2], u[3] * v[3]);
    const float c = __builtin_fmaf(u[4], v[4], u[5] * v[5]), d = __builtin_fmaf(u[6], v[6], u[7] * v[7]);
    return (a + b) + (c + d);
}

// 1 / sqrt(v) for v > 0: the hardware approximation and one Newton step with
// the rounding error of v r kept (fma), within an ulp of the exact value.
__device__ __forceinline__ float inv_sqrt(float v) {
    const float r = __builtin_amdgcn_rsqf(v);
    const float t = v * r, tl = __builtin_fmaf(v, r, -t);
    const float e = __builtin_fmaf(-tl, r, __builtin_fmaf(-t, r, 1.0f));
    return __builtin_fmaf(0.5f * r, e, r);
}

// Sums of K values over the waves that share a row (one: no barrier).  `buf`
// alternates between two LDS buffers from call to call: a wave can be at most
// one barrier behind, so the buffer it still reads is not the one written.
template <bool MULTI, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int wpr, float (*lds)[kMaxRowWaves][4], int& turn) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = lanes_sum<64>(v[i]);
    if (!MULTI) return;
    float (*buf)[4] = lds[turn & 1];
    turn++;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) buf[threadIdx.x >> 6][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = 0.0f;
    for (int w = 0; w < wpr; ++w) {
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] += buf[w][i];
    }
}

// Waves per row and chunks per lane: `chunks` per lane if eight waves then
// hold the row, else the fewest that do.
inline void row_split(int64_t cols, int chunks, int* wpr, int* nv) {
    const int64_t groups = (cols / 8 + 63) / 64;            // chunks of 64 lanes
    int64_t n = (groups + kMaxRowWaves - 1) / kMaxRowWaves;
    if (n < chunks) n = chunks < groups ? chunks : groups;
    *wpr = (int)((groups + n - 1) / n);
    *nv = (int)((groups + *wpr - 1) / *wpr);
}

}  // namespace fp8bs
