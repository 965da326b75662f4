// What the forward and backward block-norm kernels share: element access, the
// row layout over lanes, and a row's reduction and factor.
//
// Layout: a row belongs to `wpr` waves of a workgroup (kMulti), or to 64, 32 or
// 16 lanes of one wave (rows of at most 512, 256, 128 columns: head norms);
// lane l of them holds the 8-column chunks l, l + (lanes), ..., NV of them.
// All but the last chunk of a lane are inside the row, so only the last is
// guarded.
#pragma once
#include <type_traits>

#include "device_common.h"
#include "internal.h"
#include "reduce.h"

namespace fp8bs {

// Start of a row.  Uniform over the wave: with a 32-bit chunk offset the
// accesses need no 64-bit address per lane.
template <bool F32, typename T>
__device__ __forceinline__ T* row_ptr(T* p, int64_t row, int64_t ld) {
    using C = std::conditional_t<std::is_const<T>::value, const char, char>;
    return reinterpret_cast<T*>(reinterpret_cast<C*>(p) + row * ld * (F32 ? 4 : 2));
}

// Eight elements (chunk c of a row) as loaded.  They stay packed until they are used, so that a
// row's loads are all in flight before the first conversion waits for one.
template <bool F32>
struct Raw8 {
    uint4 r[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* row, uint32_t c) {
        const char* p = static_cast<const char*>(row) + c * (F32 ? 32u : 16u);
        r[0] = load_nt16(p);
        if (F32) r[F32 ? 1 : 0] = load_nt16(p + 16);
    }
    __device__ __forceinline__ void load_shared(const void* row, uint32_t c) {     // bf16, cached policy
        r[0] = *reinterpret_cast<const uint4*>(static_cast<const char*>(row) + c * 16u);
    }
    // Makes the compiler convert again after this point instead of keeping the
    // fp32 values of the last get() (twice the registers of bf16) until then.
    __device__ __forceinline__ void forget() {
        if (!F32) asm volatile("" : "+v"(r[0].x), "+v"(r[0].y), "+v"(r[0].z), "+v"(r[0].w));
    }
    __device__ __forceinline__ void zero() {
        r[0] = make_uint4(0, 0, 0, 0);
        r[F32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void scale(float c) {         // bf16 values by a power of two
        float v[8];
        unpack8(r[0], v);
        r[0] = make_uint4(pack_bf16x2(v[0] * c, v[1] * c), pack_bf16x2(v[2] * c, v[3] * c),
                          pack_bf16x2(v[4] * c, v[5] * c), pack_bf16x2(v[6] * c, v[7] * c));
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

// Norm weights: rows share them, so they keep the cached policy.
__device__ __forceinline__ void load8_shared(const void* row, uint32_t c, bool f32, float v[8]) {
    if (f32) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const char*>(row) + c * 32u);
        const float4 a = f[0], b = f[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const char*>(row) + c * 16u), v);
    }
}
template <bool F32>
__device__ __forceinline__ void store8(void* row, uint32_t c, const float v[8]) {
    char* p = static_cast<char*>(row) + c * (F32 ? 32u : 16u);
    if (F32) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
}

constexpr int kCUs = 256;            // compute units
constexpr int kMulti = 0;            // lanes per row: the workgroup's
constexpr int kMaxRowWaves = 8;      // waves that share a row
// Chunks per lane: at most 4 (8 waves x 64 lanes x 4 chunks of 8 = 16384
// columns).  The host launches NV only for rows that need the last chunk, so
// the others are inside the row for every lane.
template <int NV>
constexpr int kSure = NV - 1;

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

// 1 / sqrt(v) for normal v > 0: the hardware approximation and one Newton step
// with the rounding error of v r kept (fma), within an ulp of the exact value;
// 0 for infinity.
__device__ __forceinline__ float inv_sqrt(float v) {
    const float r = __builtin_amdgcn_rsqf(v);
    const float t = v * r, tl = __builtin_fmaf(v, r, -t);
    const float e = __builtin_fmaf(-tl, r, __builtin_fmaf(-t, r, 1.0f));
    const float n = __builtin_fmaf(0.5f * r, e, r);
    return v <= 3.4028235e38f ? n : r;
}

// Sums of K values over the lanes that share a row.  Over several waves (one:
// no barrier) `buf` alternates between two LDS buffers from call to call: a
// wave can be at most one barrier behind, so the buffer it still reads is not
// the one written.
template <int LPR, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int wpr, float (*lds)[kMaxRowWaves][4], int& turn) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = lanes_sum<LPR == kMulti ? 64 : LPR>(v[i]);
    if (LPR != kMulti) return;
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

// Mean square + eps of K vectors of a row from their sums of squares.  Where a
// mean square is past 2^128 / cols the sum overflows: such a row is summed again
// from its values (`get(k, i, v)`: chunk i of vector k) at kDown each, kDown^2
// being the inverse of the largest number of columns.  All lanes that share the
// row have the same sums; a wave with several rows goes that way together, and
// only the sums that need it are replaced.
constexpr float kDown = 0x1p-7f;
template <int LPR, int NV, int K, typename Get>
__device__ __forceinline__ void row_means(float (&sum)[K], const Get& get, float inv_n, float eps, int wpr,
                                          float (*lds)[kMaxRowWaves][4], int& turn) {
    bool over[K], any = false;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        over[k] = !(sum[k] <= 3.4028235e38f);               // an infinity or a NaN too: the same sum again
        any |= over[k];
        sum[k] = __builtin_fmaf(sum[k], inv_n, eps);
    }
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(any) == 0, 1)) return;
    float s[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        s[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v[8];
            get(k, i, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[k] = __builtin_fmaf(v[e] * kDown, v[e] * kDown, s[k]);
        }
    }
    row_sums<LPR>(s, wpr, lds, turn);
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (over[k]) sum[k] = __builtin_fmaf(s[k], inv_n / (kDown * kDown), eps);
}

// Waves per row and chunks per lane: one chunk per lane while eight waves hold
// the row, then the fewest chunks that do.  (Forward and backward with one and
// two chunks per lane, 4096x2560: 21.8 / 23.0 and 37.3 / 38.9 us.)
inline void row_split(int64_t cols, int* wpr, int* nv) {
    const int64_t groups = (cols / 8 + 63) / 64;            // chunks of 64 lanes
    *nv = (int)((groups + kMaxRowWaves - 1) / kMaxRowWaves);
    *wpr = (int)((groups + *nv - 1) / *nv);
}
// Lanes per row of a row that one wave holds in one chunk per lane.
inline int row_lanes(int64_t cols) { return cols <= 128 ? 16 : cols <= 256 ? 32 : 64; }

}  // namespace fp8bs
