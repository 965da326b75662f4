// What the routers share: a token's logits as ordered keys, a selecting
// workgroup's histogram and loss terms, and the rows of the stable (expert, token)
// order.
#pragma once
#include "device_common.h"
#include "internal.h"
#include "reduce.h"

namespace fp8bs {

constexpr int kTok = 64;            // tokens of a workgroup: the bits of one mask word per expert
constexpr int kThreads = 1024;
constexpr float kLog2e = 1.4426950408889634f;

// Order-preserving 32-bit key of a logit: larger logits have larger keys, -0
// and +0 the same one, NaN the largest.  0 is below every logit's key.
__device__ __forceinline__ uint32_t logit_key(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return z != z ? 0xffffffffu : k;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;

// A lane's logits l, l + L, ... of the row that starts at element `row`.  No
// load is conditional (past the row: the last expert's, dropped by the
// caller), so all are in flight at once.
template <int L, int V, bool F32>
__device__ __forceinline__ void load_logits(const void* base, int64_t row, int l, int E, float (&z)[V]) {
    if (F32) {
        const float* r = static_cast<const float*>(base) + row;
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = r[min(l + i * L, E - 1)];
    } else {
        const uint16_t* r = static_cast<const uint16_t*>(base) + row;
        uint16_t w[V];
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = r[min(l + i * L, E - 1)];
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = __uint_as_float((uint32_t)w[i] << 16);
    }
}

// Exclusive prefix of counts[0..E) into LDS, by the first wave; E <= 1024.
__device__ __forceinline__ void scan_experts(const int* counts, int* excl, int E) {
    if (threadIdx.x < 64) {
        int carry = 0;
        for (int b = 0; b < E; b += 64) {
            const int e = b + threadIdx.x;
            const int c = e < E ? counts[e] : 0;
            const int v = wave_scan(c);
            if (e < E) excl[e] = carry + v - c;
            carry += (int)lane_value((uint32_t)v, 63);
        }
        if (threadIdx.x == 0) excl[E] = carry;
    }
}

// Sums of K values per thread over the 16 waves of a workgroup, in a fixed
// order (all threads call; lds holds 16 K floats; every thread has the result).
template <int K>
__device__ __forceinline__ void block_sums(float (&v)[K], float* lds) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = lanes_sum<64>(v[i]);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) lds[16 * i + (threadIdx.x >> 6)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = row16_sum(lds[16 * i + (threadIdx.x & 15)]);
}

// LDS of a selecting workgroup: the experts' token masks, and the probability
// sums of half of its waves [8][L V] (the halves take turns: 1024 experts would
// pass 64 KB otherwise).
constexpr int kHalf = kThreads / 128;
__host__ __device__ constexpr size_t select_lds(int E, int lv) { return (size_t)E * 8 + (size_t)lv * 4 * kHalf; }

// The row of a workgroup's slot i with expert e, given the masks in LDS and the
// expert's first row for the workgroup, and the zeros of row_token behind the
// last row.
__device__ __forceinline__ void place_row(const RouteArgs& p, int64_t t0, int64_t i, int e,
                                          const unsigned long long* mask, int first, int total) {
    const int64_t at = t0 * p.k + i;
    const int tt = (int)((uint32_t)i / (uint32_t)p.k);
    int row = -1;
    if (e >= 0) {
        row = first + __popcll(mask[e] & ((1ull << tt) - 1));
        p.row_token[row] = (int32_t)(t0 + tt);
    }
    p.token_rows[at] = row;
    if (at >= total) p.row_token[at] = 0;
}

__device__ __forceinline__ void write_losses(const RouteArgs& p, float fp, float lse2, int64_t sum_counts, int live) {
    const float n = (float)max(live, 1);
    p.loss[0] = (float)p.E * fp / ((float)max(sum_counts, (int64_t)1) * n);
    p.loss[1] = lse2 / n;
}

// Up to 64 tokens: the whole routing in one workgroup.  select(mask, psum) makes
// the selection: per expert the mask of the tokens that chose it, psum[0..E) the
// probability sums; {sum of lse^2, routed tokens} to every thread.  psum holds
// `floats` floats.
template <class S>
__device__ __forceinline__ void route_one(const RouteArgs& p, unsigned char* dyn, int floats, S select) {
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(dyn);
    float* psum = reinterpret_cast<float*>(mask + p.E);
    int* counts = reinterpret_cast<int*>(psum + floats);
    int* base = counts + p.E;                       // [E + 1]
    __shared__ float red[16];
    for (int e = threadIdx.x; e < p.E; e += kThreads) mask[e] = 0;
    __syncthreads();
    const float2 s = select(mask, psum);
    float f[1] = {0.0f};
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        const int c = __popcll(mask[e]);
        counts[e] = c;
        p.counts[e] = c;
        f[0] = __builtin_fmaf((float)c, psum[e], f[0]);
    }
    block_sums(f, red);                             // its barrier covers counts too
    scan_experts(counts, base, p.E);
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = base[e];
    for (int64_t i = threadIdx.x; i < p.T * p.k; i += kThreads) {
        const int e = p.experts[i];
        place_row(p, 0, i, e, mask, base[max(e, 0)], base[p.E]);
    }
    if (threadIdx.x == 0) {
        p.counts[p.E] = (int)s.y;
        write_losses(p, f[0], s.x, base[p.E], (int)s.y);
    }
}

// More tokens, first launch: selection, and per workgroup the histogram (a
// byte per expert: at most 64), the probability sums and the loss terms.
template <class S>
__device__ __forceinline__ void route_select(const RouteArgs& p, const RouteWs& ws, unsigned char* dyn, S select) {
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(dyn);
    float* psum = reinterpret_cast<float*>(mask + p.E);
    for (int e = threadIdx.x; e < p.E; e += kThreads) mask[e] = 0;
    __syncthreads();
    const float2 s = select(mask, psum);
    for (int e = threadIdx.x; e < ws.epad; e += kThreads) {
        ws.hist[(int64_t)blockIdx.x * ws.epad + e] = e < p.E ? (uint8_t)__popcll(mask[e]) : (uint8_t)0;
        ws.psum[(int64_t)blockIdx.x * ws.epad + e] = e < p.E ? psum[e] : 0.0f;
    }
    if (threadIdx.x == 0) {
        ws.lse2[blockIdx.x] = s.x;
        ws.live[blockIdx.x] = (int)s.y;
    }
}

}  // namespace fp8bs
