// MoE combine: each token's output is the routing-weighted sum of its
// experts' outputs, read from the grouped (expert-sorted) down-projection
// output through the token's row positions.  It closes the MoE layer whose
// grouped GEMMs run in block-wise FP8 ("Low Precision RL", section
// "2. Unified block-wise FP8 (DeepSeek-style)", the Qwen3-30B-A3B recipe).
//
// HBM-bound: k bf16 rows read per token, one row written.  One thread owns
// one (token, 8-column chunk) pair: the k rows of a token are each read as
// one contiguous run across the workgroup (16-byte loads), up to eight rows are
// loaded before the FMAs, and the sum is an fp32 FMA chain in slot order
// (deterministic: no atomics, no order that depends on scheduling).  A slot's
// position is waited for before its row is loaded, and loads return in order,
// so one thread's slots are up to eight round trips; other waves fill them at
// 16384 tokens, nothing does in decode.  Measured, 2048 columns, top-8: 16384
// tokens 605 MB in 107 us (5.6 TB/s, the rate of a large copy), 512 tokens 7.1
// us, 32 tokens 3.6, one 2.8; on the router's maps (SKIP) 107.6, 7.8, 4.1, 3.0.
#include "device_common.h"
#include "internal.h"
#include "reduce.h"

namespace fp8bs {
namespace {

constexpr int kThreads = 256;

// SKIP: a slot whose position is outside [0, rows) contributes nothing (the
// router leaves -1 there); otherwise positions are clamped.
template <bool OUTF32, bool SKIP>
__global__ void __launch_bounds__(kThreads) k_moe_combine(const uint16_t* __restrict__ y, int32_t rows, int32_t nch,
                                                          int64_t ld_y, const int32_t* __restrict__ pos,
                                                          const float* __restrict__ w, int64_t T, int32_t k,
                                                          void* __restrict__ out, int64_t ld_out) {
    const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (idx >= T * nch) return;
    const int64_t t = idx / nch;
    const int c = (int)(idx - t * nch);
    const int32_t* pt = pos + t * k;
    const float* wt = w + t * k;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 8) {
        uint4 raw[8];
        float wj[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (j0 + u < k) {
                const int pj = pt[j0 + u];
                if (SKIP && (uint32_t)pj >= (uint32_t)rows) {
                    raw[u] = make_uint4(0, 0, 0, 0);
                    wj[u] = 0.0f;
                    continue;
                }
                // positions outside [0, rows) are clamped: a bad map reads
                // wrong rows, never outside y
                const int r = SKIP ? pj : min(max(pj, 0), rows - 1);
                raw[u] = load_nt16(y + (int64_t)r * ld_y + 8 * c);
                wj[u] = wt[j0 + u];
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (j0 + u < k) {
                const uint32_t v[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[2 * i] = __builtin_fmaf(wj[u], bf16_lo(v[i]), acc[2 * i]);
                    acc[2 * i + 1] = __builtin_fmaf(wj[u], bf16_hi(v[i]), acc[2 * i + 1]);
                }
            }
        }
    }
    if (OUTF32) {
        float* dst = static_cast<float*>(out) + t * ld_out + 8 * c;
        *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else {
        uint16_t* dst = static_cast<uint16_t*>(out) + t * ld_out + 8 * c;
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                                     pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
    }
}

// Gradient of the combine: dy[row] = w dout[t] and dw = <dout[t], y[row]> for
// every (token, slot) with a row.  WPT waves hold a token and walk the columns
// in runs of 512 each (8 per lane): per run, dout is loaded once and up to
// eight y rows are in flight, each giving its part of a dot product and
// taking its dy row at once, so nothing of a row stays in registers.
// HBM-bound: 16384 tokens x 2048, top-8, 1.14 GB in 205 us (5.6 TB/s, the rate
// of a large copy).
template <bool DO32, int WPT>
__global__ void __launch_bounds__(kThreads) k_moe_combine_bwd(const void* __restrict__ dout, int64_t ld_do,
                                                              const uint16_t* __restrict__ y, int32_t rows,
                                                              int32_t nch, int64_t ld_y,
                                                              const int32_t* __restrict__ pos,
                                                              const float* __restrict__ w, int64_t T, int32_t k,
                                                              uint16_t* __restrict__ dy, int64_t ld_dy,
                                                              float* __restrict__ dw) {
    constexpr int kWaves = kThreads / 64, kPer = kWaves / WPT;
    __shared__ float part[WPT > 1 ? kWaves : 1][8];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kPer + wave / WPT;
    const bool have = t < T;
    for (int j0 = 0; j0 < k; j0 += 8) {
        int r[8];
        float wj[8], dot[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int pj = have && j0 + u < k ? pos[t * k + j0 + u] : -1;
            r[u] = (uint32_t)pj < (uint32_t)rows ? pj : -1;
            wj[u] = r[u] >= 0 ? w[t * k + j0 + u] : 0.0f;
            dot[u] = 0.0f;
        }
        for (int c = have ? (wave % WPT) * 64 + lane : nch; c < nch; c += 64 * WPT) {
            uint4 raw[8];
            float d[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (r[u] >= 0 && dw) raw[u] = load_nt16(y + (int64_t)r[u] * ld_y + 8 * c);
            if (DO32) {
                const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(dout) + t * ld_do + 8 * c);
                const float4 a = f[0], b = f[1];
                d[0] = a.x; d[1] = a.y; d[2] = a.z; d[3] = a.w;
                d[4] = b.x; d[5] = b.y; d[6] = b.z; d[7] = b.w;
            } else {
                unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(dout) + t * ld_do + 8 * c), d);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (r[u] < 0) continue;
                if (dw) {
                    float v[8];
                    unpack8(raw[u], v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[u] = __builtin_fmaf(d[i], v[i], dot[u]);
                }
                if (dy)
                    store_nt16(dy + (int64_t)r[u] * ld_dy + 8 * c,
                               make_uint4(pack_bf16x2(wj[u] * d[0], wj[u] * d[1]), pack_bf16x2(wj[u] * d[2], wj[u] * d[3]),
                                          pack_bf16x2(wj[u] * d[4], wj[u] * d[5]), pack_bf16x2(wj[u] * d[6], wj[u] * d[7])));
            }
        }
        if (!dw) continue;
#pragma unroll
        for (int u = 0; u < 8; ++u) dot[u] = lanes_sum<64>(dot[u]);
        if (WPT > 1) {
            if (lane == 0) {
#pragma unroll
                for (int u = 0; u < 8; ++u) part[WPT > 1 ? wave : 0][u] = dot[u];
            }
            __syncthreads();
            if (wave % WPT == 0 && lane < 8 && have && j0 + lane < k) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < WPT; ++i) s += part[WPT > 1 ? wave + i : 0][lane];
                dw[t * k + j0 + lane] = s;
            }
            __syncthreads();
        } else if (have) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (lane == 0 && j0 + u < k) dw[t * k + j0 + u] = dot[u];
        }
    }
}

}  // namespace

hipError_t launch_moe_combine(const uint16_t* y, int64_t rows, int64_t H, int64_t ld_y, const int32_t* pos,
                              const float* w, int64_t T, int32_t k, void* out, int64_t ld_out, int out_f32,
                              bool skip, hipStream_t st) {
    if (T == 0 || H == 0) return hipSuccess;
    const int32_t nch = (int32_t)(H / 8);
    const int64_t blocks = (T * nch + kThreads - 1) / kThreads;
    const auto k_fn = out_f32 ? (skip ? k_moe_combine<true, true> : k_moe_combine<true, false>)
                              : (skip ? k_moe_combine<false, true> : k_moe_combine<false, false>);
    hipLaunchKernelGGL(k_fn, dim3((unsigned)blocks), dim3(kThreads), 0, st, y, (int32_t)rows, nch, ld_y, pos, w, T, k,
                       out, ld_out);
    return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const void* dout, int64_t ld_do, int do_f32, const uint16_t* y, int64_t rows,
                                  int64_t H, int64_t ld_y, const int32_t* pos, const float* w, int64_t T, int32_t k,
                                  uint16_t* dy, int64_t ld_dy, float* dw, hipStream_t st) {
    if (T == 0) return hipSuccess;
    // Waves per token: as many as have a run of columns each and, over the
    // slots, four rows of one (16384 tokens x 2048, k 8: 1 / 2 / 4 waves 224 /
    // 214 / 205 us; k 1: 34.1 / 34.8 / 41.8; 16384 x 128, k 2: 12.6 / 18.4 /
    // 30.1).
    const int64_t runs = (H / 8 + 63) / 64, rows_of = runs * (k < 8 ? k : 8);
    const int wpt = runs >= 4 && rows_of >= 16 ? 4 : runs >= 2 && rows_of >= 8 ? 2 : 1;
    const int64_t per = kThreads / 64 / wpt;
    const auto k_fn =
        do_f32 ? (wpt == 4 ? k_moe_combine_bwd<true, 4> : wpt == 2 ? k_moe_combine_bwd<true, 2> : k_moe_combine_bwd<true, 1>)
               : (wpt == 4 ? k_moe_combine_bwd<false, 4> : wpt == 2 ? k_moe_combine_bwd<false, 2> : k_moe_combine_bwd<false, 1>);
    // a launch holds fewer than 2^32 threads, with a workgroup per token 2^24
    // tokens: more go in several
    constexpr int64_t kMost = 1ll << 23;
    for (int64_t t = 0; t < T; t += kMost) {
        const int64_t n = T - t < kMost ? T - t : kMost;
        const void* d = static_cast<const char*>(dout) + t * ld_do * (do_f32 ? 4 : 2);
        hipLaunchKernelGGL(k_fn, dim3((unsigned)((n + per - 1) / per)), dim3(kThreads), 0, st, d, ld_do, y,
                           (int32_t)rows, (int32_t)(H / 8), ld_y, pos + t * k, w + t * k, n, k, dy, ld_dy,
                           dw ? dw + t * k : nullptr);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace fp8bs
