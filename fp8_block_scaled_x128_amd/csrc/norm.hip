// The norms around a block and what joins it to the residual stream.  With
// N(v; w) = v * rsqrt(mean(v^2) + eps) * w by rows:
//
//   h = residual + scale * gate * N(x; w_post)
//   y = N(h; w_pre), and y's 1x128 groups as E4M3 codes with S = max|y| / 448
//
// so the tensor that a linear layer's 1x128 quantizer would read (the "per-
// token" activations of "Unified FP8: Beyond Mixed Precision...", section
// "FP8 Quantization") is quantized where it is made.  HBM-bound: each input is
// read once, each output written once, and all between stays in fp32
// registers.
//
// Measured (a 1 GiB device copy moves 5.2 TB/s on the same card): 4096x2560
// bf16 with every output, 95 MB, 21 us (4.5 TB/s); 16384x2048 over an fp32
// stream with a gate per sequence, 437 MB, 91 us (4.8); 131072x128 29.9 us
// (5.1); one row of 2560 3.6 us, all latency: three dependent trips to memory
// (w_pre, w_post, then the row: a bf16 weight is converted, so waited for,
// before the next load) and two reductions.  Wide rows: 2048x10240 44.8 us
// (4.2 TB/s), 2032x16384 72 (4.2).  A row per workgroup without the next row in
// flight: 28.4, 90.1, 64.4 (131072x128 by wave) and 4.1 us.
#include "norm_common.h"

namespace fp8bs {
namespace {

constexpr int kRowWaves = 4;         // waves of a workgroup whose rows need one wave each
// Workgroups at most: about 5120 waves of one chunk per lane, which is where
// more rows in flight stop paying (16384x768: 1024 workgroups of two waves 34.7
// us, 2048 25.4; 4096x5120: 1024 workgroups of five waves with two chunks 49.0,
// 512 39.2; 4096x2560: 1024 of five waves 20.8, 2048 23.9), equally many per
// compute unit (16384x2048: 1024 of four waves 90.5, 1261 93.6) and two at least.
int64_t workgroups(int wpr, int nv) {
    const int64_t n = 5120 / (wpr * nv) / kCUs * kCUs;
    return n < 2 * kCUs ? 2 * kCUs : n;
}

// One row as loaded.
template <int NV, bool RES32>
struct RowIn {
    Raw8<RES32> res[NV];
    Raw8<false> x[NV], gate[NV];
    __device__ __forceinline__ void load(const NormArgs& p, int64_t row, int tid, int step, int nc) {
        const void* residual_row = row_ptr<RES32>(p.residual, row, p.ld_r);
        const void* x_row = row_ptr<false>(p.x, row, p.ld_x);
        if (p.x) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) x[i].load(x_row, c);
            }
        }
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) res[i].load(residual_row, c);
            }
        }
        if (p.gate) {
            const uint16_t* g_row = row_ptr<false>(p.gate, (int64_t)((uint32_t)row / (uint32_t)p.rows_per_gate), p.ld_gate);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) gate[i].load_shared(g_row, c);
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NV; ++i) { res[i].zero(); x[i].zero(); gate[i].zero(); }
    }
};

// LPR lanes have a row; kMulti: a workgroup has one row at a time.
// One or two chunks per lane (AHEAD): the next row is loaded while this one is
// reduced and stored, and the weights stay in registers: a weight load from
// the L2 behind the next row's loads would wait for them, since loads return
// in order.  More chunks have no registers left for it.
template <int NV, bool RES32, int LPR>
__global__ void __launch_bounds__(512) k_block_norm(NormArgs p, int wpr) {
    constexpr bool MULTI = LPR == kMulti, SHARED = LPR == 16 || LPR == 32;     // SHARED: a wave has several rows
    constexpr bool AHEAD = NV <= 2;
    constexpr int KEPT = AHEAD ? NV : 1;
    __shared__ float lds[2][kMaxRowWaves][4];
    const int tid = MULTI ? threadIdx.x : threadIdx.x % (MULTI ? 64 : LPR);
    const int sub = SHARED ? (threadIdx.x & 63) / (MULTI ? 64 : LPR) : 0;
    const int nc = p.cols >> 3, step = MULTI ? wpr * 64 : 64;
    const float inv_n = 1.0f / (float)p.cols;
    int turn = 0;
    float wpre[KEPT][8], wpost[KEPT][8];
#pragma unroll
    for (int i = 0; i < KEPT; ++i) {
        const int c = min(tid + i * step, nc - 1);          // past the row: x and residual are 0
#pragma unroll
        for (int e = 0; e < 8; ++e) wpre[i][e] = wpost[i][e] = 1.0f;
        if (AHEAD && p.w_pre) load8_shared(p.w_pre, c, p.w32, wpre[i]);
        if (AHEAD && p.w_post) load8_shared(p.w_post, c, p.w32, wpost[i]);
    }
    constexpr int kWaveRows = MULTI ? 1 : 64 / (MULTI ? 64 : LPR);
    const int64_t per = MULTI ? 1 : kRowWaves * kWaveRows;  // rows a workgroup has at a time
    const int64_t first = MULTI ? (int64_t)blockIdx.x
                                : (int64_t)blockIdx.x * per + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kWaveRows;
    // chunks of this lane's row: none past the last row (the lane stays for
    // the reductions)
    auto chunks = [&](int64_t row) { return !SHARED || row < p.rows ? nc : 0; };
    const int64_t stride = (int64_t)gridDim.x * per;
    RowIn<NV, RES32> in, ahead;
    in.zero();
    if (AHEAD) {
        ahead.zero();
        if (first < p.rows) ahead.load(p, first + sub, tid, step, chunks(first + sub));
    }
    for (int64_t row0 = first; row0 < p.rows; row0 += stride) {
        const int64_t row = row0 + sub;
        const int ncr = chunks(row);
        if (AHEAD) {
            in = ahead;
            if (row0 + stride < p.rows) ahead.load(p, row + stride, tid, step, chunks(row + stride));
        } else {
            in.load(p, row, tid, step, ncr);
        }
        float r = 1.0f;
        if (p.w_post) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[8];
                in.x[i].get(v);
                ss[0] += sumsq8(v);
            }
            row_sums<LPR>(ss, wpr, lds, turn);
#pragma unroll
            for (int i = 0; i < NV; ++i) in.x[i].forget();
            row_means<LPR, NV>(ss, [&](int, int i, float v[8]) { in.x[i].get(v); }, inv_n, p.eps, wpr, lds, turn);
            r = inv_sqrt(ss[0]);
        }
        float h[NV][8];
        float ss[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * step;
            float v[8], gate[8];
            in.res[i].get(h[i]);
            in.x[i].get(v);
            if (!AHEAD && p.w_post) load8_shared(p.w_post, min(c, nc - 1), p.w32, wpost[i % KEPT]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * r * wpost[i % KEPT][e];
            if (p.gate) {
                in.gate[i].get(gate);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= gate[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = __builtin_fmaf(v[e], p.scale, h[i][e]);
            if (p.h && (i < kSure<NV> || c < ncr)) store8<RES32>(row_ptr<RES32>(p.h, row, p.ld_h), c, h[i]);
            ss[0] += sumsq8(h[i]);
        }
        if (!p.w_pre) continue;
        // y from the unrounded h: the bf16 rounding of the stored stream does
        // not enter y, its scales or its codes
        row_sums<LPR>(ss, wpr, lds, turn);
        const auto h_at = [&](int, int i, float v[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = h[i][e];
        };
        row_means<LPR, NV>(ss, h_at, inv_n, p.eps, wpr, lds, turn);
        r = inv_sqrt(ss[0]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * step;
            const bool in_row = i < kSure<NV> || c < ncr;
            if (!AHEAD) load8_shared(p.w_pre, min(c, nc - 1), p.w32, wpre[i % KEPT]);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * r * wpre[i % KEPT][e];
            if (p.y && in_row) store8<false>(row_ptr<false>(p.y, row, p.ld_y), c, h[i]);
            if (p.q) {
                // 16 lanes hold a 128-column group; lanes past the row hold zeros
                const float s = row16_max(absmax8(h[i])) / kE4M3Max;
                uint32_t w0, w1;
                encode8(h[i], s, w0, w1);
                if (in_row) {
                    *reinterpret_cast<uint2*>(p.q + row * p.ld_q + 8u * (uint32_t)c) = make_uint2(w0, w1);
                    if ((c & 15) == 0) p.s[row * p.ssr + (int64_t)(c >> 4) * p.ssg] = s;
                }
            }
        }
    }
}

template <int NV, int LPR>
hipError_t launch_types(const NormArgs& p, int wpr, hipStream_t st) {
    const int per = LPR == kMulti ? 1 : kRowWaves * 64 / (LPR == kMulti ? 64 : LPR), waves = LPR == kMulti ? wpr : kRowWaves;
    const int64_t blocks = (p.rows + per - 1) / per, most = workgroups(waves, NV);
    hipLaunchKernelGGL((p.res32 ? k_block_norm<NV, true, LPR> : k_block_norm<NV, false, LPR>),
                       dim3((unsigned)(blocks < most ? blocks : most)), dim3(64 * waves), 0, st, p, wpr);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& p, hipStream_t st) {
    int wpr, nv;
    row_split(p.cols, &wpr, &nv);
    if (wpr == 1) {
        switch (row_lanes(p.cols)) {
            case 16: return launch_types<1, 16>(p, wpr, st);
            case 32: return launch_types<1, 32>(p, wpr, st);
            default: return launch_types<1, 64>(p, wpr, st);
        }
    }
    switch (nv) {
        case 1: return launch_types<1, kMulti>(p, wpr, st);
        case 2: return launch_types<2, kMulti>(p, wpr, st);
        case 3: return launch_types<3, kMulti>(p, wpr, st);
        default: return launch_types<4, kMulti>(p, wpr, st);
    }
}

}  // namespace fp8bs
