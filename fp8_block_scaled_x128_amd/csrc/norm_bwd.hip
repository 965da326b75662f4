// Gradient of the block norm (norm.hip) from the saved h and x.  The norms'
// factors are formed again: a sum of squares beside the sums that the
// gradient needs anyway.
//
//   hh = h r;  g = dy w_pre;  dH = dh + r (g - hh mean(g hh));  dres = dH
//   dw_pre = sum_rows dy hh
//   xh = x r';  dn = scale gate dH;  dgate = sum scale dH xh w_post
//   dw_post = sum_rows dn xh;  dx = r' (dn w_post - xh mean(dn w_post xh))
//
// HBM-bound.  A workgroup walks units of consecutive rows that share a gate
// row; its column sums of dw_pre and dw_post stay in registers over all its
// rows and leave one partial row each, which k_col_reduce adds in workgroup
// order (no atomics: the same bits every time).
#include "norm_common.h"

namespace fp8bs {
namespace {

constexpr int kWaves = 8;                // waves of a workgroup whose rows need one wave each
constexpr int kSlots = 512;              // workgroups at most

// Adds the waves' register sums in wave order (one wave per row: 8 rows at a
// time); the last wave's registers hold the result.
__device__ __forceinline__ void combine_waves(float (&a)[8], float (*comb)[8], int wave) {
    const int lane = threadIdx.x & 63;
    for (int w = 0; w < kWaves; ++w) {
        __syncthreads();
        if (wave == w) {
            float4* s = reinterpret_cast<float4*>(comb[lane]);
            if (w > 0) {
                const float4 u = s[0], v = s[1];
                a[0] += u.x; a[1] += u.y; a[2] += u.z; a[3] += u.w;
                a[4] += v.x; a[5] += v.y; a[6] += v.z; a[7] += v.w;
            }
            s[0] = make_float4(a[0], a[1], a[2], a[3]);
            s[1] = make_float4(a[4], a[5], a[6], a[7]);
        }
    }
    __syncthreads();
}

// One row as loaded.
template <int NV, bool RES32, bool DY32, bool GACC>
struct RowIn {
    Raw8<RES32> dh[NV], h[NV];
    Raw8<DY32> dy[NV];
    Raw8<false> x[NV], gate[GACC ? 1 : NV];
    __device__ __forceinline__ void load(const NormBwdArgs& p, int64_t row, int tid, int step, int nc) {
        if (p.w_pre) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) {
                    h[i].load(p.h, row * p.ld_h + 8 * c);
                    dy[i].load(p.dy, row * p.ld_dy + 8 * c);
                }
            }
        }
        if (p.x) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) x[i].load(p.x, row * p.ld_x + 8 * c);
            }
        }
        if (p.dh) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) dh[i].load(p.dh, row * p.ld_dh + 8 * c);
            }
        }
        if (!GACC && p.gate) {
            const int64_t g = (int64_t)((uint32_t)row / (uint32_t)p.rows_per_gate) * p.ld_gate;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) gate[GACC ? 0 : i].load(p.gate, g + 8 * c);
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            dh[i].zero(); h[i].zero(); dy[i].zero(); x[i].zero(); gate[GACC ? 0 : i].zero();
        }
    }
};

// MULTI: a workgroup has one row at a time, else each of its waves has one.
// GACC: the gate's gradient is summed over the rows of a gate row.
// One or two chunks per lane (AHEAD): the next row is loaded while this one is
// reduced and stored, and the weights stay in registers: a weight load from
// the L2 behind the next row's loads would wait for them, since loads return
// in order.  More chunks have no registers left for it.
template <int NV, bool RES32, bool DY32, bool MULTI, bool GACC>
__global__ void __launch_bounds__(512) k_block_norm_bwd(NormBwdArgs p, NormBwdPlan pl) {
    constexpr bool AHEAD = NV <= 2;
    __shared__ float lds[2][kMaxRowWaves][4];
    __shared__ float comb[MULTI ? 1 : 64][8];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wpr = pl.wpr;
    const int tid = MULTI ? threadIdx.x : (threadIdx.x & 63);
    const int nc = p.cols >> 3, step = MULTI ? wpr * 64 : 64;
    const float inv_n = 1.0f / (float)p.cols;
    int turn = 0;
    float awpre[NV][8], awpost[NV][8], agate[NV][8];
    constexpr int KEPT = AHEAD ? NV : 1;
    float wpre[KEPT][8], wpost[KEPT][8], wgate[KEPT][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            awpre[i][e] = awpost[i][e] = 0.0f;
            wpre[i % KEPT][e] = wpost[i % KEPT][e] = wgate[i % KEPT][e] = 1.0f;
        }
        const int c = min(tid + i * step, nc - 1);      // past the row: dy, dh and x are 0
        if (AHEAD && p.w_pre) load8_shared(p.w_pre, 8 * c, p.w32, wpre[i % KEPT]);
        if (AHEAD && p.w_post) load8_shared(p.w_post, 8 * c, p.w32, wpost[i % KEPT]);
    }
    // units by workgroup, its waves taking rows in turn; or (short gate rows)
    // by wave
    const bool by_wave = !MULTI && pl.by_wave;
    const int64_t u0 = by_wave ? (int64_t)blockIdx.x * kWaves + wave : blockIdx.x;
    const int64_t ustep = by_wave ? (int64_t)gridDim.x * kWaves : gridDim.x;
    const int rstep = MULTI || by_wave ? 1 : kWaves;
    for (int64_t u = u0; u < pl.units; u += ustep) {
        const int64_t g = u / pl.splits;
        const int64_t r0 = g * pl.unit_rows + (u - g * pl.splits) * pl.chunk + (rstep == 1 ? 0 : wave);
        const int64_t r1 = min(min(r0 - (rstep == 1 ? 0 : wave) + pl.chunk, (g + 1) * pl.unit_rows), p.rows);
        if (GACC) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = min(tid + i * step, nc - 1);
                if (AHEAD) load8_shared(p.gate, g * p.ld_gate + 8 * c, false, wgate[i % KEPT]);
#pragma unroll
                for (int e = 0; e < 8; ++e) agate[i][e] = 0.0f;
            }
        }
        RowIn<NV, RES32, DY32, GACC> in, ahead;
        in.zero();
        if (AHEAD) {
            ahead.zero();
            if (r0 < r1) ahead.load(p, r0, tid, step, nc);
        }
        for (int64_t row = r0; row < r1; row += rstep) {
            if (AHEAD) {
                in = ahead;
                if (row + rstep < r1) ahead.load(p, row + rstep, tid, step, nc);
            } else {
                in.load(p, row, tid, step, nc);
            }
            float sums[3] = {0.0f, 0.0f, 0.0f};     // sum h^2, sum dy w_pre h, sum x^2
            if (p.w_pre) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = min(tid + i * step, nc - 1);
                    float h[8], dy[8];
                    if (!AHEAD) load8_shared(p.w_pre, 8 * c, p.w32, wpre[i % KEPT]);
                    in.h[i].get(h);
                    in.dy[i].get(dy);
                    sums[0] += sumsq8(h);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dy[e] *= wpre[i % KEPT][e];
                    sums[1] += dot8(dy, h);
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[8];
                in.x[i].get(x);
                sums[2] += sumsq8(x);
            }
            row_sums<MULTI>(sums, wpr, lds, turn);
            float dh[NV][8];
#pragma unroll
            for (int i = 0; i < NV; ++i) in.dh[i].get(dh[i]);
            if (p.w_pre) {
                const float r = inv_sqrt(__builtin_fmaf(sums[0], inv_n, p.eps));
                const float m = sums[1] * inv_n * r * r;        // mean(g hh) r: times h, hh mean(g hh)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = min(tid + i * step, nc - 1);
                    float h[8], dy[8];
                    if (!AHEAD) load8_shared(p.w_pre, 8 * c, p.w32, wpre[i % KEPT]);
                    in.h[i].get(h);
                    in.dy[i].get(dy);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        awpre[i][e] = __builtin_fmaf(dy[e] * r, h[e], awpre[i][e]);
                        dh[i][e] = __builtin_fmaf(r, __builtin_fmaf(-m, h[e], dy[e] * wpre[i % KEPT][e]), dh[i][e]);
                    }
                }
            }
            if (p.dres) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = tid + i * step;
                    if (i < kSure<NV> || c < nc) store8<RES32>(p.dres, row * p.ld_dres + 8 * c, dh[i]);
                }
            }
            if (!p.x) continue;
            const float rx = p.w_post ? inv_sqrt(__builtin_fmaf(sums[2], inv_n, p.eps)) : 1.0f;
            float dot[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = min(tid + i * step, nc - 1);
                float dg[8], x[8];
                in.x[i].get(x);
                if (!AHEAD && p.w_post) load8_shared(p.w_post, 8 * c, p.w32, wpost[i % KEPT]);
                if (!AHEAD && GACC) load8_shared(p.gate, g * p.ld_gate + 8 * c, false, wgate[i % KEPT]);
                if (!GACC && p.gate) in.gate[GACC ? 0 : i].get(wgate[i % KEPT]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float dn = dh[i][e] * p.scale;
                    const float xh = x[e] * rx;
                    if (GACC || p.gate) {
                        dg[e] = dn * (xh * wpost[i % KEPT][e]);
                        if (GACC) agate[i][e] += dg[e];
                        dn *= wgate[i % KEPT][e];
                    }
                    awpost[i][e] = __builtin_fmaf(dn, xh, awpost[i][e]);
                    dn *= wpost[i % KEPT][e];
                    dot[0] = __builtin_fmaf(dn, xh, dot[0]);
                    dh[i][e] = dn;                      // the gradient at xh from here on
                }
                if (!GACC && p.dgate && (i < kSure<NV> || tid + i * step < nc)) {
                    if (p.dgate32) store8<true>(p.dgate, row * p.ld_dgate + 8 * c, dg);
                    else store8<false>(p.dgate, row * p.ld_dgate + 8 * c, dg);
                }
            }
            if (!p.dx) continue;
            float m = 0.0f;
            if (p.w_post) {
                row_sums<MULTI>(dot, wpr, lds, turn);
                m = dot[0] * inv_n * rx * rx;           // mean(g xh) r': times x
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                float d[8], x[8];
                in.x[i].get(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = __builtin_fmaf(-m, x[e], dh[i][e] * rx);
                if (i < kSure<NV> || c < nc) store8<false>(p.dx, row * p.ld_dx + 8 * c, d);
            }
        }
        if (GACC) {
            if (!MULTI && !by_wave) {
#pragma unroll
                for (int i = 0; i < NV; ++i) combine_waves(agate[i], comb, wave);
            }
            if (MULTI || by_wave || wave == kWaves - 1) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = tid + i * step;
                    if (i >= kSure<NV> && c >= nc) continue;
                    if (pl.splits > 1) store8<true>(pl.ws_gate, u * p.cols + 8 * c, agate[i]);
                    else if (p.dgate32) store8<true>(p.dgate, g * p.ld_dgate + 8 * c, agate[i]);
                    else store8<false>(p.dgate, g * p.ld_dgate + 8 * c, agate[i]);
                }
            }
        }
    }
    if (!MULTI) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (p.dw_pre) combine_waves(awpre[i], comb, wave);
            if (p.dw_post) combine_waves(awpost[i], comb, wave);
        }
        if (wave != kWaves - 1) return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * step;
        if (i >= kSure<NV> && c >= nc) continue;
        if (p.dw_pre) store8<true>(pl.ws_pre, (int64_t)blockIdx.x * p.cols + 8 * c, awpre[i]);
        if (p.dw_post) store8<true>(pl.ws_post, (int64_t)blockIdx.x * p.cols + 8 * c, awpost[i]);
    }
}

// Column sums of partial rows: job 0 / 1 (dw_pre, dw_post) over the
// workgroups, job 2 + g (dgate row g) over its units, each in order.  A
// workgroup takes 32 columns; its 128 row lanes add every 128th partial, then
// meet in LDS in a fixed order.
constexpr int kRedCols = 32, kRedRows = 128;
__global__ void __launch_bounds__(1024) k_col_reduce(NormBwdArgs p, NormBwdPlan pl) {
    __shared__ float4 acc[kRedRows][kRedCols / 4];
    const int tx = threadIdx.x % (kRedCols / 4), ty = threadIdx.x / (kRedCols / 4);
    const int c = blockIdx.x * kRedCols + 4 * tx;
    const int j = blockIdx.y;
    const bool gate = j >= 2;
    const float* src = j == 0 ? pl.ws_pre : j == 1 ? pl.ws_post : pl.ws_gate + (int64_t)(j - 2) * pl.splits * p.cols;
    const int64_t n = gate ? pl.splits : pl.slots;
    if ((j == 0 && !p.dw_pre) || (j == 1 && !p.dw_post)) return;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < p.cols) {
        for (int64_t r = ty; r < n; r += kRedRows) {
            const float4 v = *reinterpret_cast<const float4*>(src + r * p.cols + c);
            a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
        }
    }
    acc[ty][tx] = a;
    __syncthreads();
    for (int s = kRedRows / 2; s > 0; s >>= 1) {
        if (ty < s) {
            const float4 b = acc[ty + s][tx];
            float4 t = acc[ty][tx];
            t.x += b.x; t.y += b.y; t.z += b.z; t.w += b.w;
            acc[ty][tx] = t;
        }
        __syncthreads();
    }
    if (ty == 0 && c < p.cols) {
        const float4 t = acc[0][tx];
        if (!gate) {
            *reinterpret_cast<float4*>((j == 0 ? p.dw_pre : p.dw_post) + c) = t;
        } else if (p.dgate32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.dgate) + (int64_t)(j - 2) * p.ld_dgate + c) = t;
        } else {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dgate) + (int64_t)(j - 2) * p.ld_dgate + c) =
                make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
        }
    }
}

template <int NV, bool MULTI, bool GACC>
hipError_t launch_types(const NormBwdArgs& p, const NormBwdPlan& pl, hipStream_t st) {
    const auto k = p.res32 ? (p.dy32 ? k_block_norm_bwd<NV, true, true, MULTI, GACC>
                                     : k_block_norm_bwd<NV, true, false, MULTI, GACC>)
                           : (p.dy32 ? k_block_norm_bwd<NV, false, true, MULTI, GACC>
                                     : k_block_norm_bwd<NV, false, false, MULTI, GACC>);
    hipLaunchKernelGGL(k, dim3((unsigned)pl.slots), dim3(MULTI ? 64 * pl.wpr : 64 * kWaves), 0, st, p, pl);
    return hipGetLastError();
}

template <int NV>
hipError_t launch_nv(const NormBwdArgs& p, const NormBwdPlan& pl, hipStream_t st) {
    if constexpr (NV <= 2) {
        if (pl.wpr == 1)
            return pl.grouped ? launch_types<NV, false, true>(p, pl, st) : launch_types<NV, false, false>(p, pl, st);
    }
    return pl.grouped ? launch_types<NV, true, true>(p, pl, st) : launch_types<NV, true, false>(p, pl, st);
}

}  // namespace

NormBwdPlan plan_block_norm_bwd(int64_t rows, int64_t cols, int64_t rows_per_gate, bool dw_pre, bool dw_post,
                                bool dgate) {
    NormBwdPlan pl{};
    // two chunks per lane where there are rows enough to walk (4096x2560, one
    // and two chunks: 44.6 and 39.8 us with the reduction; 16384x2048: 130 and
    // 132); one where every row can have a workgroup and latency counts
    row_split(cols, rows <= kSlots ? 1 : 2, &pl.wpr, &pl.nv);
    pl.grouped = dgate && rows_per_gate > 1;
    pl.unit_rows = pl.grouped ? rows_per_gate : (rows > 0 ? rows : 1);
    const int64_t groups = (rows + pl.unit_rows - 1) / pl.unit_rows;
    const int64_t longest = rows < pl.unit_rows ? rows : pl.unit_rows;
    // gate rows of few rows go to single waves, whole
    pl.by_wave = pl.wpr == 1 && pl.grouped && rows_per_gate < 64;
    int64_t splits = groups > 0 && !pl.by_wave ? kSlots / groups : 1;
    if (splits < 1) splits = 1;
    if (splits > longest) splits = longest > 0 ? longest : 1;
    pl.chunk = (longest + splits - 1) / splits;
    if (pl.chunk < 1) pl.chunk = 1;
    pl.splits = (longest + pl.chunk - 1) / pl.chunk;
    if (pl.splits < 1) pl.splits = 1;
    pl.units = groups * pl.splits;
    const int64_t want = pl.by_wave ? (pl.units + kWaves - 1) / kWaves : pl.units;
    pl.slots = (int32_t)(want < kSlots ? want : kSlots);
    pl.groups = groups;
    size_t f = 0;
    pl.off_pre = f;
    if (dw_pre) f += (size_t)pl.slots * cols;
    pl.off_post = f;
    if (dw_post) f += (size_t)pl.slots * cols;
    pl.off_gate = f;
    if (pl.grouped && pl.splits > 1) f += (size_t)pl.units * cols;
    pl.ws_floats = f;
    return pl;
}

hipError_t launch_block_norm_bwd(const NormBwdArgs& p, float* ws, hipStream_t st) {
    NormBwdPlan pl = plan_block_norm_bwd(p.rows, p.cols, p.rows_per_gate, p.dw_pre, p.dw_post, p.dgate);
    pl.ws_pre = ws + pl.off_pre;
    pl.ws_post = ws + pl.off_post;
    pl.ws_gate = ws + pl.off_gate;
    hipError_t e = hipSuccess;
    if (p.rows > 0) {
        switch (pl.nv) {
            case 1: e = launch_nv<1>(p, pl, st); break;
            case 2: e = launch_nv<2>(p, pl, st); break;
            case 3: e = launch_nv<3>(p, pl, st); break;
            case 4: e = launch_nv<4>(p, pl, st); break;
            default: e = launch_nv<kMaxNv>(p, pl, st); break;
        }
        if (e != hipSuccess) return e;
    }
    const bool gate = p.rows > 0 && pl.grouped && pl.splits > 1;
    if (!p.dw_pre && !p.dw_post && !gate) return e;
    hipLaunchKernelGGL(k_col_reduce, dim3((unsigned)((p.cols + kRedCols - 1) / kRedCols),
                                          (unsigned)(2 + (gate ? pl.groups : 0))),
                       dim3(1024), 0, st, p, pl);
    return hipGetLastError();
}

}  // namespace fp8bs
