// The norms around a block and what joins it to the residual stream, forward
// and backward.  With N(v; w) = v * rsqrt(mean(v^2) + eps) * w by rows:
//
//   h = residual + scale * gate * N(x; w_post)
//   y = N(h; w_pre), and y's 1x128 groups as E4M3 codes with S = max|y| / 448
//
// so the tensor that a linear layer's 1x128 quantizer would read (the "per-
// token" activations of "Unified FP8: Beyond Mixed Precision...", section
// "FP8 Quantization") is quantized where it is made.  Everything is
// HBM-bound: each input is read once, each output written once, and all that
// lies between stays in fp32 registers.
#include "device_common.h"
#include "internal.h"
#include "reduce.h"

namespace fp8bs {
namespace {

// Eight consecutive elements of a row, as fp32.  Streamed: an activation is
// read once here.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float v[8]) {
    if (F32) {
        const float* f = static_cast<const float*>(p) + i;
        const uint4 a = load_nt16(f), b = load_nt16(f + 4);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
        v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
        unpack8(load_nt16(static_cast<const uint16_t*>(p) + i), v);
    }
}
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

// Sums of K values over the wpr waves that share a row.  `buf` alternates
// between two LDS buffers from call to call: a wave can be at most one
// barrier behind, so the buffer it still reads is not the one being written.
constexpr int kMaxWaves = 16;
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int wpr, float (*lds)[kMaxWaves][4], int& turn) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = lanes_sum<64>(v[i]);
    if (wpr == 1) return;
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

// A row belongs to `wpr` waves; lane l of them holds the 8-column chunks l,
// l + 64 wpr, ...  With wpr == 1 a workgroup's waves have a row each.
template <int NV, bool RES32>
__global__ void __launch_bounds__(1024) k_block_norm(NormArgs p, int wpr) {
    __shared__ float lds[2][kMaxWaves][4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tid = wpr == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int per = wpr == 1 ? blockDim.x >> 6 : 1;   // rows a workgroup has at a time
    const int nc = p.cols >> 3, step = wpr * 64;
    const float inv_n = 1.0f / (float)p.cols;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * per + (wpr == 1 ? wave : 0); row < p.rows; row += (int64_t)gridDim.x * per) {
        float h[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * step;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
            if (c < nc && p.residual) load8<RES32>(p.residual, row * p.ld_r + 8 * c, h[i]);
        }
        if (p.x) {
            float x[NV][8];
            float ss[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
                if (c < nc) load8<false>(p.x, row * p.ld_x + 8 * c, x[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss[0] = __builtin_fmaf(x[i][e], x[i][e], ss[0]);
            }
            float r = p.scale;
            if (p.w_post) {
                row_sums(ss, wpr, lds, turn);
                r = 1.0f / sqrtf(__builtin_fmaf(ss[0], inv_n, p.eps));
            }
            const int64_t gate_row = p.gate ? (int64_t)((uint32_t)row / (uint32_t)p.rows_per_gate) * p.ld_gate : 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (c >= nc) continue;
                float w[8], g[8];
                if (p.w_post) load8_shared(p.w_post, 8 * c, p.w32, w);
                if (p.gate) load8_shared(p.gate, gate_row + 8 * c, false, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float n = x[i][e] * r;
                    if (p.w_post) n *= w[e] * p.scale;
                    if (p.gate) n *= g[e];
                    h[i][e] += n;
                }
            }
        }
        if (p.h) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (c < nc) store8<RES32>(p.h, row * p.ld_h + 8 * c, h[i]);
            }
        }
        if (!p.w_pre) continue;
        // y from the unrounded h: the bf16 rounding of the stored stream does not
        // enter y, its scales or its codes
        float ss[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ss[0] = __builtin_fmaf(h[i][e], h[i][e], ss[0]);
        }
        row_sums(ss, wpr, lds, turn);
        const float r = 1.0f / sqrtf(__builtin_fmaf(ss[0], inv_n, p.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * step;
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 0.0f;
            if (c < nc) load8_shared(p.w_pre, 8 * c, p.w32, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * r * w[e];
            if (p.y && c < nc) store8<false>(p.y, row * p.ld_y + 8 * c, h[i]);
            if (p.q) {
                // 16 lanes hold a 128-column group; lanes past the row hold zeros
                const float s = row16_max(absmax8(h[i])) / kE4M3Max;
                uint32_t w0, w1;
                encode8(h[i], s, w0, w1);
                if (c < nc) {
                    *reinterpret_cast<uint2*>(p.q + row * p.ld_q + 8 * c) = make_uint2(w0, w1);
                    if ((c & 15) == 0) p.s[row * p.ssr + (int64_t)(c >> 4) * p.ssg] = s;
                }
            }
        }
    }
}

// ------------------------------------------------------------- backward
// From the saved h and x (their norms' factors are formed again: a sum of
// squares beside the sums that the gradient needs anyway):
//
//   hh = h r;  g = dy w_pre;  dH = dh + r (g - hh mean(g hh))
//   dw_pre = sum_rows dy hh;  dres = dH
//   xh = x r';  dn = scale gate dH;  dgate = sum scale dH xh w_post
//   dw_post = sum_rows dn xh;  dx = r' (dn w_post - xh mean(dn w_post xh))
//
// Rows are dealt to slots (a workgroup, or with wpr == 1 a wave) in runs that
// stay inside one gate row; a slot keeps its column sums of dw_pre and dw_post
// in registers over all its rows and leaves one partial row of each, which
// k_col_reduce adds in slot order (no atomics: the same bits every time).
template <int NV, bool RES32, bool DY32>
__global__ void __launch_bounds__(1024) k_block_norm_bwd(NormBwdArgs p, NormBwdPlan pl) {
    __shared__ float lds[2][kMaxWaves][4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wpr = pl.wpr;
    const int tid = wpr == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int slot = wpr == 1 ? blockIdx.x * (blockDim.x >> 6) + wave : blockIdx.x;
    if (slot >= pl.slots) return;
    const int nc = p.cols >> 3, step = wpr * 64;
    const float inv_n = 1.0f / (float)p.cols;
    int turn = 0;
    float awpre[NV][8], awpost[NV][8], agate[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) awpre[i][e] = awpost[i][e] = 0.0f;
    }
    for (int64_t u = slot; u < pl.units; u += pl.slots) {
        const int64_t g = u / pl.splits;
        const int64_t r0 = g * pl.unit_rows + (u - g * pl.splits) * pl.chunk;
        const int64_t r1 = min(min(r0 + pl.chunk, (g + 1) * pl.unit_rows), p.rows);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) agate[i][e] = 0.0f;
        }
        for (int64_t row = r0; row < r1; ++row) {
            float dh[NV][8], x[NV][8];
            float sums[3] = {0.0f, 0.0f, 0.0f};     // sum h^2, sum dy w_pre h, sum x^2
            float h[NV][8], dy[NV][8];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
#pragma unroll
                for (int e = 0; e < 8; ++e) dh[i][e] = x[i][e] = h[i][e] = dy[i][e] = 0.0f;
                if (c >= nc) continue;
                if (p.dh) load8<RES32>(p.dh, row * p.ld_dh + 8 * c, dh[i]);
                if (p.w_pre) {
                    load8<RES32>(p.h, row * p.ld_h + 8 * c, h[i]);
                    load8<DY32>(p.dy, row * p.ld_dy + 8 * c, dy[i]);
                }
                if (p.x) load8<false>(p.x, row * p.ld_x + 8 * c, x[i]);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (c < nc && p.w_pre) {
                    float w[8];
                    load8_shared(p.w_pre, 8 * c, p.w32, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        sums[0] = __builtin_fmaf(h[i][e], h[i][e], sums[0]);
                        sums[1] = __builtin_fmaf(dy[i][e] * w[e], h[i][e], sums[1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sums[2] = __builtin_fmaf(x[i][e], x[i][e], sums[2]);
            }
            row_sums(sums, wpr, lds, turn);
            if (p.w_pre) {
                const float r = 1.0f / sqrtf(__builtin_fmaf(sums[0], inv_n, p.eps));
                const float m = sums[1] * inv_n * r * r;        // mean(g hh) r: times h, hh mean(g hh)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = tid + i * step;
                    if (c >= nc) continue;
                    float w[8];
                    load8_shared(p.w_pre, 8 * c, p.w32, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        awpre[i][e] = __builtin_fmaf(dy[i][e] * r, h[i][e], awpre[i][e]);
                        dh[i][e] = __builtin_fmaf(r, __builtin_fmaf(-m, h[i][e], dy[i][e] * w[e]), dh[i][e]);
                    }
                }
            }
            if (p.dres) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = tid + i * step;
                    if (c < nc) store8<RES32>(p.dres, row * p.ld_dres + 8 * c, dh[i]);
                }
            }
            if (!p.x) continue;
            const float rx = p.w_post ? 1.0f / sqrtf(__builtin_fmaf(sums[2], inv_n, p.eps)) : 1.0f;
            const int64_t gate_row = p.gate ? (int64_t)((uint32_t)row / (uint32_t)p.rows_per_gate) : 0;
            float dot[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (c >= nc) continue;
                float w[8], gt[8], dg[8];
                if (p.w_post) load8_shared(p.w_post, 8 * c, p.w32, w);
                if (p.gate) load8_shared(p.gate, gate_row * p.ld_gate + 8 * c, false, gt);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float dn = dh[i][e] * p.scale;
                    const float xh = x[i][e] * rx;
                    if (p.gate) {
                        dg[e] = dn * (p.w_post ? xh * w[e] : xh);
                        agate[i][e] += dg[e];
                        dn *= gt[e];
                    }
                    if (p.w_post) {
                        awpost[i][e] = __builtin_fmaf(dn, xh, awpost[i][e]);
                        dn *= w[e];
                        dot[0] = __builtin_fmaf(dn, xh, dot[0]);
                    }
                    dh[i][e] = dn;                      // the gradient at xh from here on
                }
                if (p.dgate && p.rows_per_gate == 1) {
                    if (p.dgate32) store8<true>(p.dgate, row * p.ld_dgate + 8 * c, dg);
                    else store8<false>(p.dgate, row * p.ld_dgate + 8 * c, dg);
                }
            }
            if (!p.dx && !p.w_post) continue;
            float m = 0.0f;
            if (p.w_post) {
                row_sums(dot, wpr, lds, turn);
                m = dot[0] * inv_n * rx * rx;           // mean(g xh) r': times x
            }
            if (p.dx) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = tid + i * step;
                    if (c >= nc) continue;
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] = __builtin_fmaf(-m, x[i][e], dh[i][e] * rx);
                    store8<false>(p.dx, row * p.ld_dx + 8 * c, d);
                }
            }
        }
        if (p.dgate && p.rows_per_gate > 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (c >= nc) continue;
                if (pl.splits > 1) store8<true>(pl.ws_gate, u * p.cols + 8 * c, agate[i]);
                else if (p.dgate32) store8<true>(p.dgate, g * p.ld_dgate + 8 * c, agate[i]);
                else store8<false>(p.dgate, g * p.ld_dgate + 8 * c, agate[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * step;
        if (c >= nc) continue;
        if (p.dw_pre) store8<true>(pl.ws_pre, (int64_t)slot * p.cols + 8 * c, awpre[i]);
        if (p.dw_post) store8<true>(pl.ws_post, (int64_t)slot * p.cols + 8 * c, awpost[i]);
    }
}

// Column sums of partial rows: output row g (grid z) of job 0 / 1 / 2
// (dw_pre, dw_post, dgate) is the sum of its n partial rows in order.  A
// workgroup takes 64 columns; its 64 row lanes add every 64th partial, then
// meet in LDS in a fixed order.
constexpr int kRedCols = 64, kRedRows = 64;
__global__ void __launch_bounds__(1024) k_col_reduce(NormBwdArgs p, NormBwdPlan pl) {
    __shared__ float4 acc[kRedRows][kRedCols / 4];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
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

// Waves per row and chunks per lane: the fewest chunks per lane that 16
// waves allow, in as few waves as then hold the row.
void row_split(int64_t cols, int* wpr, int* nv) {
    const int64_t chunks = cols / 8;
    int v = 1;
    while ((chunks + 64 * v - 1) / (64 * v) > kMaxWaves) v *= 2;
    *nv = v;
    *wpr = (int)((chunks + 64 * v - 1) / (64 * v));
}

constexpr int64_t kMaxBlocks = 1 << 20;     // a grid holds fewer than 2^32 threads

template <int NV>
hipError_t launch_norm_nv(const NormArgs& p, int wpr, hipStream_t st) {
    const dim3 block(wpr == 1 ? 256 : 64 * wpr);
    const int64_t blocks = wpr == 1 ? (p.rows + 3) / 4 : p.rows;
    const dim3 grid((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
    if (p.res32) hipLaunchKernelGGL((k_block_norm<NV, true>), grid, block, 0, st, p, wpr);
    else hipLaunchKernelGGL((k_block_norm<NV, false>), grid, block, 0, st, p, wpr);
    return hipGetLastError();
}

template <int NV>
hipError_t launch_bwd_nv(const NormBwdArgs& p, const NormBwdPlan& pl, hipStream_t st) {
    const dim3 block(pl.wpr == 1 ? 256 : 64 * pl.wpr);
    const dim3 grid((unsigned)(pl.wpr == 1 ? (pl.slots + 3) / 4 : pl.slots));
    if (p.res32 && p.dy32) hipLaunchKernelGGL((k_block_norm_bwd<NV, true, true>), grid, block, 0, st, p, pl);
    else if (p.res32) hipLaunchKernelGGL((k_block_norm_bwd<NV, true, false>), grid, block, 0, st, p, pl);
    else if (p.dy32) hipLaunchKernelGGL((k_block_norm_bwd<NV, false, true>), grid, block, 0, st, p, pl);
    else hipLaunchKernelGGL((k_block_norm_bwd<NV, false, false>), grid, block, 0, st, p, pl);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& p, hipStream_t st) {
    int wpr, nv;
    row_split(p.cols, &wpr, &nv);
    switch (nv) {
        case 1: return launch_norm_nv<1>(p, wpr, st);
        case 2: return launch_norm_nv<2>(p, wpr, st);
        default: return launch_norm_nv<4>(p, wpr, st);
    }
}

NormBwdPlan plan_block_norm_bwd(int64_t rows, int64_t cols, int64_t rows_per_gate, bool dw_pre, bool dw_post,
                                bool dgate) {
    NormBwdPlan pl{};
    row_split(cols, &pl.wpr, &pl.nv);
    // about 1024 slots: four workgroups a compute unit
    constexpr int64_t kSlots = 1024;
    const bool grouped = dgate && rows_per_gate > 1;
    pl.unit_rows = grouped ? rows_per_gate : (rows > 0 ? rows : 1);
    const int64_t groups = (rows + pl.unit_rows - 1) / pl.unit_rows;
    const int64_t longest = rows < pl.unit_rows ? rows : pl.unit_rows;
    int64_t splits = groups > 0 ? kSlots / groups : 1;
    if (splits < 1) splits = 1;
    if (splits > longest) splits = longest > 0 ? longest : 1;
    pl.chunk = (longest + splits - 1) / splits;
    if (pl.chunk < 1) pl.chunk = 1;
    pl.splits = (longest + pl.chunk - 1) / pl.chunk;
    if (pl.splits < 1) pl.splits = 1;
    pl.units = groups * pl.splits;
    pl.slots = (int32_t)(pl.units < kSlots ? pl.units : kSlots);
    pl.groups = groups;
    size_t f = 0;
    pl.off_pre = f;
    if (dw_pre) f += (size_t)pl.slots * cols;
    pl.off_post = f;
    if (dw_post) f += (size_t)pl.slots * cols;
    pl.off_gate = f;
    if (grouped && pl.splits > 1) f += (size_t)pl.units * cols;
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
            case 1: e = launch_bwd_nv<1>(p, pl, st); break;
            case 2: e = launch_bwd_nv<2>(p, pl, st); break;
            default: e = launch_bwd_nv<4>(p, pl, st); break;
        }
        if (e != hipSuccess) return e;
    }
    const bool gate = p.rows > 0 && p.dgate && p.rows_per_gate > 1 && pl.splits > 1;
    if (!p.dw_pre && !p.dw_post && !gate) return e;
    hipLaunchKernelGGL(k_col_reduce, dim3((unsigned)((p.cols + kRedCols - 1) / kRedCols),
                                          (unsigned)(2 + (gate ? pl.groups : 0))),
                       dim3(1024), 0, st, p, pl);
    return hipGetLastError();
}

}  // namespace fp8bs
