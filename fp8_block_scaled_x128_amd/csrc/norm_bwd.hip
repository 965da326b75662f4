// Gradient of the block norm (norm.hip) from the saved h and x.  The norms'
// factors are formed again: a sum of squares beside the sums that the
// gradient needs anyway.
//
//   hh = h r;  g = dy w_pre;  dH = dh + r (g - hh mean(g hh));  dres = dH
//   dw_pre = sum_rows dy hh
//   xh = x r';  dn = scale gate dH;  dgate = sum scale dH xh w_post
//   dw_post = sum_rows dn xh;  dx = r' (dn w_post - xh mean(dn w_post xh))
//
// HBM-bound.  A workgroup walks units of rows that share a gate row; its column
// sums of dw_pre and dw_post stay in registers over all its rows and leave one
// partial row each, which k_col_reduce adds in a fixed order (every 128th row,
// then a tree; no atomics: the same bits every time).
//
// Measured: 4096x2560 with an fp32 dy, 147 MB, 31 us (4.7 TB/s) and 4.5 us
// for the column sums; 16384x2048 over an fp32 stream with the gradient of a
// gate per sequence, 604 MB, 127.5 us (4.7 TB/s) and 5.3 us; 131072x128 40 us
// in all.  Without the next row in flight and with conversions between the
// loads the first two ran 65 and 143 us.
#include "norm_common.h"

namespace fp8bs {
namespace {

// Waves of a workgroup whose rows need one wave each: a gradient summed over gate
// rows has no registers for two workgroups of eight on a compute unit, three of
// four fit (28800x128 with a gate per 48 rows 24.2 -> 19.4 us); without it four
// cost more (32768x512 41.0 -> 39.2 with eight).
constexpr int row_waves(bool gate_sum) { return gate_sum ? 4 : 8; }

// Sums over the waves (rows that one wave holds), added in wave order: thread t
// returns those of columns 2 t and 2 t + 1, from the sums that lanes 0 .. LPR -
// 1 of each wave hold.
template <int LPR, int WAVES>
__device__ __forceinline__ float2 column_sums(const float (&a)[8], float (*comb)[512], int wave) {
    const int lane = threadIdx.x & 63, t = threadIdx.x & (4 * LPR - 1);
    __syncthreads();                                // the last call's sums have been read
    if (lane < LPR) {
        float4* s = reinterpret_cast<float4*>(&comb[wave][8 * lane]);
        s[0] = make_float4(a[0], a[1], a[2], a[3]);
        s[1] = make_float4(a[4], a[5], a[6], a[7]);
    }
    __syncthreads();
    float2 v = *reinterpret_cast<const float2*>(&comb[0][2 * t]);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
        const float2 u = *reinterpret_cast<const float2*>(&comb[w][2 * t]);
        v.x += u.x;
        v.y += u.y;
    }
    return v;
}
// Adds the sums of a wave's rows.
template <int LPR>
__device__ __forceinline__ void add_rows(float (&a)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = LPR == 16 ? rows_sum(a[e]) : LPR == 32 ? halves_sum(a[e]) : a[e];
}

// Adds eight values to a lane's sums in LDS.
__device__ __forceinline__ void add_lds(float4* a, const float v[8]) {
    float4* b = a + 64 * kMaxRowWaves;
    const float4 u = *a, w = *b;
    *a = make_float4(u.x + v[0], u.y + v[1], u.z + v[2], u.w + v[3]);
    *b = make_float4(w.x + v[4], w.y + v[5], w.z + v[6], w.w + v[7]);
}

// A row's weights as loaded, and their values (`kind` 0: bf16, 1: fp32, 2:
// none, all 1).
template <int NV>
struct Weights {
    uint4 r[NV][2];
    __device__ __forceinline__ void load(const void* p, bool f32, int tid, int step, int nc) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t c = min(tid + i * step, nc - 1);
            if (f32) {
                const uint4* f = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + c * 32u);
                r[i][0] = f[0];
                r[i][1] = f[1];
            } else {
                r[i][0] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + c * 16u);
            }
        }
    }
    __device__ __forceinline__ void get(int i, int kind, float v[8]) const {
        if (kind == 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 1.0f;
        } else if (kind == 1) {
            const uint4 a = r[i][0], b = r[i][1];
            v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
            v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
            v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
            v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
        } else {
            unpack8(r[i][0], v);
        }
    }
};

// What there is of a gate: none; a gradient per row (or none wanted); a
// gradient summed over the rows of a gate row.
enum { kGateNone, kGateRow, kGateSum };

// Waves per SIMD that the registers have to leave room for: what the plan below
// counts on per compute unit.  Rows of one wave: three workgroups of four waves
// with gate sums, two of eight without a gate.  Rows of several with one chunk
// per lane and no gate: ten waves in two workgroups of five, which three waves
// per SIMD do not hold (4096x2560, all fp32: 48.4 us, 54.2 with three).
constexpr int min_waves(int nv, int lpr, bool res32, bool dy32, int gate) {
    if (lpr == kMulti) return nv == 1 && gate == kGateNone ? 4 : 2;
    if (lpr == 64 && gate == kGateSum) return 3;
    return gate == kGateNone && !res32 && !(dy32 && lpr < 64) ? 4 : 2;
}

// One row as loaded.
template <int NV, bool RES32, bool DY32, int GATE>
struct RowIn {
    Raw8<RES32> dh[NV], h[NV];
    Raw8<DY32> dy[NV];
    static constexpr bool GATE_IN = GATE == kGateRow || (GATE == kGateSum && NV > 2);     // the gate comes with the row
    Raw8<false> x[NV], gate[GATE_IN ? NV : 1];
    __device__ __forceinline__ void load(const NormBwdArgs& p, int64_t row, int tid, int step, int nc) {
        const void* h_row = row_ptr<RES32>(p.h, row, p.ld_h);
        const void* dy_row = row_ptr<DY32>(p.dy, row, p.ld_dy);
        const void* dh_row = row_ptr<RES32>(p.dh, row, p.ld_dh);
        const void* x_row = row_ptr<false>(p.x, row, p.ld_x);
        if (p.w_pre) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) {
                    h[i].load(h_row, c);
                    dy[i].load(dy_row, c);
                }
            }
        }
        if (p.x) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) x[i].load(x_row, c);
            }
        }
        if (p.dh) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) dh[i].load(dh_row, c);
            }
        }
        if (GATE_IN) {
            const uint16_t* g_row = row_ptr<false>(p.gate, (int64_t)((uint32_t)row / (uint32_t)p.rows_per_gate), p.ld_gate);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                if (i < kSure<NV> || c < nc) gate[GATE_IN ? i : 0].load_shared(g_row, c);
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            dh[i].zero(); h[i].zero(); dy[i].zero(); x[i].zero(); gate[GATE_IN ? i : 0].zero();
        }
    }
};

// LPR lanes have a row; kMulti: a workgroup has one row at a time.
//
// The next row is loaded while this one is reduced and stored, as far as the
// registers go (AHEAD).  Loads return in order, so a weight load from the L2
// behind the next row's loads would wait for them: up to two chunks per lane
// the weights stay in registers (KEEP), above that each row's are loaded ahead
// of the next row's data.
// Column sums are in registers too up to two chunks per lane; above that (2048x
// 10240 with register sums: 99 us, 71 with both launches now) each lane keeps
// its columns' sums in LDS, 8 bytes a column and weight (halves of a chunk 16
// bytes apart from lane to lane: no bank conflicts).  Rows of more than 8192
// columns spill all the same, since a row's packed weights live from before its
// loads to its end: with three chunks per lane 5 (all bf16, no gate) to 115
// registers, with four 77 to 273 (2032x16384: 3.0 TB/s, 2048x10240 3.9).
template <int NV, bool RES32, bool DY32, int LPR, int GATE>
__global__ void __launch_bounds__(64 * (LPR == kMulti ? kMaxRowWaves : row_waves(GATE == kGateSum)),
                                  min_waves(NV, LPR, RES32, DY32, GATE)) k_block_norm_bwd(NormBwdArgs p, NormBwdPlan pl) {
    constexpr bool MULTI = LPR == kMulti, SHARED = LPR == 16 || LPR == 32;     // SHARED: a wave has several rows
    constexpr bool GACC = GATE == kGateSum;
    constexpr int WAVES = row_waves(GACC);          // of a workgroup whose rows need one wave each
    constexpr bool KEEP = NV <= 2;
    constexpr bool AHEAD = NV <= 2 || (NV == 3 && GATE == kGateNone);
    constexpr int KEPT = KEEP ? NV : 1;
    __shared__ float lds[2][kMaxRowWaves][4];
    __shared__ __align__(16) float comb[MULTI ? 1 : WAVES][512];
    __shared__ float4 lacc[KEEP ? 1 : NV * 4][KEEP ? 1 : 64 * kMaxRowWaves];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wpr = pl.wpr;
    const int tid = MULTI ? threadIdx.x : threadIdx.x % (MULTI ? 64 : LPR);
    const int sub = SHARED ? (threadIdx.x & 63) / (MULTI ? 64 : LPR) : 0;
    const int nc = p.cols >> 3, step = MULTI ? wpr * 64 : 64;
    const float inv_n = 1.0f / (float)p.cols;
    int turn = 0;
    float awpre[KEPT][8], awpost[KEPT][8], agate[GACC ? NV : 1][8];
    Weights<KEEP ? 1 : NV> rpre, rpost;                 // as loaded, for !KEEP
    float wpre[KEPT][8], wpost[KEPT][8], wgate[8];
    float kgate[GACC && KEEP ? NV : 1][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) wgate[e] = 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = min(tid + i * step, nc - 1);      // past the row: dy, dh and x are 0
        if (KEEP) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                awpre[i % KEPT][e] = awpost[i % KEPT][e] = 0.0f;
                wpre[i % KEPT][e] = wpost[i % KEPT][e] = 1.0f;
            }
            if (p.w_pre) load8_shared(p.w_pre, c, p.w32, wpre[i % KEPT]);
            if (p.w_post) load8_shared(p.w_post, c, p.w32, wpost[i % KEPT]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) lacc[(i * 4 + j) % (KEEP ? 1 : NV * 4)][tid] = make_float4(0, 0, 0, 0);
        }
    }
    // units by workgroup, its waves taking rows in turn; or (short gate rows)
    // by wave
    const bool by_wave = !MULTI && pl.by_wave;
    const int64_t u0 = by_wave ? (int64_t)blockIdx.x * WAVES + wave : blockIdx.x;
    const int64_t ustep = by_wave ? (int64_t)gridDim.x * WAVES : gridDim.x;
    // a unit's rows: a run of a gate row's rows, or every splits-th of all
    // rows, as many at a time as the workgroup (or wave) holds
    constexpr int kWaveRows = MULTI ? 1 : 64 / (MULTI ? 64 : LPR);
    const int at_once = MULTI ? 1 : by_wave ? kWaveRows : WAVES * kWaveRows;
    const int64_t rstep = GACC ? at_once : pl.splits * at_once;
    for (int64_t u = u0; u < pl.units; u += ustep) {
        const int64_t g = u / pl.splits;
        const int64_t s = u - g * pl.splits;
        const int64_t r0 = g * pl.unit_rows + s * (GACC ? pl.chunk : at_once) + (MULTI || by_wave ? 0 : wave * kWaveRows);
        const int64_t r1 = min(min((g + 1) * pl.unit_rows, GACC ? g * pl.unit_rows + (s + 1) * pl.chunk : p.rows), p.rows);
        // chunks of this lane's row: none past the last row (the lane stays
        // for the reductions)
        auto chunks = [&](int64_t row) { return !SHARED || row < r1 ? nc : 0; };
        if (GACC) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = min(tid + i * step, nc - 1);
                if (KEEP) load8_shared(row_ptr<false>(p.gate, g, p.ld_gate), c, false, kgate[GACC && KEEP ? i : 0]);
#pragma unroll
                for (int e = 0; e < 8; ++e) agate[GACC ? i : 0][e] = 0.0f;
            }
        }
        RowIn<NV, RES32, DY32, GATE> in, ahead;
        in.zero();
        if (AHEAD) {
            ahead.zero();
            if (r0 < r1) ahead.load(p, r0 + sub, tid, step, chunks(r0 + sub));
        }
        for (int64_t row0 = r0; row0 < r1; row0 += rstep) {
            const int64_t row = row0 + sub;
            const int ncr = chunks(row);
            // a lane whose row is past the last keeps zeros
            if (AHEAD) in = ahead;
            if (!KEEP) {
                if (p.w_pre) rpre.load(p.w_pre, p.w32, tid, step, nc);
                if (p.w_post) rpost.load(p.w_post, p.w32, tid, step, nc);
            }
            if (!AHEAD) {
                in.load(p, row, tid, step, ncr);
            } else if (row0 + rstep < r1) {
                if (SHARED) ahead.zero();
                ahead.load(p, row + rstep, tid, step, chunks(row + rstep));
            }
            float sums[3] = {0.0f, 0.0f, 0.0f};     // sum h^2, sum dy w_pre h, sum x^2
            if (p.w_pre) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float h[8], dy[8];
                    if (!KEEP) rpre.get(KEEP ? 0 : i, p.w32, wpre[i % KEPT]);
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
            row_sums<LPR>(sums, wpr, lds, turn);
            float means[2] = {sums[0], sums[2]};
            const auto value = [&](int k, int i, float v[8]) {
                if (k == 0) { auto t = in.h[i]; t.forget(); t.get(v); }
                else { auto t = in.x[i]; t.forget(); t.get(v); }
            };
            row_means<LPR, NV>(means, value, inv_n, p.eps, wpr, lds, turn);
#pragma unroll
            for (int i = 0; i < NV; ++i) { in.h[i].forget(); in.dy[i].forget(); in.x[i].forget(); }
            float dh[NV][8];
#pragma unroll
            for (int i = 0; i < NV; ++i) in.dh[i].get(dh[i]);
            if (p.w_pre) {
                const float r = inv_sqrt(means[0]);
                const float m = sums[1] * inv_n * r * r;        // mean(g hh) r: times h, hh mean(g hh)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float h[8], dy[8];
                    if (!KEEP) rpre.get(KEEP ? 0 : i, p.w32, wpre[i % KEPT]);
                    in.h[i].get(h);
                    in.dy[i].get(dy);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (KEEP) awpre[i % KEPT][e] = __builtin_fmaf(dy[e] * r, h[e], awpre[i % KEPT][e]);
                        dh[i][e] = __builtin_fmaf(r, __builtin_fmaf(-m, h[e], dy[e] * wpre[i % KEPT][e]), dh[i][e]);
                        h[e] *= dy[e] * r;
                    }
                    if (!KEEP) add_lds(&lacc[KEEP ? 0 : i * 4][tid], h);
                }
            }
            if (p.dres) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = tid + i * step;
                    if (i < kSure<NV> || c < ncr) store8<RES32>(row_ptr<RES32>(p.dres, row, p.ld_dres), c, dh[i]);
                }
            }
            if (!p.x) continue;
            const float rx = p.w_post ? inv_sqrt(means[1]) : 1.0f;
            float dot[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float dg[8], x[8], aw[8];
                in.x[i].get(x);
                if (!KEEP) rpost.get(KEEP ? 0 : i, p.w_post ? p.w32 : 2, wpost[i % KEPT]);
                if (GACC && KEEP) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) wgate[e] = kgate[GACC && KEEP ? i : 0][e];
                } else if (GATE != kGateNone) {
                    in.gate[GATE == kGateNone || (GACC && KEEP) ? 0 : i].get(wgate);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float dn = dh[i][e] * p.scale;
                    const float xh = x[e] * rx;
                    if (GATE != kGateNone) {
                        dg[e] = dn * (xh * wpost[i % KEPT][e]);
                        if (GACC) agate[GACC ? i : 0][e] += dg[e];
                        dn *= wgate[e];
                    }
                    if (KEEP) awpost[i % KEPT][e] = __builtin_fmaf(dn, xh, awpost[i % KEPT][e]);
                    aw[e] = dn * xh;
                    dn *= wpost[i % KEPT][e];
                    dot[0] = __builtin_fmaf(dn, xh, dot[0]);
                    dh[i][e] = dn;                      // the gradient at xh from here on
                }
                if (!KEEP) add_lds(&lacc[KEEP ? 0 : i * 4 + 2][tid], aw);
                if (GATE == kGateRow && p.dgate && (i < kSure<NV> || tid + i * step < ncr)) {
                    if (p.dgate32) store8<true>(row_ptr<true>(p.dgate, row, p.ld_dgate), tid + i * step, dg);
                    else store8<false>(row_ptr<false>(p.dgate, row, p.ld_dgate), tid + i * step, dg);
                }
            }
            if (!p.dx) continue;
            float m = 0.0f;
            if (p.w_post) {
                row_sums<LPR>(dot, wpr, lds, turn);
#pragma unroll
                for (int i = 0; i < NV; ++i) in.x[i].forget();
                m = dot[0] * inv_n * rx * rx;           // mean(g xh) r': times x
                // of rows with very large values the square of the factor would
                // underflow: a power of two goes from x to it
                if (__builtin_expect(__builtin_amdgcn_ballot_w64(rx < 0x1p-32f) != 0, 0)) {
                    const bool large = rx < 0x1p-32f;
                    m = dot[0] * inv_n * rx * (large ? rx * 0x1p64f : rx);
#pragma unroll
                    for (int i = 0; i < NV; ++i) in.x[i].scale(large ? 0x1p-64f : 1.0f);
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * step;
                float d[8], x[8];
                in.x[i].get(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = __builtin_fmaf(-m, x[e], dh[i][e] * rx);
                if (i < kSure<NV> || c < ncr) store8<false>(row_ptr<false>(p.dx, row, p.ld_dx), c, d);
            }
        }
        if (GACC) {
            void* dst = pl.splits > 1 ? (void*)row_ptr<true>(pl.ws_gate, u, p.cols)
                        : p.dgate32   ? (void*)row_ptr<true>(p.dgate, g, p.ld_dgate)
                                      : (void*)row_ptr<false>(p.dgate, g, p.ld_dgate);
            const bool f32 = pl.splits > 1 || p.dgate32;
            if (!MULTI) add_rows<LPR>(agate[0]);
            if (!MULTI && !by_wave) {
                const float2 v = column_sums<MULTI ? 64 : LPR, WAVES>(agate[0], comb, wave);
                if (2 * (int)threadIdx.x < p.cols) {
                    if (f32) static_cast<float2*>(dst)[threadIdx.x] = v;
                    else static_cast<uint32_t*>(dst)[threadIdx.x] = pack_bf16x2(v.x, v.y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = tid + i * step;
                    if ((i >= kSure<NV> && c >= nc) || sub > 0) continue;
                    if (f32) store8<true>(dst, c, agate[GACC ? i : 0]);
                    else store8<false>(dst, c, agate[GACC ? i : 0]);
                }
            }
        }
    }
    if (!MULTI) {
        add_rows<LPR>(awpre[0]);
        add_rows<LPR>(awpost[0]);
        const int64_t at = (int64_t)blockIdx.x * p.cols;
        if (p.dw_pre) {
            const float2 v = column_sums<MULTI ? 64 : LPR, WAVES>(awpre[0], comb, wave);
            if (2 * (int)threadIdx.x < p.cols) reinterpret_cast<float2*>(pl.ws_pre + at)[threadIdx.x] = v;
        }
        if (p.dw_post) {
            const float2 v = column_sums<MULTI ? 64 : LPR, WAVES>(awpost[0], comb, wave);
            if (2 * (int)threadIdx.x < p.cols) reinterpret_cast<float2*>(pl.ws_post + at)[threadIdx.x] = v;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * step;
        if (i >= kSure<NV> && c >= nc) continue;
        if (KEEP) {
            if (p.dw_pre) store8<true>(row_ptr<true>(pl.ws_pre, blockIdx.x, p.cols), c, awpre[i % KEPT]);
            if (p.dw_post) store8<true>(row_ptr<true>(pl.ws_post, blockIdx.x, p.cols), c, awpost[i % KEPT]);
        } else {
            const float4* a = &lacc[KEEP ? 0 : i * 4][tid];
            constexpr int kRow = KEEP ? 0 : 64 * kMaxRowWaves;
            float4* pre = reinterpret_cast<float4*>(pl.ws_pre + (int64_t)blockIdx.x * p.cols + 8 * c);
            float4* post = reinterpret_cast<float4*>(pl.ws_post + (int64_t)blockIdx.x * p.cols + 8 * c);
            if (p.dw_pre) { pre[0] = a[0]; pre[1] = a[kRow]; }
            if (p.dw_post) { post[0] = a[2 * kRow]; post[1] = a[3 * kRow]; }
        }
    }
}

// Column sums of partial rows.  Jobs 0 and 1 (dw_pre, dw_post) add the
// workgroups' rows, job 2 + g (dgate row g) the rows of its units: a workgroup
// takes 32 columns, its 128 row lanes add every 128th row and meet in LDS in a
// fixed order.
__device__ __forceinline__ void store_dgate(const NormBwdArgs& p, int64_t g, int c, const float4 t) {
    if (p.dgate32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.dgate) + g * p.ld_dgate + c) = t;
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dgate) + g * p.ld_dgate + c) =
            make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
}

constexpr int kRedCols = 32, kRedRows = 128, kRedThreads = kRedCols / 4 * kRedRows;
__global__ void __launch_bounds__(kRedThreads) k_col_reduce(NormBwdArgs p, NormBwdPlan pl) {
    __shared__ float4 acc[kRedRows][kRedCols / 4];
    const int tx = threadIdx.x % (kRedCols / 4), ty = threadIdx.x / (kRedCols / 4);
    const int c = blockIdx.x * kRedCols + 4 * tx;
    const int j = blockIdx.y;
    const float* src = j == 0 ? pl.ws_pre : j == 1 ? pl.ws_post : pl.ws_gate + (int64_t)(j - 2) * pl.splits * p.cols;
    const int64_t n = j >= 2 ? pl.splits : pl.slots;
    if ((j == 0 && !p.dw_pre) || (j == 1 && !p.dw_post)) return;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < p.cols) {
#pragma unroll 4
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
        if (j < 2) *reinterpret_cast<float4*>((j == 0 ? p.dw_pre : p.dw_post) + c) = t;
        else store_dgate(p, j - 2, c, t);
    }
}

// Gate rows of few units (at most kFewUnits): a thread adds four columns of
// one.  (8192x2048 with a gate row per 33 rows, two units each: the gradient
// took 99 us with a workgroup per 32 columns of every gate row, 52 with this.)
constexpr int kFewUnits = 32;
__global__ void __launch_bounds__(256) k_gate_reduce(NormBwdArgs p, NormBwdPlan pl) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = p.cols >> 2;
    if (i >= pl.groups * per) return;
    const int64_t g = i / per;
    const int c = (int)(i - g * per) * 4;
    const float* src = pl.ws_gate + g * pl.splits * p.cols + c;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int64_t r = 0; r < pl.splits; ++r) {
        const float4 v = *reinterpret_cast<const float4*>(src + r * p.cols);
        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
    store_dgate(p, g, c, a);
}

template <int NV, int LPR, int GATE>
hipError_t launch_types(const NormBwdArgs& p, const NormBwdPlan& pl, hipStream_t st) {
    const auto k = p.res32 ? (p.dy32 ? k_block_norm_bwd<NV, true, true, LPR, GATE>
                                     : k_block_norm_bwd<NV, true, false, LPR, GATE>)
                           : (p.dy32 ? k_block_norm_bwd<NV, false, true, LPR, GATE>
                                     : k_block_norm_bwd<NV, false, false, LPR, GATE>);
    hipLaunchKernelGGL(k, dim3((unsigned)pl.slots), dim3(64 * (LPR == kMulti ? pl.wpr : row_waves(GATE == kGateSum))), 0, st, p, pl);
    return hipGetLastError();
}

template <int NV, int LPR>
hipError_t launch_gate(const NormBwdArgs& p, const NormBwdPlan& pl, hipStream_t st) {
    return pl.grouped ? launch_types<NV, LPR, kGateSum>(p, pl, st)
           : p.gate   ? launch_types<NV, LPR, kGateRow>(p, pl, st)
                      : launch_types<NV, LPR, kGateNone>(p, pl, st);
}

hipError_t launch_rows(const NormBwdArgs& p, const NormBwdPlan& pl, hipStream_t st) {
    if (pl.wpr == 1) {
        switch (row_lanes(p.cols)) {
            case 16: return launch_gate<1, 16>(p, pl, st);
            case 32: return launch_gate<1, 32>(p, pl, st);
            default: return launch_gate<1, 64>(p, pl, st);
        }
    }
    switch (pl.nv) {
        case 1: return launch_gate<1, kMulti>(p, pl, st);
        case 2: return launch_gate<2, kMulti>(p, pl, st);
        case 3: return launch_gate<3, kMulti>(p, pl, st);
        default: return launch_gate<4, kMulti>(p, pl, st);
    }
}

}  // namespace

NormBwdPlan plan_block_norm_bwd(int64_t rows, int64_t cols, int64_t rows_per_gate, bool dw_pre, bool dw_post,
                                bool dgate, bool res32, bool dy32) {
    NormBwdPlan pl{};
    row_split(cols, &pl.wpr, &pl.nv);
    pl.grouped = dgate && rows_per_gate > 1;
    pl.unit_rows = pl.grouped ? rows_per_gate : (rows > 0 ? rows : 1);
    const int64_t groups = (rows + pl.unit_rows - 1) / pl.unit_rows;
    const int64_t longest = rows < pl.unit_rows ? rows : pl.unit_rows;
    // Workgroups at most: about 2560 waves of one chunk per lane, equally many
    // per compute unit (4096x2560, five waves: 256 / 512 / 768 workgroups 40.7 /
    // 32.9 / 39.9 us; 16384x768, two waves: 512 / 1024 61.4 / 41.1; 4096x5120,
    // five waves with two chunks: 256 / 512 56.0 / 64.5; 16384x2048 gated, four
    // waves: 512 / 632 132 / 145).  Every workgroup more costs a row of partial
    // sums.  Rows of one wave or less: three workgroups of four waves per
    // compute unit with gate sums; else two of eight, or one where the
    // registers of fp32 rows leave room for no second (16384x128, fp32 stream:
    // 17.7 / 14.9 us, fp32 dy 16.1 / 12.8; 32768x512, fp32 stream 63.7 / 60.4,
    // fp32 dy, which leaves room, 45.6 / 46.5).
    const int waves = row_waves(pl.grouped);
    const bool single = res32 || (dy32 && row_lanes(cols) < 64);
    int64_t most = 2560 / (pl.wpr * pl.nv) / kCUs * kCUs;
    most = pl.wpr == 1 ? (pl.grouped ? 3 : single ? 1 : 2) * kCUs : most < kCUs ? kCUs : most > 4 * kCUs ? 4 * kCUs : most;
    // Many gate rows of few rows each go to single waves, whole: no barrier
    // and no sum over waves for each.  A wave walks its gate row in `passes`
    // alone, so few gate rows or long ones are faster by workgroup (us by wave
    // / by workgroup, 128 columns: 100 and 300 gate rows of 8 rows 8.4 / 7.7 and
    // 8.9 / 9.4; 600, 2100, 6000 of 16 13.1 / 12.3, 20.0 / 22.2, 34.6 / 42.1;
    // 1100 and 6000 of 32 22.7 / 20.7 and 60.7 / 65.4, of 48 28.6 / 24.6 and 98.2
    // / 96.0; 512 columns, a row per pass: 1100 of 4 and 8 16.7 / 17.1 and 23.7 /
    // 21.3, 6000 36.8 / 43.5 and 68.8 / 69.2).
    const int64_t wave_rows = 64 / row_lanes(cols), passes = (pl.unit_rows + wave_rows - 1) / wave_rows;
    pl.by_wave = pl.wpr == 1 && pl.grouped && passes <= 8 && groups >= 256 * passes;
    int64_t splits = groups > 0 && !pl.by_wave ? most / groups : 1;
    if (splits < 1) splits = 1;
    const int64_t at_once = pl.wpr == 1 && !pl.by_wave ? waves * wave_rows : 1;
    if (splits > (longest + at_once - 1) / at_once) splits = (longest + at_once - 1) / at_once;
    if (splits < 1) splits = 1;
    pl.splits = splits;
    pl.chunk = (longest + splits - 1) / splits;
    pl.units = groups * pl.splits;
    const int64_t want = pl.by_wave ? (pl.units + waves - 1) / waves : pl.units;
    pl.slots = (int32_t)(want < most ? want : most);
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
    NormBwdPlan pl = plan_block_norm_bwd(p.rows, p.cols, p.rows_per_gate, p.dw_pre, p.dw_post, p.dgate, p.res32,
                                         p.dy32);
    pl.ws_pre = ws + pl.off_pre;
    pl.ws_post = ws + pl.off_post;
    pl.ws_gate = ws + pl.off_gate;
    hipError_t e = hipSuccess;
    if (p.rows > 0) {
        e = launch_rows(p, pl, st);
        if (e != hipSuccess) return e;
    }
    const bool gate = p.rows > 0 && pl.grouped && pl.splits > 1, few = pl.splits <= kFewUnits;
    if (gate && few) {
        hipLaunchKernelGGL(k_gate_reduce, dim3((unsigned)((pl.groups * (p.cols / 4) + 255) / 256)), dim3(256), 0, st, p,
                           pl);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!p.dw_pre && !p.dw_post && (!gate || few)) return e;
    hipLaunchKernelGGL(k_col_reduce, dim3((unsigned)((p.cols + kRedCols - 1) / kRedCols),
                                          (unsigned)(2 + (gate && !few ? pl.groups : 0))),
                       dim3(kRedThreads), 0, st, p, pl);
    return hipGetLastError();
}

}  // namespace fp8bs
