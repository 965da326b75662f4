// The router of a MoE layer: top-k selection, the expert-sorted row maps that
// the grouped GEMMs and the combine read, the balance and z losses, and the
// gradient of all of them at the logits (the routing that "Low Precision RL",
// section "2. Unified block-wise FP8 (DeepSeek-style)", runs its
// Qwen3-30B-A3B recipe with).
//
//   selected  the k largest logits, ties to the lower expert
//   lse_t     log sum_e exp z_te;  p_te = exp(z_te - lse_t)
//   w_tj      exp(z_j - m) / sum over the selected, or p of the selected
//   balance   E sum_e f_e P_e, f_e = counts_e / sum counts, P_e = mean_t p_te
//   z loss    mean_t lse_t^2
//
// 10.6 MB move for 16384 tokens of 128 experts, 2 us at the rate of a copy; what
// bounds the routing is the selection's rounds (820 vector instructions a
// wave, 5.5 us of issue) and the latency of two dependent launches, in the
// second of which each workgroup goes through 113 scalar branches (the steps of
// lanes_sum_mod on the number of experts) before its first barrier.  With more
// experts a round scans as many more values per lane, and the histograms that
// every placing workgroup adds grow with experts times tokens squared.
// Measured, top-8: 16384 tokens 9.4 us (selection) and 7.9 (placement), of 512
// experts 21.5 and 14; 32768 of 512 38.7 and 21.4; 32 tokens 5.8 in one launch;
// 262144 tokens 133 in three (72.6, 4.7, 55.4).  The gradient at 16384 tokens 7.1.
// A third launch that scanned the histograms made it 30.7 us, logits loaded one
// after the other 26, placement sums by LDS shuffles 21.
#include "route_common.h"

namespace fp8bs {
namespace {

// Selection.  L lanes hold a token's logits, lane l the experts l, l + L, ...
// Each of the k rounds takes the largest key among the lanes and, of equal
// keys, the lowest expert; lane j keeps slot j (and slot j + L).  The
// workgroup's 64 tokens leave in LDS, per expert, the mask of the tokens that
// chose it: the histogram is its population count, and a slot's rank among
// earlier tokens that of the bits below it, so the stable (expert, token)
// order needs no sort.  On return psum[0..E) holds the probability sums, and
// {sum of lse^2, routed tokens} are returned to every thread.
template <int L, int V, bool F32>
__device__ __forceinline__ float2 select_tokens(const RouteArgs& p, int64_t t0, unsigned long long* mask, float* psum) {
    constexpr int kGroups = kThreads / L;
    __shared__ float red[32];
    const int l = threadIdx.x % L, grp = threadIdx.x / L;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    float sums[2] = {0.0f, 0.0f};                   // lse^2, tokens: in lane 0 of a group
    for (int tt = grp; tt < kTok; tt += kGroups) {
        const int64_t t = t0 + tt;
        if (t0 + tt - grp % (64 / L) >= p.T) break;   // no lane of the wave has a token
        float z[V];
        load_logits<L, V, F32>(p.logits, min(t, p.T - 1) * p.ld, l, p.E, z);
        const bool have = t < p.T && (!p.mask || p.mask[t]);
        uint32_t left[V];
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // a mask, not a choice: no branch around each key
            left[i] = logit_key(z[i]) & ((have && l + i * L < p.E) ? 0xffffffffu : 0u);
            best = max(best, left[i]);
        }
        const uint32_t top = lanes_umax<L>(best);
        const bool live = top > kKeyNegInf;
        const float m = live ? key_logit(top) : 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float v = __builtin_amdgcn_exp2f((z[i] - m) * kLog2e);
            z[i] = left[i] ? v : 0.0f;              // from here on exp(z - m)
            sum += z[i];
        }
        sum = lanes_sum<L>(sum);
        uint32_t ksel[2] = {0, 0}, esel[2] = {0, 0};
        uint32_t mx = top;
        for (int j = 0; j < p.k; ++j) {
            if (j > 0) {
                best = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) best = max(best, left[i]);
                mx = lanes_umax<L>(best);
            }
            uint32_t at = 0x10000u;
#pragma unroll
            for (int i = V - 1; i >= 0; --i) at = left[i] == mx ? (uint32_t)(i * L) : at;
            at = lanes_umin<L>(at + l);
            const uint32_t mine = at - l;
#pragma unroll
            for (int i = 0; i < V; ++i) left[i] = mine == (uint32_t)(i * L) ? 0u : left[i];
            if (l == j) { ksel[0] = mx; esel[0] = at; }
            if (l + L == j) { ksel[1] = mx; esel[1] = at; }
        }
        float w[2], wsum = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w[u] = ksel[u] > kKeyNegInf ? __builtin_amdgcn_exp2f((key_logit(ksel[u]) - m) * kLog2e) : 0.0f;
            wsum += w[u];
        }
        const float norm = p.renorm ? lanes_sum<L>(wsum) : sum;
        const float lse = live ? m + logf(sum) : -INFINITY;
        if (t < p.T) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = l + u * L;
                if (j < p.k) {
                    const bool ok = ksel[u] > kKeyNegInf;
                    p.experts[t * p.k + j] = ok ? (int)esel[u] : -1;
                    p.weights[t * p.k + j] = ok ? w[u] / norm : 0.0f;
                    if (ok) atomicOr(&mask[esel[u]], 1ull << tt);
                }
            }
            if (l == 0) p.lse[t] = lse;
        }
        if (live) {
            const float inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(z[i], inv, acc[i]);
            if (l == 0) {
                sums[0] = __builtin_fmaf(lse, lse, sums[0]);
                sums[1] += 1.0f;
            }
        }
    }
    // the 64 / L groups of a wave in registers, waves w and w + 8, then those
    // in order
    const int wave = threadIdx.x >> 6;
    float* mine = psum + (wave & (kHalf - 1)) * (L * V) + l;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (L == 16) acc[i] = rows_sum(acc[i]);
    if (wave >= kHalf && (threadIdx.x & 63) < L) {
#pragma unroll
        for (int i = 0; i < V; ++i) mine[i * L] = acc[i];
    }
    __syncthreads();
    if (wave < kHalf && (threadIdx.x & 63) < L) {
#pragma unroll
        for (int i = 0; i < V; ++i) mine[i * L] += acc[i];
    }
    block_sums(sums, red);                          // its barrier covers psum and mask too
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kHalf; ++w) s += psum[w * (L * V) + e];
        psum[e] = s;                                // column e is this thread's alone
    }
    return make_float2(sums[0], sums[1]);
}

template <int L, int V, bool F32>
__global__ void __launch_bounds__(kThreads) k_route_one(RouteArgs p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    route_one(p, dyn, L * V * kHalf,
              [&](unsigned long long* mask, float* psum) { return select_tokens<L, V, F32>(p, 0, mask, psum); });
}

template <int L, int V, bool F32>
__global__ void __launch_bounds__(kThreads) k_route_select(RouteArgs p, RouteWs ws) {
    extern __shared__ __align__(16) unsigned char dyn[];
    route_select(p, ws, dyn, [&](unsigned long long* mask, float* psum) {
        return select_tokens<L, V, F32>(p, (int64_t)blockIdx.x * kTok, mask, psum);
    });
}

// Histogram bytes of 16 experts as 16-bit sums, two to a word: word 2 i + h
// holds experts 4 i + h and 4 i + h + 2.
__device__ __forceinline__ void add_bytes(uint32_t (&a)[8], const uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[2 * i] += w[i] & 0x00ff00ffu;
        a[2 * i + 1] += (w[i] >> 8) & 0x00ff00ffu;
    }
}

// Last launch: every workgroup adds the histograms of all workgroups and of
// those before it (32 KB from the L2 at 16384 tokens and 128 experts), scans
// the counts over the experts and places its tokens' rows; one more workgroup
// forms the counts, offsets and losses.  More than kDirect workgroups of
// tokens (SUPER) are first added up in runs of kRun by k_route_super, and a
// workgroup adds the runs and the histograms of its own run.  Sums of at most
// 512 x 64 fit 16 bits.
constexpr int kDirect = 512, kRun = 256;
template <bool SUPER>
__global__ void __launch_bounds__(kThreads) k_route_place(RouteArgs p, RouteWs ws, int nblk) {
    extern __shared__ __align__(16) unsigned char dyn[];
    const int epad = ws.epad, nch = epad >> 4;      // chunks of 16 experts: a power of two, at most 64
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(dyn);
    int* counts = reinterpret_cast<int*>(mask + epad);
    int* base = counts + epad;                      // [epad + 1], padded to 16 bytes
    int* earlier = base + epad + 4;                 // [epad] rows of workgroups before this one
    uint32_t* part = reinterpret_cast<uint32_t*>(earlier + epad);      // [8 waves][nch][16]
    // the workgroup without tokens goes first: it has the longest way
    const int blk = (int)blockIdx.x - 1;
    const int64_t t0 = (int64_t)blk * kTok;
    const bool tokens = blk >= 0;
    const int n = tokens ? (int)min((int64_t)kTok, p.T - t0) * p.k : 0;
    int es[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = threadIdx.x + u * kThreads;
        es[u] = i < n ? p.experts[t0 * p.k + i] : -1;
    }
    // the losses' probability sums, four experts per thread and every
    // (4096 / epad)-th workgroup's (or run's); the counts come later
    const int e4 = (threadIdx.x * 4) & (epad - 1), prows = kThreads * 4 / epad;
    float4 ps = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float s[3] = {0.0f, 0.0f, 0.0f};                // counts . probabilities, lse^2, tokens (at most 2^22: exact)
    if (!tokens) {
        const float* src = SUPER ? ws.run_psum : ws.psum;
        const int n = SUPER ? (nblk + kRun - 1) / kRun : nblk;
#pragma unroll 8
        for (int b = threadIdx.x * 4 / epad; b < n; b += prows) {
            const float4 v = *reinterpret_cast<const float4*>(src + (int64_t)b * epad + e4);
            ps.x += v.x; ps.y += v.y; ps.z += v.z; ps.w += v.w;
        }
        for (int b = threadIdx.x; b < nblk; b += kThreads) { s[1] += ws.lse2[b]; s[2] += (float)ws.live[b]; }
    }
    uint32_t tot[8], pre[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) tot[i] = pre[i] = 0;
    const int ch = threadIdx.x & (nch - 1), rows = kThreads / nch;
    const int b1 = SUPER ? max(blk, 0) : nblk, b0 = SUPER ? b1 & ~(kRun - 1) : 0;
    // two rows in flight; rows past the last are loaded again and not added
    for (int b = b0 + threadIdx.x / nch; b < b1; b += 2 * rows) {
        uint4 v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            v[u] = *reinterpret_cast<const uint4*>(ws.hist + (int64_t)min(b + u * rows, b1 - 1) * epad + 16 * ch);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (b + u * rows < b1) add_bytes(tot, v[u]);
            if (b + u * rows < min(b1, blk)) add_bytes(pre, v[u]);
        }
    }
    for (int e = threadIdx.x; e < epad; e += kThreads) mask[e] = 0;
    lanes_sum_mod(tot, nch);
    lanes_sum_mod(pre, nch);
    const int wave = threadIdx.x >> 6;
    uint4* d4 = reinterpret_cast<uint4*>(part + ((wave & (kHalf - 1)) * nch + ch) * 16);
    if (wave >= kHalf && (int)(threadIdx.x & 63) < nch) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            d4[i] = make_uint4(tot[4 * i], tot[4 * i + 1], tot[4 * i + 2], tot[4 * i + 3]);
            d4[2 + i] = make_uint4(pre[4 * i], pre[4 * i + 1], pre[4 * i + 2], pre[4 * i + 3]);
        }
    }
    __syncthreads();
    if (wave < kHalf && (int)(threadIdx.x & 63) < nch) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 a = d4[i], b = d4[2 + i];
            d4[i] = make_uint4(a.x + tot[4 * i], a.y + tot[4 * i + 1], a.z + tot[4 * i + 2], a.w + tot[4 * i + 3]);
            d4[2 + i] = make_uint4(b.x + pre[4 * i], b.y + pre[4 * i + 1], b.z + pre[4 * i + 2], b.w + pre[4 * i + 3]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (es[u] >= 0) atomicOr(&mask[es[u]], 1ull << ((uint32_t)(threadIdx.x + u * kThreads) / (uint32_t)p.k));
    int before = 0;
    // an expert's runs: a lane of its own per expert and row lane, met in LDS
    int* runs = reinterpret_cast<int*>(part + kHalf * epad);          // [2][kThreads]
    int rtot = 0, rpre = 0;
    const int nrun = SUPER ? (nblk + kRun - 1) / kRun : 0;
    if (SUPER) {
        const int e = threadIdx.x & (epad - 1);
#pragma unroll 8
        for (int r = threadIdx.x / epad; r < nrun; r += kThreads / epad) {
            const int c = ws.run_cnt[(int64_t)r * epad + e];
            rtot += c;
            if (r < blk / kRun) rpre += c;
        }
    }
    if ((int)threadIdx.x < epad) {
        const int e = threadIdx.x, i = e & 15;
        const int word = 2 * (i >> 2) + (i & 1), sh = (i & 2) * 8;
        int c = 0;
        for (int w = 0; w < kHalf; ++w) {
            const uint32_t* src = part + (w * nch + (e >> 4)) * 16;
            c += (int)((src[word] >> sh) & 0xffffu);
            before += (int)((src[8 + word] >> sh) & 0xffffu);
        }
        counts[e] = SUPER ? 0 : c;
        earlier[e] = before;
    }
    __syncthreads();
    if (SUPER) {
        runs[threadIdx.x] = rtot;
        runs[kThreads + threadIdx.x] = rpre;
        __syncthreads();
        if ((int)threadIdx.x < epad) {
            int c = 0;
            for (int r = threadIdx.x; r < kThreads; r += epad) { c += runs[r]; before += runs[kThreads + r]; }
            counts[threadIdx.x] = c;
            earlier[threadIdx.x] = before;
        }
        __syncthreads();
    }
    scan_experts(counts, base, p.E);
    __syncthreads();
    const int total = base[p.E];
    if (tokens) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = threadIdx.x + u * kThreads, e = max(es[u], 0);
            if (i < n) place_row(p, t0, i, es[u], mask, base[e] + earlier[e], total);
        }
        return;
    }
    __shared__ float red[48];
    s[0] = __builtin_fmaf((float)counts[e4], ps.x, (float)counts[e4 + 1] * ps.y) +
           __builtin_fmaf((float)counts[e4 + 2], ps.z, (float)counts[e4 + 3] * ps.w);
    block_sums(s, red);
    for (int e = threadIdx.x; e <= p.E; e += kThreads) {
        p.offsets[e] = base[e];
        p.counts[e] = e < p.E ? counts[e] : (int)s[2];
    }
    if (threadIdx.x == 0) write_losses(p, s[0], s[1], total, (int)s[2]);
}

// Counts and probability sums of runs of kRun workgroups, in order.  A
// workgroup takes one run and 64 experts; its 16 row lanes take 16 rows each.
__global__ void __launch_bounds__(kThreads) k_route_super(RouteArgs p, RouteWs ws, int nblk) {
    __shared__ int cnt[16][64];
    __shared__ float prob[16][64];
    const int r = threadIdx.x >> 6, l = threadIdx.x & 63, e = blockIdx.y * 64 + l;
    const int b0 = blockIdx.x * kRun + r * (kRun / 16);
    int c = 0;
    float f = 0.0f;
    if (e < ws.epad) {
#pragma unroll
        for (int i = 0; i < kRun / 16; ++i) {
            const int64_t at = (int64_t)min(b0 + i, nblk - 1) * ws.epad + e;
            const int h = ws.hist[at];
            const float v = ws.psum[at];
            c += b0 + i < nblk ? h : 0;
            f += b0 + i < nblk ? v : 0.0f;
        }
    }
    cnt[r][l] = c;
    prob[r][l] = f;
    __syncthreads();
    if (r > 0 || e >= ws.epad) return;
    for (int i = 1; i < 16; ++i) { c += cnt[i][l]; f += prob[i][l]; }
    ws.run_cnt[(int64_t)blockIdx.x * ws.epad + e] = c;
    ws.run_psum[(int64_t)blockIdx.x * ws.epad + e] = f;
}

// Backward.  Each term of the gradient at z_te:
//   balance, z   p_te (g0 E / n (f_e - sum_j f_j p_tj) + 2 g1 lse_t / n)
//   weights      renormalized: w_j (dw_j - sum_i w_i dw_i) at the selected;
//                else p_te (dw_e [selected] - sum_i w_i dw_i)
// L lanes hold a token; the selected slots' part meets the experts' lanes
// through one LDS row per token.  Latency-bound at these sizes: everything a
// token needs is loaded before the first use of any of it.
template <int L, int V, bool F32>
__global__ void __launch_bounds__(256) k_route_bwd(RouteBwdArgs p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int kGroups = 256 / L;
    const int l = threadIdx.x % L, grp = threadIdx.x / L;
    float* part = reinterpret_cast<float*>(dyn) + (int64_t)grp * (L * V);
    float f[V], fsum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = l + i * L;
        f[i] = (p.dloss && e < p.E) ? (float)p.counts[e] : 0.0f;
        fsum += f[i];
        part[e] = 0.0f;
    }
    float gb = 0.0f, gz = 0.0f;
    if (p.dloss) {
        const float n = (float)max(p.counts[p.E], 1);
        gb = p.dloss[0] * (float)p.E / n;
        gz = 2.0f * p.dloss[1] / n;
    }
    fsum = lanes_sum<L>(fsum);
    const float finv = 1.0f / fmaxf(fsum, 1.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] *= finv;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    // whole waves take part while any of their tokens is left: the reductions
    // need all lanes
    for (int64_t t1 = (int64_t)blockIdx.x * kGroups; t1 < p.T; t1 += step) {
        const bool have = t1 + grp < p.T;
        const int64_t t = have ? t1 + grp : p.T - 1;
        const float lse = p.lse[t];
        float z[V];
        load_logits<L, V, F32>(p.logits, t * p.ld, l, p.E, z);
        float w[2] = {0.0f, 0.0f}, dw[2] = {0.0f, 0.0f};
        int es[2] = {-1, -1};
        if (p.dweights) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = l + u * L;
                if (j < p.k) {
                    es[u] = p.experts[t * p.k + j];
                    w[u] = p.weights[t * p.k + j];
                    dw[u] = p.dweights[t * p.k + j];
                }
            }
        }
        const bool live = !(lse == -INFINITY);
        // p from the largest logit and the sum, as in the forward pass: exp(z -
        // lse) is wrong where lse has lost log(sum) to rounding (logits of the
        // type's lowest value)
        uint32_t key[V], best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = logit_key(z[i]) & ((live && l + i * L < p.E) ? 0xffffffffu : 0u);
            best = max(best, key[i]);
        }
        const float m = key_logit(lanes_umax<L>(best));
        float pr[V], dot = 0.0f, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float v = __builtin_amdgcn_exp2f((z[i] - m) * kLog2e);
            pr[i] = key[i] ? v : 0.0f;
            sum += pr[i];
            dot = __builtin_fmaf(pr[i], f[i], dot);
        }
        sum = lanes_sum<L>(sum);
        const float inv = live ? 1.0f / sum : 0.0f;
        dot = lanes_sum<L>(dot) * inv;
        float wd = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (!live || es[u] < 0 || es[u] >= p.E) { es[u] = -1; w[u] = dw[u] = 0.0f; }
            wd = __builtin_fmaf(w[u], dw[u], wd);
        }
        wd = lanes_sum<L>(wd);
        // the group's LDS row, within one wave: ordered by the fences
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (es[u] >= 0) part[es[u]] = p.renorm ? w[u] * (dw[u] - wd) : w[u] * dw[u];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float zt = gz * (live ? lse : 0.0f) - (p.renorm ? 0.0f : wd);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = l + i * L;
            const float d = __builtin_fmaf(pr[i] * inv, __builtin_fmaf(gb, f[i] - dot, zt), part[e]);
            part[e] = 0.0f;
            if (have && e < p.E) {
                if (F32) static_cast<float*>(p.dlogits)[t * p.ld_d + e] = d;
                else static_cast<uint16_t*>(p.dlogits)[t * p.ld_d + e] = (uint16_t)f32_to_bf16_rne(d);
            }
        }
    }
}

// Lanes and values per token by the number of experts.  Sixteen lanes of many
// values beat a wave of few in the selection, whose rounds then serve four
// tokens at once (16384 tokens of 512 experts: 35.1 against 41.4 us); the
// gradient has no rounds and more to hold (26.9 against 16.3 us).
template <template <int, int> class F, typename... A>
hipError_t by_experts(int E, A&&... a) {
    if (E <= 16) return F<16, 1>::run(a...);
    if (E <= 32) return F<16, 2>::run(a...);
    if (E <= 64) return F<16, 4>::run(a...);
    if (E <= 128) return F<16, 8>::run(a...);
    if (E <= 256) return F<16, 16>::run(a...);
    if (E <= 512) return F<F<64, 8>::kLanes512, 512 / F<64, 8>::kLanes512>::run(a...);
    return F<64, 16>::run(a...);
}

template <int L, int V>
struct Select {
    static constexpr int kLanes512 = 16;
    static hipError_t run(const RouteArgs& p, const RouteWs& ws, int nblk, hipStream_t st) {
        if (nblk <= 1) {
            const size_t lds = select_lds(p.E, L * V) + (size_t)p.E * 8 + 8;
            if (p.logits32) hipLaunchKernelGGL((k_route_one<L, V, true>), dim3(1), dim3(kThreads), lds, st, p);
            else hipLaunchKernelGGL((k_route_one<L, V, false>), dim3(1), dim3(kThreads), lds, st, p);
        } else {
            const size_t lds = select_lds(p.E, L * V);
            if (p.logits32) hipLaunchKernelGGL((k_route_select<L, V, true>), dim3(nblk), dim3(kThreads), lds, st, p, ws);
            else hipLaunchKernelGGL((k_route_select<L, V, false>), dim3(nblk), dim3(kThreads), lds, st, p, ws);
        }
        return hipGetLastError();
    }
};

template <int L, int V>
struct Backward {
    static constexpr int kLanes512 = 64;
    static hipError_t run(const RouteBwdArgs& p, hipStream_t st) {
        constexpr int kGroups = 256 / L;
        const int64_t blocks = (p.T + kGroups - 1) / kGroups;
        const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048));
        const size_t lds = sizeof(float) * kGroups * L * V;
        if (p.logits32) hipLaunchKernelGGL((k_route_bwd<L, V, true>), grid, dim3(256), lds, st, p);
        else hipLaunchKernelGGL((k_route_bwd<L, V, false>), grid, dim3(256), lds, st, p);
        return hipGetLastError();
    }
};

}  // namespace

// Workspace: per workgroup of tokens the histogram bytes [epad] and the
// probability sums [epad]; per workgroup the loss terms; for more than kDirect of
// them the runs' counts and probability sums [epad].
static RouteWs route_ws(int64_t T, int32_t E, void* base, size_t* bytes) {
    const int64_t nblk = (T + kTok - 1) / kTok;
    RouteWs ws{};
    ws.epad = 16;
    while (ws.epad < E) ws.epad *= 2;
    size_t off = 0;
    auto take = [&](size_t n) { const size_t o = off; off += (n + 15) / 16 * 16; return static_cast<char*>(base) + o; };
    if (nblk > 1) {
        ws.hist = reinterpret_cast<uint8_t*>(take((size_t)nblk * ws.epad));
        ws.psum = reinterpret_cast<float*>(take((size_t)nblk * ws.epad * 4));
        ws.lse2 = reinterpret_cast<float*>(take((size_t)nblk * 4));
        ws.live = reinterpret_cast<int32_t*>(take((size_t)nblk * 4));
    }
    if (nblk > kDirect) {
        const size_t n = (size_t)((nblk + kRun - 1) / kRun) * ws.epad * 4;
        ws.run_cnt = reinterpret_cast<int32_t*>(take(n));
        ws.run_psum = reinterpret_cast<float*>(take(n));
    }
    *bytes = off;
    return ws;
}

size_t route_ws_bytes(int64_t T, int32_t E) {
    size_t bytes;
    route_ws(T, E, nullptr, &bytes);
    return bytes;
}

RouteWs route_workspace(int64_t T, int32_t E, void* ws) {
    size_t bytes;
    return route_ws(T, E, ws, &bytes);
}

hipError_t launch_moe_route(const RouteArgs& p, void* wsp, hipStream_t st) {
    const int nblk = (int)((p.T + kTok - 1) / kTok);
    const RouteWs ws = route_workspace(p.T, p.E, wsp);
    const hipError_t e = by_experts<Select>(p.E, p, ws, nblk, st);
    return e != hipSuccess || nblk <= 1 ? e : launch_route_rows(p, ws, st);
}

hipError_t launch_route_rows(const RouteArgs& p, const RouteWs& ws, hipStream_t st) {
    const int nblk = (int)((p.T + kTok - 1) / kTok);
    hipError_t e;
    const size_t lds = (size_t)ws.epad * 20 + 16 + (size_t)kThreads * 8 + (size_t)kHalf * ws.epad * 4;
    if (nblk <= kDirect) {
        hipLaunchKernelGGL(k_route_place<false>, dim3(nblk + 1), dim3(kThreads), lds, st, p, ws, nblk);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(k_route_super, dim3((nblk + kRun - 1) / kRun, (ws.epad + 63) / 64), dim3(kThreads), 0, st, p, ws,
                       nblk);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(k_route_place<true>, dim3(nblk + 1), dim3(kThreads), lds, st, p, ws, nblk);
    return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const RouteBwdArgs& p, hipStream_t st) {
    if (p.T == 0) return hipSuccess;
    return by_experts<Backward>(p.E, p, st);
}

}  // namespace fp8bs
