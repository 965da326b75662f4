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
#include "device_common.h"
#include "internal.h"
#include "reduce.h"

namespace fp8bs {
namespace {

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

template <bool F32>
__device__ __forceinline__ float load_logit(const void* z, int64_t i) {
    if (F32) return static_cast<const float*>(z)[i];
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(z)[i] << 16);
}

// Exclusive prefix of counts[0..E) into LDS, by the first wave; E <= 1024.
__device__ __forceinline__ void scan_experts(const int* counts, int* excl, int E) {
    if (threadIdx.x < 64) {
        int carry = 0;
        for (int b = 0; b < E; b += 64) {
            const int e = b + threadIdx.x;
            const int c = e < E ? counts[e] : 0;
            int v = c;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(v, d, 64);
                if ((int)threadIdx.x >= d) v += o;
            }
            if (e < E) excl[e] = carry + v - c;
            carry += __shfl(v, 63, 64);
        }
        if (threadIdx.x == 0) excl[E] = carry;
    }
}

// Sum of one value per thread over the workgroup, in a fixed order (all
// threads call; the result is valid in thread 0).
__device__ __forceinline__ float block_sum(float v, float* lds) {
    v = lanes_sum<64>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
    if (threadIdx.x == 0)
        for (int w = 0; w < (int)(blockDim.x >> 6); ++w) s += lds[w];
    return s;
}

// Selection.  L lanes hold a token's logits, lane l the experts l, l + L, ...
// Each of the k rounds takes the largest key among the lanes and, of equal
// keys, the lowest expert.  The workgroup's 64 tokens leave in LDS, per
// expert, the mask of the tokens that chose it: the histogram is its
// population count, and a slot's rank among earlier tokens that of the bits
// below it, so the stable (expert, token) order needs no sort.
template <int L, int V, bool F32>
__device__ __forceinline__ void select_tokens(const RouteArgs& p, int64_t t0, unsigned long long* mask,
                                              float* psum, float* s_lse2, int* s_live) {
    constexpr int kGroups = kThreads / L;
    const int l = threadIdx.x % L, grp = threadIdx.x / L;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    float lse2 = 0.0f;
    int live_n = 0;
    for (int tt = grp; tt < kTok; tt += kGroups) {
        const int64_t t = t0 + tt;
        const bool have = t < p.T && (!p.mask || p.mask[t]);
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = l + i * L;
            key[i] = 0;
            if (have && e < p.E) key[i] = logit_key(load_logit<F32>(p.logits, t * p.ld + e));
        }
        uint32_t left[V];
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) { left[i] = key[i]; best = max(best, key[i]); }
        const uint32_t top = lanes_umax<L>(best);
        const bool live = top > kKeyNegInf;
        const float m = live ? key_logit(top) : 0.0f;
        float ex[V], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            ex[i] = key[i] ? __builtin_amdgcn_exp2f((key_logit(key[i]) - m) * kLog2e) : 0.0f;
            sum += ex[i];
        }
        sum = lanes_sum<L>(sum);
        const float lse = live ? m + logf(sum) : -INFINITY;
        float wsel = 0.0f, wnorm = 0.0f;            // lane j holds slot j's weight (slots past L: in turn)
        int esel = -1;
        float wsel2 = 0.0f;
        int esel2 = -1;
        for (int j = 0; j < p.k; ++j) {
            uint32_t b = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) b = max(b, left[i]);
            const uint32_t mx = lanes_umax<L>(b);
            uint32_t at = 0xffffffffu;
#pragma unroll
            for (int i = V - 1; i >= 0; --i) at = left[i] == mx ? (uint32_t)(l + i * L) : at;
            at = lanes_umin<L>(at);
            const bool ok = mx > kKeyNegInf;
#pragma unroll
            for (int i = 0; i < V; ++i) left[i] = (uint32_t)(l + i * L) == at ? 0u : left[i];
            const float w = ok ? __builtin_amdgcn_exp2f((key_logit(mx) - m) * kLog2e) : 0.0f;
            wnorm += w;
            if (l == (j % L)) {
                if (j < L) { wsel = w; esel = ok ? (int)at : -1; }
                else { wsel2 = w; esel2 = ok ? (int)at : -1; }
            }
            if (ok && l == 0) atomicOr(&mask[at], 1ull << tt);
        }
        const float norm = p.renorm ? wnorm : sum;
        if (t < p.T) {
            if (l < p.k) {
                p.experts[t * p.k + l] = esel;
                p.weights[t * p.k + l] = esel >= 0 ? wsel / norm : 0.0f;
            }
            if (l + L < p.k) {
                p.experts[t * p.k + l + L] = esel2;
                p.weights[t * p.k + l + L] = esel2 >= 0 ? wsel2 / norm : 0.0f;
            }
            if (l == 0) p.lse[t] = lse;
        }
        if (live) {
            const float inv = 1.0f / sum;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(ex[i], inv, acc[i]);
            lse2 = __builtin_fmaf(lse, lse, lse2);
            live_n++;
        }
    }
    // per-expert probability sums of the workgroup: the 64 / L groups of a
    // wave by shuffles, then the waves in order through LDS
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (L == 16) {
            acc[i] += __shfl_xor(acc[i], 16, 64);
            acc[i] += __shfl_xor(acc[i], 32, 64);
        }
    }
    for (int w = 0; w < kThreads / 64; ++w) {
        __syncthreads();
        if ((int)(threadIdx.x >> 6) == w && (threadIdx.x & 63) < L) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = l + i * L;
                if (e < p.E) psum[e] = (w ? psum[e] : 0.0f) + acc[i];
            }
        }
    }
    // lane 0 of every group holds its tokens' lse^2 and count
    float v[2] = {l == 0 ? lse2 : 0.0f, l == 0 ? (float)live_n : 0.0f};
    const float a = block_sum(v[0], s_lse2), b = block_sum(v[1], s_lse2);
    if (threadIdx.x == 0) { s_lse2[0] = a; *s_live = (int)b; }
    __syncthreads();
}

// The rows of a workgroup's tokens, given in LDS the first row of each expert
// for them, and the zeros of row_token behind the last row.
__device__ __forceinline__ void place_rows(const RouteArgs& p, int64_t t0, const unsigned long long* mask,
                                           const int* base, int total) {
    const int64_t n = min((int64_t)kTok, p.T - t0) * p.k;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const int64_t at = t0 * p.k + i;
        const int tt = (int)(i / p.k);
        const int e = p.experts[at];
        int row = -1;
        if (e >= 0) {
            row = base[e] + __popcll(mask[e] & ((1ull << tt) - 1));
            p.row_token[row] = (int32_t)(t0 + tt);
        }
        p.token_rows[at] = row;
        if (at >= total) p.row_token[at] = 0;
    }
}

__device__ __forceinline__ void write_losses(const RouteArgs& p, float fp, float lse2, int64_t sum_counts, int live) {
    const float n = (float)max(live, 1);
    p.loss[0] = (float)p.E * fp / ((float)max(sum_counts, (int64_t)1) * n);
    p.loss[1] = lse2 / n;
}

// Up to 64 tokens: the whole routing in one workgroup and one launch.
template <int L, int V, bool F32>
__global__ void __launch_bounds__(kThreads) k_route_one(RouteArgs p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(dyn);
    float* psum = reinterpret_cast<float*>(mask + p.E);
    int* counts = reinterpret_cast<int*>(psum + p.E);
    int* base = counts + p.E;                       // [E + 1]
    __shared__ float red[kThreads / 64];
    __shared__ int s_live;
    for (int e = threadIdx.x; e < p.E; e += kThreads) mask[e] = 0;
    __syncthreads();
    select_tokens<L, V, F32>(p, 0, mask, psum, red, &s_live);
    const float lse2 = red[0];
    const int live = s_live;
    for (int e = threadIdx.x; e < p.E; e += kThreads) counts[e] = __popcll(mask[e]);
    __syncthreads();
    scan_experts(counts, base, p.E);
    __syncthreads();
    float f = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        p.counts[e] = counts[e];
        p.offsets[e] = base[e];
        f = __builtin_fmaf((float)counts[e], psum[e], f);
    }
    place_rows(p, 0, mask, base, base[p.E]);
    f = block_sum(f, red);
    if (threadIdx.x == 0) {
        p.counts[p.E] = live;
        p.offsets[p.E] = base[p.E];
        write_losses(p, f, lse2, base[p.E], live);
    }
}

// More tokens, first launch: selection, and per workgroup the histogram, the
// probability sums and the loss terms.
template <int L, int V, bool F32>
__global__ void __launch_bounds__(kThreads) k_route_select(RouteArgs p, RouteWs ws) {
    extern __shared__ __align__(16) unsigned char dyn[];
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(dyn);
    float* psum = reinterpret_cast<float*>(mask + p.E);
    __shared__ float red[kThreads / 64];
    __shared__ int s_live;
    for (int e = threadIdx.x; e < p.E; e += kThreads) mask[e] = 0;
    __syncthreads();
    select_tokens<L, V, F32>(p, (int64_t)blockIdx.x * kTok, mask, psum, red, &s_live);
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        ws.hist[(int64_t)blockIdx.x * p.E + e] = __popcll(mask[e]);
        ws.psum[(int64_t)blockIdx.x * p.E + e] = psum[e];
    }
    if (threadIdx.x == 0) {
        ws.lse2[blockIdx.x] = red[0];
        ws.live[blockIdx.x] = s_live;
    }
}

// Second launch: per expert, the running row count over the workgroups (in
// place of the histogram) and the sum of the probabilities.  One wave per
// expert.
__global__ void __launch_bounds__(256) k_route_scan(RouteArgs p, RouteWs ws, int nblk) {
    const int e = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (e >= p.E) return;
    int carry = 0;
    float s = 0.0f;
    for (int b0 = 0; b0 < nblk; b0 += 64) {
        const int b = b0 + lane;
        const int c = b < nblk ? ws.hist[(int64_t)b * p.E + e] : 0;
        if (b < nblk) s += ws.psum[(int64_t)b * p.E + e];
        int v = c;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(v, d, 64);
            if (lane >= d) v += o;
        }
        if (b < nblk) ws.hist[(int64_t)b * p.E + e] = carry + v - c;
        carry += __shfl(v, 63, 64);
    }
    s = lanes_sum<64>(s);
    if (lane == 0) {
        p.counts[e] = carry;
        ws.total[e] = s;
    }
}

// Third launch: every workgroup scans the counts over the experts and places
// its tokens' rows; one more forms the losses.
__global__ void __launch_bounds__(kThreads) k_route_place(RouteArgs p, RouteWs ws, int nblk) {
    extern __shared__ __align__(16) unsigned char dyn[];
    unsigned long long* mask = reinterpret_cast<unsigned long long*>(dyn);
    int* counts = reinterpret_cast<int*>(mask + p.E);
    int* base = counts + p.E;                       // [E + 1]
    __shared__ float red[kThreads / 64];
    for (int e = threadIdx.x; e < p.E; e += kThreads) { mask[e] = 0; counts[e] = p.counts[e]; }
    __syncthreads();
    scan_experts(counts, base, p.E);
    const int64_t t0 = (int64_t)blockIdx.x * kTok;
    if ((int)blockIdx.x < nblk) {
        const int64_t n = min((int64_t)kTok, p.T - t0) * p.k;
        for (int64_t i = threadIdx.x; i < n; i += kThreads) {
            const int e = p.experts[t0 * p.k + i];
            if (e >= 0) atomicOr(&mask[e], 1ull << (int)(i / p.k));
        }
    }
    __syncthreads();
    const int total = base[p.E];
    if ((int)blockIdx.x < nblk) {
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kThreads) base[e] += ws.hist[(int64_t)blockIdx.x * p.E + e];
        __syncthreads();
        place_rows(p, t0, mask, base, total);
        return;
    }
    float f = 0.0f, l2 = 0.0f, lv = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        f = __builtin_fmaf((float)counts[e], ws.total[e], f);
        p.offsets[e] = base[e];
    }
    int live = 0;
    for (int b = threadIdx.x; b < nblk; b += kThreads) { l2 += ws.lse2[b]; live += ws.live[b]; }
    f = block_sum(f, red);
    l2 = block_sum(l2, red);
    // token counts below 2^24 a thread and 2^31 in all: summed as integers
    __shared__ int s_live;
    if (threadIdx.x == 0) s_live = 0;
    __syncthreads();
    atomicAdd(&s_live, live);
    __syncthreads();
    (void)lv;
    if (threadIdx.x == 0) {
        p.offsets[p.E] = total;
        p.counts[p.E] = s_live;
        write_losses(p, f, l2, total, s_live);
    }
}

// Backward.  Each term of the gradient at z_te:
//   balance, z   p_te (g0 E / n (f_e - sum_j f_j p_tj) + 2 g1 lse_t / n)
//   weights      renormalized: w_j (dw_j - sum_i w_i dw_i) at the selected;
//                else p_te (dw_e [selected] - sum_i w_i dw_i)
// L lanes hold a token; the selected slots' part meets the experts' lanes
// through one LDS row per token.
template <int L, int V, bool F32>
__global__ void __launch_bounds__(256) k_route_bwd(RouteBwdArgs p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int kGroups = 256 / L;
    const int l = threadIdx.x % L, grp = threadIdx.x / L;
    float* part = reinterpret_cast<float*>(dyn) + (int64_t)grp * (L * V);
    float f[V];
    float fsum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = l + i * L;
        f[i] = (p.dloss && e < p.E) ? (float)p.counts[e] : 0.0f;
        part[e] = 0.0f;
    }
    // counts are whole numbers: their sum is exact below 2^24 and rounded once above
    for (int e = l; p.dloss && e < p.E; e += L) fsum += (float)p.counts[e];
    fsum = lanes_sum<L>(fsum);
    float gb = 0.0f, gz = 0.0f;
    if (p.dloss) {
        const float n = (float)max(p.counts[p.E], 1);
        gb = p.dloss[0] * (float)p.E / n;
        gz = 2.0f * p.dloss[1] / n;
    }
    const float finv = 1.0f / fmaxf(fsum, 1.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] *= finv;
    for (int64_t t = (int64_t)blockIdx.x * kGroups + grp; t < p.T; t += (int64_t)gridDim.x * kGroups) {
        const float lse = p.lse[t];
        const bool live = !(lse == -INFINITY);
        // p from the largest logit and the sum, as in the forward pass: exp(z -
        // lse) is wrong where lse has lost log(sum) to rounding (logits of the
        // type's lowest value)
        float pr[V], dot = 0.0f, sum = 0.0f;
        uint32_t key[V], best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = l + i * L;
            key[i] = (live && e < p.E) ? logit_key(load_logit<F32>(p.logits, t * p.ld + e)) : 0u;
            best = max(best, key[i]);
        }
        const float m = key_logit(lanes_umax<L>(best));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            pr[i] = key[i] ? __builtin_amdgcn_exp2f((key_logit(key[i]) - m) * kLog2e) : 0.0f;
            sum += pr[i];
            dot = __builtin_fmaf(pr[i], f[i], dot);
        }
        sum = lanes_sum<L>(sum);
        const float inv = live ? 1.0f / sum : 0.0f;
        dot = lanes_sum<L>(dot) * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) pr[i] *= inv;
        float wd = 0.0f;
        float w[2] = {0.0f, 0.0f}, dw[2] = {0.0f, 0.0f};
        int es[2] = {-1, -1};
        if (p.dweights && live) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = l + u * L;
                if (j < p.k) {
                    es[u] = p.experts[t * p.k + j];
                    w[u] = es[u] >= 0 ? p.weights[t * p.k + j] : 0.0f;
                    dw[u] = es[u] >= 0 ? p.dweights[t * p.k + j] : 0.0f;
                    wd = __builtin_fmaf(w[u], dw[u], wd);
                }
            }
        }
        wd = lanes_sum<L>(wd);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (es[u] >= 0 && es[u] < p.E) part[es[u]] = p.renorm ? w[u] * (dw[u] - wd) : w[u] * dw[u];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float zt = gz * (live ? lse : 0.0f) - (p.renorm ? 0.0f : wd);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = l + i * L;
            const float d = __builtin_fmaf(pr[i], __builtin_fmaf(gb, f[i] - dot, zt), part[e]);
            part[e] = 0.0f;
            if (e < p.E) {
                if (F32) static_cast<float*>(p.dlogits)[t * p.ld_d + e] = d;
                else static_cast<uint16_t*>(p.dlogits)[t * p.ld_d + e] = (uint16_t)f32_to_bf16_rne(d);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Lanes and values per token by the number of experts.
template <template <int, int> class F, typename... A>
hipError_t by_experts(int E, A&&... a) {
    if (E <= 16) return F<16, 1>::run(a...);
    if (E <= 32) return F<16, 2>::run(a...);
    if (E <= 64) return F<16, 4>::run(a...);
    if (E <= 128) return F<16, 8>::run(a...);
    if (E <= 256) return F<64, 4>::run(a...);
    if (E <= 512) return F<64, 8>::run(a...);
    return F<64, 16>::run(a...);
}

template <int L, int V>
struct Select {
    static hipError_t run(const RouteArgs& p, const RouteWs& ws, int nblk, hipStream_t st) {
        if (nblk <= 1) {
            const size_t lds = (size_t)p.E * 20 + 8;
            if (p.logits32) hipLaunchKernelGGL((k_route_one<L, V, true>), dim3(1), dim3(kThreads), lds, st, p);
            else hipLaunchKernelGGL((k_route_one<L, V, false>), dim3(1), dim3(kThreads), lds, st, p);
        } else {
            const size_t lds = (size_t)p.E * 12;
            if (p.logits32) hipLaunchKernelGGL((k_route_select<L, V, true>), dim3(nblk), dim3(kThreads), lds, st, p, ws);
            else hipLaunchKernelGGL((k_route_select<L, V, false>), dim3(nblk), dim3(kThreads), lds, st, p, ws);
        }
        return hipGetLastError();
    }
};

template <int L, int V>
struct Backward {
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

size_t route_ws_bytes(int64_t T, int32_t E) {
    const int64_t nblk = (T + kTok - 1) / kTok;
    if (nblk <= 1) return 0;
    return (size_t)(nblk * (2 * (int64_t)E + 2) + E) * 4;
}

hipError_t launch_moe_route(const RouteArgs& p, void* wsp, hipStream_t st) {
    const int nblk = (int)((p.T + kTok - 1) / kTok);
    RouteWs ws{};
    ws.hist = static_cast<int32_t*>(wsp);
    ws.psum = reinterpret_cast<float*>(ws.hist + (int64_t)nblk * p.E);
    ws.lse2 = ws.psum + (int64_t)nblk * p.E;
    ws.live = reinterpret_cast<int32_t*>(ws.lse2 + nblk);
    ws.total = reinterpret_cast<float*>(ws.live + nblk);
    hipError_t e = by_experts<Select>(p.E, p, ws, nblk, st);
    if (e != hipSuccess || nblk <= 1) return e;
    hipLaunchKernelGGL(k_route_scan, dim3((p.E + 3) / 4), dim3(256), 0, st, p, ws, nblk);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(k_route_place, dim3(nblk + 1), dim3(kThreads), (size_t)p.E * 16 + 8, st, p, ws, nblk);
    return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const RouteBwdArgs& p, hipStream_t st) {
    if (p.T == 0) return hipSuccess;
    return by_experts<Backward>(p.E, p, st);
}

}  // namespace fp8bs
