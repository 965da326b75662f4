// The router with scores, a selection bias and groups of experts, and its gradient.
//
//   s_e     sigmoid(z_e), or softmax(z)_e;  v_e = s_e + bias_e
//   groups  E / groups consecutive experts each; a group's value is its largest v or
//           the sum of its two largest; the `keep` best groups stay, ties to the lower
//   taken   of their experts the k largest v, ties to the lower expert
//   w_j     scale s_j / (sum of the taken s + 1e-20), or scale s_j
//   total   sum_e s_e (sigmoid), log sum_e exp z_e (softmax);  p_e = s_e / (sum s + 1e-20)
//   losses  as the plain router's with these p; the z loss only with softmax
//
// Which experts are taken is decided as in 64 bits.  Without a bias the logits
// themselves are compared, which is exact.  Else values are compared in fp32, and a
// token of which two (or two groups) come closer than the fp32 error is selected again in
// 64 bits by its whole wave: two roundings would otherwise decide which expert gets the
// token, and with it every row behind.  That is about one token in 700 over 256 experts
// where values are spread (fp32 logits, a bias that has moved); equal values are as close
// as any, so bf16 logits under a bias of zeros, as at the start of training, repeat a
// third of the tokens, and equal logits all: 16384 x 256 in 59 and 68 us, not 36 (45 with
// equal logits and no bias, where only the groups' sums tie).
//
// The lanes of a token are dealt to the groups, a power of two each, and hold
// consecutive experts, so that a group's maxima meet in a few lane steps.  The rest
// is the plain router's: histograms, rows and losses come from the same code.
// Bound by vector issue: a token's `k` rounds of maxima over its lanes are dependent.
// 16384 tokens of 256 experts (16.8 MB of logits, 3 us): selection 27 us, rows 10;
// 32 tokens of 128 in one launch 9.0; the gradient, one pass over logits and result, a
// load or a store per value, 12 us at 16384 x 256 (2.7 TB/s) and 3.7 at 1000 x 60.
#include "route_common.h"

namespace fp8bs {
namespace {

constexpr float kEps = 1e-20f;

// Lanes: group = l / q; its part l % q holds `w` experts (fewer at the group's end).
struct GateLanes {
    int per, q, w;
    bool vec, vec_bias;             // rows, and the bias, in pieces of four
};

struct Score {
    float s, rest;                  // s and s (1 - s) of a sigmoid
};
// exp(-|z|) <= 1: no overflow, and 1 - s without cancellation.  Absolute error of s
// at most 6.6 * 2^-24: t errs by t (1.5 |z| + 2) 2^-24 <= 2.6 * 2^-24 (argument,
// hardware exp2), then the reciprocal, the sum and a product, 4 * 2^-24 in all.
__device__ __forceinline__ Score sigmoid(float z) {
    const float t = __builtin_amdgcn_exp2f(-fabsf(z) * kLog2e);
    const float r = __builtin_amdgcn_rcpf(1.0f + t);
    return {z >= 0.0f ? r : t * r, t * r * r};
}

// Order-preserving 64-bit key of a value, as logit_key.
__device__ __forceinline__ uint64_t value_key(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    const uint64_t k = (b >> 63) ? ~b : b | (1ull << 63);
    return v != v ? ~0ull : k;
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
}
constexpr uint64_t kKeyNegInf64 = 0x000fffffffffffffull;

template <class K> struct Keys;
template <> struct Keys<uint32_t> { static constexpr uint32_t kNegInf = kKeyNegInf; };
template <> struct Keys<uint64_t> { static constexpr uint64_t kNegInf = kKeyNegInf64; };

__device__ __forceinline__ uint32_t lane_xor(uint32_t v, int d) { return (uint32_t)__shfl_xor((int)v, d, 64); }
__device__ __forceinline__ uint64_t lane_xor(uint64_t v, int d) {
    return (uint64_t)lane_xor((uint32_t)(v >> 32), d) << 32 | lane_xor((uint32_t)v, d);
}
__device__ __forceinline__ uint32_t lane_at(uint32_t v, int lane) { return (uint32_t)__shfl((int)v, lane, 64); }
__device__ __forceinline__ float lane_at(float v, int lane) { return __shfl(v, lane, 64); }
__device__ __forceinline__ double lane_at(double v, int lane) { return __shfl(v, lane, 64); }
template <int L>
__device__ __forceinline__ uint32_t lanes_kmax(uint32_t v) { return lanes_umax<L>(v); }
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_mov64(uint64_t v) {
    return (uint64_t)dpp_mov<CTRL>((uint32_t)(v >> 32)) << 32 | dpp_mov<CTRL>((uint32_t)v);
}
template <int L>
__device__ __forceinline__ uint64_t lanes_kmax(uint64_t v) {
    static_assert(L == 64, "one token per wave");
    v = max(v, dpp_mov64<kDppXor1>(v));
    v = max(v, dpp_mov64<kDppXor2>(v));
    v = max(v, dpp_mov64<kDppHalfMirror>(v));
    v = max(v, dpp_mov64<kDppMirror>(v));
    auto at = [&](int lane) { return (uint64_t)lane_value((uint32_t)(v >> 32), lane) << 32 | lane_value((uint32_t)v, lane); };
    return max(max(at(0), at(16)), max(at(32), at(48)));
}
__device__ __forceinline__ uint32_t lane_dpp(uint32_t v, int d) {
    return d == 1 ? dpp_mov<kDppXor1>(v) : d == 2 ? dpp_mov<kDppXor2>(v) : d == 4 ? dpp_mov<kDppHalfMirror>(v)
                                                                                    : dpp_mov<kDppMirror>(v);
}
__device__ __forceinline__ uint64_t lane_dpp(uint64_t v, int d) {
    return (uint64_t)lane_dpp((uint32_t)(v >> 32), d) << 32 | lane_dpp((uint32_t)v, d);
}
template <int L>
__device__ __forceinline__ double lanes_sum64(double v) {
#pragma unroll
    for (int d = 1; d < L; d <<= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// One token's selection by keys (0: not there).  val maps a key to its value; the
// values' type F says whether close ones are reported (float: they may be in the
// wrong order; tol0 + 2^-22 |v| bounds twice a value's error) or taken as they are
// (double).  Groups are compared by half their values, whose sums stay finite.  Such a
// sum errs by its two values' errors and its own rounding, at most tol0 / 2 + 2^-23 mag
// with mag = |v1 / 2| + |v2 / 2|, which biases that cancel in the sum leave large: of two
// groups the one with the larger mag reports that they are nearer than tol0 + 2^-22 mag
// (2^-21: room for the roundings here).  EXACT: the keys' own order is the values' (no
// bias), so only sums of values can be in doubt.  On return lane j has slot j's key and
// expert in ksel[0], esel[0], and slot j + L's in [1].
template <int L, int V, bool EXACT, class K, class F, class VAL>
__device__ __forceinline__ bool pick(K (&left)[V], const GateArgs& g, const GateLanes& n, int l, int e0, F tol0, VAL val,
                                     K (&ksel)[2], uint32_t (&esel)[2]) {
    constexpr K kNone = Keys<K>::kNegInf;
    constexpr bool kReport = sizeof(F) == 4;
    bool close = false;
    if (g.keep < g.groups) {
        const int group = l / n.q, row = (threadIdx.x & 63) & ~(L - 1);
        K m1 = 0, m2 = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            m2 = max(m2, min(m1, left[i]));
            m1 = max(m1, left[i]);
        }
        // inside sixteen lanes the steps are lane moves: once pairs (quads, ...) agree,
        // a mirror image serves as the other pair (quad, ...)
#pragma unroll
        for (int d = 1; d < L; d <<= 1) {
            if (d < n.q) {
                const K a = d < 16 ? lane_dpp(m1, d) : lane_xor(m1, d), b = d < 16 ? lane_dpp(m2, d) : lane_xor(m2, d);
                m2 = max(min(m1, a), max(m2, b));
                m1 = max(m1, a);
            }
        }
        int rank = 0;
        if (EXACT && !g.top2) {                     // by the logits' 32-bit keys
            for (int j = 0; j < g.groups; ++j) {
                const uint32_t o = lane_at((uint32_t)m1, row + j * n.q);
                rank += o > m1 || (o == m1 && j < group);
            }
        } else {
            // NaN counts as infinity, a group without experts as the least
            F mine = m1 > kNone ? (F)0.5 * val(m1) : (F)-INFINITY, mag = mine < 0 ? -mine : mine;
            if (g.top2 && m2 > kNone) {
                const F second = (F)0.5 * val(m2);
                mine += second;
                mag += second < 0 ? -second : second;
            }
            if (mine != mine) mine = (F)INFINITY;
            for (int j = 0; j < g.groups; ++j) {
                const F o = lane_at(mine, row + j * n.q);
                rank += o > mine || (o == mine && j < group);
                // an infinite difference, or none between infinities, is not close
                if (kReport) close |= j != group && fabsf((float)(o - mine)) <= (float)tol0 + 0x1p-21f * (float)mag;
            }
            close = close && mine > (F)-INFINITY && mine < (F)INFINITY;
        }
        if (rank >= g.keep) {
#pragma unroll
            for (int i = 0; i < V; ++i) left[i] = 0;
        }
    }
    ksel[0] = ksel[1] = 0;
    esel[0] = esel[1] = 0;
    K last = 0;
    // one more round tells how close the best one left is
    const int rounds = kReport && !EXACT ? g.r.k + 1 : g.r.k;
    for (int j = 0; j < rounds; ++j) {
        K best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, left[i]);
        const K mx = lanes_kmax<L>(best);
        if (kReport && !EXACT) {
            const float a = (float)val(last), b = (float)val(mx);
            close |= j > 0 && mx > kNone && a - b <= (float)tol0 + 0x1p-22f * fabsf(a);
            last = mx;
        }
        uint32_t at = 0x10000u;
#pragma unroll
        for (int i = V - 1; i >= 0; --i) at = left[i] == mx ? (uint32_t)i : at;
        const uint32_t lowest = lanes_umin<L>(at + (uint32_t)e0);
        const uint32_t mine = lowest - (uint32_t)e0;
#pragma unroll
        for (int i = 0; i < V; ++i) left[i] = mine == (uint32_t)i ? (K)0 : left[i];
        if (l == j && j < g.r.k) { ksel[0] = mx; esel[0] = lowest; }
        if (l + L == j && j < g.r.k) { ksel[1] = mx; esel[1] = lowest; }
    }
    return close;
}

// A lane's logits e0, e0 + 1, ... of the row that starts at element `row`; no
// address leaves the row, what is past the lane's share is dropped by the caller.
template <int V, bool F32>
__device__ __forceinline__ void load_run(const void* base, int64_t row, int e0, int E, bool vec, float (&z)[V]) {
    if (vec && V >= 4) {
#pragma unroll
        for (int i = 0; i + 3 < V; i += 4) {
            const int64_t at = row + min(e0 + i, E - 4);
            if (F32) {
                const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
                z[i] = v.x; z[i + 1] = v.y; z[i + 2] = v.z; z[i + 3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
                z[i] = bf16_lo(v.x); z[i + 1] = bf16_hi(v.x); z[i + 2] = bf16_lo(v.y); z[i + 3] = bf16_hi(v.y);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t at = row + min(e0 + i, E - 1);
        z[i] = F32 ? static_cast<const float*>(base)[at]
                   : __uint_as_float((uint32_t)static_cast<const uint16_t*>(base)[at] << 16);
    }
}
template <bool F32>
__device__ __forceinline__ float logit_at(const void* base, int64_t at) {
    return F32 ? static_cast<const float*>(base)[at]
               : __uint_as_float((uint32_t)static_cast<const uint16_t*>(base)[at] << 16);
}

// One token's selection with values in 64 bits, by the whole wave (n: its 64 lanes
// dealt to the groups).  Lane j returns slot j's expert, or -1.
template <int V, bool F32, bool SIG>
__device__ __forceinline__ int pick_again(const GateArgs& g, const GateLanes& n, int64_t t, float m) {
    const int l = threadIdx.x & 63, group = l / n.q, part = l % n.q;
    const int e0 = group < g.groups ? group * n.per + part * n.w : 0;
    const int cnt = group < g.groups ? max(min(n.per - part * n.w, n.w), 0) : 0;
    float z[V];
    load_run<V, F32>(g.r.logits, t * g.r.ld, e0, g.r.E, n.vec, z);
    double sum = 1.0;
    if (!SIG) {
        sum = 0.0;
#pragma unroll 1
        for (int i = 0; i < cnt; ++i) {
            float x = z[0];
#pragma unroll
            for (int u = 1; u < V; ++u) x = i == u ? z[u] : x;
            sum += exp((double)x - (double)m);
        }
        sum = lanes_sum64<64>(sum);
    }
    auto score = [&](float x) {
        return SIG ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)m) / sum;
    };
    uint32_t esel[2];
    bool ok;
    if (g.bias) {
        uint64_t left[V], ksel[2];
#pragma unroll
        for (int i = 0; i < V; ++i) left[i] = 0;
        // one exponential in the code, not V of them
#pragma unroll 1
        for (int i = 0; i < cnt; ++i) {
            float x = z[0];
#pragma unroll
            for (int u = 1; u < V; ++u) x = i == u ? z[u] : x;
            const uint64_t key = x == -INFINITY ? 0 : value_key(score(x) + (double)g.bias[e0 + i]);
#pragma unroll
            for (int u = 0; u < V; ++u) left[u] = i == u ? key : left[u];
        }
        pick<64, V, false>(left, g, n, l, e0, 0.0, [](uint64_t k) { return key_value(k); }, ksel, esel);
        ok = ksel[0] > kKeyNegInf64;
    } else {
        uint32_t left[V], ksel[2];
#pragma unroll
        for (int i = 0; i < V; ++i) left[i] = i < cnt ? logit_key(z[i]) : 0u;
        pick<64, V, true>(left, g, n, l, e0, 0.0, [&](uint32_t k) { return score(key_logit(k)); }, ksel, esel);
        ok = ksel[0] > kKeyNegInf;
    }
    return ok ? (int)esel[0] : -1;
}

// As the plain router's selection: masks and probability sums in LDS, {sum of
// lse^2, routed tokens} to every thread.
template <int L, int V, int VW, bool F32, bool SIG>
__device__ __forceinline__ float2 gate_tokens(const GateArgs& g, const GateLanes& n, const GateLanes& nw, int64_t t0,
                                              unsigned long long* mask, float* psum) {
    constexpr int kGroups = kThreads / L;
    const RouteArgs& p = g.r;
    __shared__ float red[32];
    const int l = threadIdx.x % L, grp = threadIdx.x / L;
    const int group = l / n.q, part = l % n.q;
    const int e0 = group < g.groups ? group * n.per + part * n.w : 0;
    const int cnt = group < g.groups ? max(min(n.per - part * n.w, n.w), 0) : 0;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    float sums[2] = {0.0f, 0.0f};                   // lse^2, tokens: in lane 0 of a group
    for (int tt = grp; tt < kTok; tt += kGroups) {
        if (t0 + tt - grp % (64 / L) >= p.T) break; // no lane of the wave has a token
        const int64_t t = min(t0 + tt, p.T - 1);
        const bool have = t0 + tt < p.T && (!p.mask || p.mask[t]);
        float s[V];
        load_run<V, F32>(p.logits, t * p.ld, e0, p.E, n.vec, s);
        float b[V];
        if (g.bias) load_run<V, true>(g.bias, 0, e0, p.E, n.vec_bias, b);
        uint32_t left[V], best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            left[i] = logit_key(s[i]) & ((have && i < cnt) ? 0xffffffffu : 0u);
            best = max(best, left[i]);
        }
        const uint32_t top = lanes_umax<L>(best);
        const bool live = top > kKeyNegInf;
        const float m = live ? key_logit(top) : 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float v = SIG ? sigmoid(s[i]).s : __builtin_amdgcn_exp2f((s[i] - m) * kLog2e);
            s[i] = left[i] ? v : 0.0f;
            sum += s[i];
        }
        sum = lanes_sum<L>(sum);
        const float inv = live ? 1.0f / (SIG ? sum + kEps : sum) : 0.0f;
        if (!SIG) {
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] *= inv;
        }
        // Twice a value's error.  Softmax: the exponent errs by 2.5 |z - m| 2^-24
        // relative to p, and p |z - m| <= 0.37 times the largest p = 1 / sum; the sum,
        // common to all, by at most 57 * 2^-24 (up to 20 from its terms, 38 from
        // chains of 32 and 6).
        const float tol0 = SIG ? 0x1p-20f : 0x1p-16f * inv;
        uint32_t ksel[2], esel[2];
        bool ok[2], close;
        if (g.bias) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float v = s[i] + b[i];
                left[i] = left[i] > kKeyNegInf ? logit_key(v) : 0u;
            }
            close = pick<L, V, false>(left, g, n, l, e0, tol0, [](uint32_t k) { return key_logit(k); }, ksel, esel);
        } else {
            close = pick<L, V, true>(left, g, n, l, e0, tol0, [&](uint32_t k) {
                const float z = key_logit(k);
                return SIG ? sigmoid(z).s : __builtin_amdgcn_exp2f((z - m) * kLog2e) * inv;
            }, ksel, esel);
        }
        ok[0] = ksel[0] > kKeyNegInf;
        ok[1] = ksel[1] > kKeyNegInf;
        // the tokens of this wave whose order fp32 leaves open, one after the other
        for (unsigned long long open = __ballot(close); open;) {
            const int row = (__ffsll(open) - 1) & ~(L - 1);
            open &= L == 64 ? 0 : ~(((1ull << (L & 63)) - 1) << row);
            const int e = pick_again<VW, F32, SIG>(g, nw, (int64_t)__builtin_amdgcn_readlane((int)t, row), lane_at(m, row));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int got = __shfl(e, l + u * L, 64);
                if ((int)(threadIdx.x & 63 & ~(L - 1)) == row) {
                    ok[u] = got >= 0 && l + u * L < 64;
                    esel[u] = (uint32_t)max(got, 0);
                }
            }
        }
        float w[2], wsum = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w[u] = 0.0f;
            if (ok[u]) {
                const float z = logit_at<F32>(p.logits, t * p.ld + esel[u]);
                w[u] = SIG ? sigmoid(z).s : __builtin_amdgcn_exp2f((z - m) * kLog2e) * inv;
            }
            wsum += w[u];
        }
        const float norm = p.renorm ? lanes_sum<L>(wsum) + kEps : 1.0f;
        const float total = !live ? -INFINITY : SIG ? sum : m + logf(sum);
        if (t0 + tt < p.T) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = l + u * L;
                if (j < p.k) {
                    p.experts[t * p.k + j] = ok[u] ? (int)esel[u] : -1;
                    p.weights[t * p.k + j] = ok[u] ? g.scale * (w[u] / norm) : 0.0f;
                    if (ok[u]) atomicOr(&mask[esel[u]], 1ull << tt);
                }
            }
            if (l == 0) p.lse[t] = total;
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = SIG ? __builtin_fmaf(s[i], inv, acc[i]) : acc[i] + s[i];
            if (l == 0) {
                if (!SIG) sums[0] = __builtin_fmaf(total, total, sums[0]);
                sums[1] += 1.0f;
            }
        }
    }
    // the 64 / L groups of a wave in registers, waves w and w + 8, then those
    // in order
    const int wave = threadIdx.x >> 6;
    float* mine = psum + (wave & (kHalf - 1)) * p.E + e0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (L == 16) acc[i] = rows_sum(acc[i]);
    if (wave >= kHalf && (threadIdx.x & 63) < L) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < cnt) mine[i] = acc[i];
    }
    __syncthreads();
    if (wave < kHalf && (threadIdx.x & 63) < L) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < cnt) mine[i] += acc[i];
    }
    block_sums(sums, red);                          // its barrier covers psum and mask too
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kHalf; ++w) v += psum[w * p.E + e];
        psum[e] = v;                                // column e is this thread's alone
    }
    return make_float2(sums[0], sums[1]);
}

template <int L, int V, int VW, bool F32, bool SIG>
__global__ void __launch_bounds__(kThreads) k_gate_one(GateArgs g, GateLanes n, GateLanes nw) {
    extern __shared__ __align__(16) unsigned char dyn[];
    route_one(g.r, dyn, kHalf * g.r.E, [&](unsigned long long* mask, float* psum) {
        return gate_tokens<L, V, VW, F32, SIG>(g, n, nw, 0, mask, psum);
    });
}

template <int L, int V, int VW, bool F32, bool SIG>
__global__ void __launch_bounds__(kThreads) k_gate_select(GateArgs g, GateLanes n, GateLanes nw, RouteWs ws) {
    extern __shared__ __align__(16) unsigned char dyn[];
    route_select(g.r, ws, dyn, [&](unsigned long long* mask, float* psum) {
        return gate_tokens<L, V, VW, F32, SIG>(g, n, nw, (int64_t)blockIdx.x * kTok, mask, psum);
    });
}

// Backward.  With a_e the gradient at the score of expert e,
//   weights   a_j += scale dw_j, or renormalized scale (dw_j - sum_i w'_i dw_i) / norm,
//             w' = s / norm, norm = sum of the taken s + 1e-20, at the taken experts
//   balance   a_e += g0 E / n (f_e - sum_i f_i p_i) / (sum s + 1e-20) (sigmoid),
//             a_e += g0 E / n f_e (softmax)
//   sigmoid   dz_e = a_e s_e (1 - s_e)
//   softmax   dz_e = p_e (a_e - sum_i p_i a_i + 2 g1 lse / n)
// A token's lanes hold every L-th expert; the taken ones' part meets them through
// one LDS row per token.
template <int L, int V, bool F32, bool SIG>
__global__ void __launch_bounds__(256) k_gate_bwd(GateBwdArgs p) {
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
        gz = SIG ? 0.0f : 2.0f * p.dloss[1] / n;
    }
    fsum = lanes_sum<L>(fsum);
    const float finv = gb / fmaxf(fsum, 1.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] *= finv;       // g0 E / n f_e
    const int64_t step = (int64_t)gridDim.x * kGroups;
    // whole waves take part while any of their tokens is left: the reductions
    // need all lanes
    for (int64_t t1 = (int64_t)blockIdx.x * kGroups; t1 < p.T; t1 += step) {
        const bool have = t1 + grp < p.T;
        const int64_t t = have ? t1 + grp : p.T - 1;
        const float total = p.total[t];
        const bool live = !(total == -INFINITY);
        float z[V];
        load_logits<L, V, F32>(p.logits, t * p.ld, l, p.E, z);
        float zs[2] = {0.0f, 0.0f}, dw[2] = {0.0f, 0.0f};
        int es[2] = {-1, -1};
        if (p.dweights) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = l + u * L;
                if (j < p.k) {
                    es[u] = p.experts[t * p.k + j];
                    dw[u] = p.scale * p.dweights[t * p.k + j];
                }
                if (!live || es[u] < 0 || es[u] >= p.E) es[u] = -1;
                if (es[u] >= 0) zs[u] = logit_at<F32>(p.logits, t * p.ld + es[u]);
            }
        }
        float s[V], d[V], sum = 0.0f, dot = 0.0f, m = 0.0f;
        if (SIG) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Score c = sigmoid(z[i]);
                const bool in = live && l + i * L < p.E;
                s[i] = in ? c.s : 0.0f;
                d[i] = in ? c.rest : 0.0f;
                sum += s[i];
                dot = __builtin_fmaf(s[i], f[i], dot);
            }
        } else {
            uint32_t key[V], best = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                key[i] = logit_key(z[i]) & ((live && l + i * L < p.E) ? 0xffffffffu : 0u);
                best = max(best, key[i]);
            }
            m = key_logit(lanes_umax<L>(best));
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float v = __builtin_amdgcn_exp2f((z[i] - m) * kLog2e);
                s[i] = key[i] ? v : 0.0f;
                sum += s[i];
                dot = __builtin_fmaf(s[i], f[i], dot);
            }
        }
        sum = lanes_sum<L>(sum);
        const float inv = live ? 1.0f / (SIG ? sum + kEps : sum) : 0.0f;
        dot = lanes_sum<L>(dot) * inv;
        // the taken experts' scores and their gradients
        float w[2], wsum = 0.0f, wd = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w[u] = 0.0f;
            if (es[u] >= 0) w[u] = SIG ? sigmoid(zs[u]).s : __builtin_amdgcn_exp2f((zs[u] - m) * kLog2e) * inv;
            else dw[u] = 0.0f;
            wsum += w[u];
        }
        if (p.renorm) {
            const float norm = 1.0f / (lanes_sum<L>(wsum) + kEps);
            const float mean = lanes_sum<L>(__builtin_fmaf(w[0], dw[0], w[1] * dw[1])) * norm;
#pragma unroll
            for (int u = 0; u < 2; ++u) dw[u] = (dw[u] - mean) * norm;
        }
        if (!SIG) wd = lanes_sum<L>(__builtin_fmaf(w[0], dw[0], w[1] * dw[1]));
        // the group's LDS row, within one wave: ordered by the fences
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (es[u] >= 0) part[es[u]] = dw[u];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float zt = gz * (live ? total : 0.0f) - wd - dot;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = l + i * L;
            const float g = SIG ? d[i] * __builtin_fmaf(f[i] - dot, inv, part[e]) : s[i] * inv * (f[i] + part[e] + zt);
            part[e] = 0.0f;
            if (have && e < p.E) {
                const float r = live ? g : 0.0f;
                if (F32) static_cast<float*>(p.dlogits)[t * p.ld_d + e] = r;
                else static_cast<uint16_t*>(p.dlogits)[t * p.ld_d + e] = (uint16_t)f32_to_bf16_rne(r);
            }
        }
    }
}

// bias_e += rate sign(mean(counts) - counts_e), the comparison in whole numbers.
__global__ void __launch_bounds__(1024) k_bias_update(float* bias, const int32_t* counts, int E, float rate) {
    __shared__ long long part[16];
    const int e = threadIdx.x;
    const long long c = e < E ? counts[e] : 0;
    long long sum = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if ((e & 63) == 0) part[e >> 6] = sum;
    __syncthreads();
    sum = 0;
    for (int i = 0; i < 16; ++i) sum += part[i];
    if (e < E && c * E != sum) bias[e] += c * E < sum ? rate : -rate;
}

template <int L, int V, int VW, bool SIG>
hipError_t run_gate(const GateArgs& g, const GateLanes& n, const GateLanes& nw, const RouteWs& ws, int nblk, hipStream_t st) {
    size_t lds = select_lds(g.r.E, g.r.E);
    if (nblk <= 1) {
        lds += (size_t)g.r.E * 8 + 8;
        if (g.r.logits32) hipLaunchKernelGGL((k_gate_one<L, V, VW, true, SIG>), dim3(1), dim3(kThreads), lds, st, g, n, nw);
        else hipLaunchKernelGGL((k_gate_one<L, V, VW, false, SIG>), dim3(1), dim3(kThreads), lds, st, g, n, nw);
    } else {
        if (g.r.logits32)
            hipLaunchKernelGGL((k_gate_select<L, V, VW, true, SIG>), dim3(nblk), dim3(kThreads), lds, st, g, n, nw, ws);
        else
            hipLaunchKernelGGL((k_gate_select<L, V, VW, false, SIG>), dim3(nblk), dim3(kThreads), lds, st, g, n, nw, ws);
    }
    return hipGetLastError();
}

template <int L, int V, int VW>
hipError_t run_gate(const GateArgs& g, const GateLanes& n, const GateLanes& nw, const RouteWs& ws, int nblk, hipStream_t st) {
    return g.sigmoid ? run_gate<L, V, VW, true>(g, n, nw, ws, nblk, st) : run_gate<L, V, VW, false>(g, n, nw, ws, nblk, st);
}

template <int L, int V>
hipError_t run_bwd(const GateBwdArgs& p, hipStream_t st) {
    constexpr int kGroups = 256 / L;
    const int64_t blocks = (p.T + kGroups - 1) / kGroups;
    const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048));
    const size_t lds = sizeof(float) * kGroups * L * V;
#define FP8BS_BWD(F32, SIG) hipLaunchKernelGGL((k_gate_bwd<L, V, F32, SIG>), grid, dim3(256), lds, st, p)
    if (p.sigmoid) {
        if (p.logits32) FP8BS_BWD(true, true);
        else FP8BS_BWD(false, true);
    } else {
        if (p.logits32) FP8BS_BWD(true, false);
        else FP8BS_BWD(false, false);
    }
#undef FP8BS_BWD
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route_grouped(const GateArgs& g, void* wsp, hipStream_t st) {
    const int nblk = (int)((g.r.T + kTok - 1) / kTok);
    const RouteWs ws = route_workspace(g.r.T, g.r.E, wsp);
    const int per = g.r.E / g.groups;
    int lanes = 1;                                  // groups, rounded up to a power of two
    while (lanes < g.groups) lanes *= 2;
    const uintptr_t align = g.r.logits32 ? 16 : 8;
    const bool vec = per % 4 == 0 && g.r.ld % 4 == 0 && reinterpret_cast<uintptr_t>(g.r.logits) % align == 0;
    const bool vec_bias = per % 4 == 0 && reinterpret_cast<uintptr_t>(g.bias) % 16 == 0;
    auto deal = [&](int L) {
        GateLanes n{per, L / lanes, 0, vec, vec_bias};
        n.w = (per + n.q - 1) / n.q;
        if (per % 4 == 0) n.w = (n.w + 3) / 4 * 4;
        return n;
    };
    // sixteen lanes per token while they hold it in 16 values each, without scratch.
    // Beyond that every kernel spills registers: 64 lanes of 8 values 200 bytes a lane,
    // of 16 600, of 32 1450, and sixteen lanes of 32 more than they (16384 tokens of 512
    // experts 86 us, with 64 lanes 68; of 384 66, of 1024 165, where the plain router takes
    // 33, 33 and 59).  64 lanes hold every token in 32 (1024 experts in 2^k + 1 groups),
    // and a token that is selected again has them anyway.
    const GateLanes nw = deal(64);
    const bool wide = lanes > 16 || deal(16).w > 16;
    const GateLanes n = wide ? nw : deal(16);
    hipError_t e;
    if (wide) e = n.w <= 8 ? run_gate<64, 8, 8>(g, n, nw, ws, nblk, st)
                           : n.w <= 16 ? run_gate<64, 16, 16>(g, n, nw, ws, nblk, st)
                                       : run_gate<64, 32, 32>(g, n, nw, ws, nblk, st);
    else if (n.w <= 4) e = run_gate<16, 4, 4>(g, n, nw, ws, nblk, st);
    else if (n.w <= 8) e = run_gate<16, 8, 4>(g, n, nw, ws, nblk, st);
    else e = run_gate<16, 16, 4>(g, n, nw, ws, nblk, st);
    return e != hipSuccess || nblk <= 1 ? e : launch_route_rows(g.r, ws, st);
}

hipError_t launch_moe_route_grouped_bwd(const GateBwdArgs& p, hipStream_t st) {
    if (p.T == 0) return hipSuccess;
    if (p.E <= 64) return run_bwd<16, 4>(p, st);
    if (p.E <= 128) return run_bwd<16, 8>(p, st);
    if (p.E <= 256) return run_bwd<16, 16>(p, st);
    if (p.E <= 512) return run_bwd<64, 8>(p, st);
    return run_bwd<64, 16>(p, st);
}

hipError_t launch_moe_bias_update(float* bias, const int32_t* counts, int32_t E, float rate, hipStream_t st) {
    hipLaunchKernelGGL(k_bias_update, dim3(1), dim3(1024), 0, st, bias, counts, E, rate);
    return hipGetLastError();
}

}  // namespace fp8bs
