// Products of 8-bit integers with a scale per row of either operand: dense, and
// grouped over the experts of a MoE layer.
//
//   C[m, n] = sa[m] sb[n] sum_k a[m, k] b[n, k]
//
// The sum is exact: |a b| <= 2^14, so up to K = 131071 it stays inside the 32-bit
// accumulators of the integer matrix instructions, in any order.  It is converted
// to fp32 once and multiplied by sa, then sb (three roundings), then rounded to
// the output type: results do not depend on tile sizes or K ranges.
//
// Tiles (k_i8_tile).  A workgroup of four waves, two by two, computes 32 TN weight
// rows (n) x 32 TM activation rows (m); K advances in slices of 128 bytes that
// global_load_lds copies straight into LDS, two slices resident.  LDS rows are 128
// bytes with the 16-byte chunk c of row r at slot c ^ (r & 7), so the fragment
// reads of sixteen rows hit all banks.  Weight rows are the matrix instruction's
// first operand: a lane's four outputs are consecutive n of one m.
// With TM = TN = 8 a wave computes 128 x 128: per slice a compute unit reads 128 KB
// of fragments and writes 64 KB of copies (1536 cycles at 128 bytes each) beside
// 2048 cycles of matrix work, where eight waves of 64 x 128 would read 192 KB.
// With one wave per SIMD nothing else hides a wave's latencies, so it works half
// a slice ahead of itself: while one half's matrix instructions run, the other
// half's fragments are read.
#include <algorithm>

#include "device_common.h"
#include "internal.h"
#include "reduce.h"

namespace fp8bs {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int BK = 128;                 // K bytes per slice



struct I8Args {
    int32_t M, N, K;
    const uint8_t* a; int64_t lda; const float* sa;
    const uint8_t* b; int64_t ldb; int64_t b_sg; const float* sb; int64_t sb_sg;
    void* c; int64_t ldc;
    int32_t G; const int32_t* offsets; const int32_t* a_rows;
};

__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) { return (uint32_t)(uintptr_t)(const lds_u8*)p; }
__device__ __forceinline__ i32x4 lds_read16(uint32_t addr) {
    return *reinterpret_cast<const __attribute__((address_space(3))) i32x4*>((uintptr_t)addr);
}
__device__ __forceinline__ void lds_write16(uint32_t addr, i32x4 v) {
    *reinterpret_cast<__attribute__((address_space(3))) i32x4*>((uintptr_t)addr) = v;
}

// Lane l's 16 bytes at base + off land at LDS address dst + 16 l (dst
// wave-uniform).  Inline assembly, since the compiler cannot tell which slice a
// copy writes and would wait for all copies before each LDS read; the kernel
// waits itself: vmcnt on the issuing wave, then a barrier.
__device__ __forceinline__ void copy16(const void* base, uint32_t off, uint32_t dst) {
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(m0), "v"(off), "s"(base) : "memory", "m0");
}

__device__ __forceinline__ i32x4 mfma(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Four outputs of one row at columns n .. n + 3 (n < N, N % 8 == 0).
template <bool OUT32>
__device__ __forceinline__ void store4(void* c, int64_t at, const float (&v)[4]) {
    if (OUT32) *reinterpret_cast<float4*>(static_cast<float*>(c) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c) + at) =
             make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// Rows of a group's tile and where its operands are.
struct Tile {
    int32_t m0, m1, n0;                 // rows [m0, m1), first column
    const uint8_t* b; const float* sb;
};

// Row tiles of group g (0 past the last one).
template <int BM>
__device__ __forceinline__ int group_tiles(const I8Args& p, int g) {
    return g < p.G ? (p.offsets[g + 1] - p.offsets[g] + BM - 1) / BM : 0;
}

template <int TM, int TN, bool GROUPED, bool GATHER, bool OUT32>
__global__ void __launch_bounds__(256, (TM * TN > 16 ? 1 : 2)) k_i8_tile(I8Args p) {
    constexpr int BM = 32 * TM, BN = 32 * TN;
    constexpr int kABytes = BM * BK, kBuf = (BM + BN) * BK;       // a slice: activations, then weights
    constexpr int kCopyA = BM / 32, kCopyB = BN / 32;             // copies (8 rows each) per wave
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * kBuf];
    __shared__ int s_found[4];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & 1, wm = wave >> 1;
    const int q = lane >> 4, r16 = lane & 15;

    // ------------------------------------------------------------ which tile
    Tile t;
    const int ntn = (p.N + BN - 1) / BN;
    if (!GROUPED) {
        // consecutive tiles on one XCD (workgroups are dealt round-robin to the
        // eight), in groups of 8 row tiles that sweep n: the tiles an XCD runs at
        // a time share their panels in its L2
        const int ntm = (p.M + BM - 1) / BM, nblk = ntn * ntm, per = nblk / 8, bid = blockIdx.x;
        const int id = bid < per * 8 ? (bid % 8) * per + bid / 8 : bid;
        const int gsz = 8 * ntn, first = id / gsz * 8, rows = min(ntm - first, 8);
        t.m0 = (first + id % gsz % rows) * BM;
        t.m1 = min(p.M, t.m0 + BM);
        t.n0 = id % gsz / rows * BN;
        t.b = p.b;
        t.sb = p.sb;
    } else {
        // the list of all groups' row tiles, each with its ntn column tiles in
        // turn, in eight runs, one per XCD; the first wave adds up the groups'
        // tile counts
        if (wave == 0) {
            const int bid = blockIdx.x;
            int total = 0;
            for (int gb = 0; gb < p.G; gb += 64) total += group_tiles<BM>(p, gb + lane);
            total = (int)lane_value((uint32_t)wave_scan(total), 63);
            const int per = (total * ntn + 7) / 8, id = (bid % 8) * per + bid / 8;
            const int want = bid / 8 < per && id < total * ntn ? id / ntn : -1;
            if (lane == 0) { s_found[0] = -1; s_found[3] = id % ntn; }
            for (int gb = 0, carry = 0; gb < p.G && carry <= want; gb += 64) {
                const int g = gb + lane, cnt = group_tiles<BM>(p, g), sum = wave_scan(cnt), start = carry + sum - cnt;
                if (want >= start && want < start + cnt) {
                    s_found[0] = g;
                    s_found[1] = p.offsets[g] + (want - start) * BM;
                    s_found[2] = p.offsets[g + 1];
                }
                carry += (int)lane_value((uint32_t)sum, 63);
            }
        }
        __syncthreads();
        const int g = __builtin_amdgcn_readfirstlane(s_found[0]);
        if (g < 0) return;                          // uniform: behind the last tile
        t.m0 = __builtin_amdgcn_readfirstlane(s_found[1]);
        t.m1 = min(__builtin_amdgcn_readfirstlane(s_found[2]), t.m0 + BM);
        t.n0 = __builtin_amdgcn_readfirstlane(s_found[3]) * BN;
        t.b = p.b + (int64_t)g * p.b_sg;
        t.sb = p.sb + (int64_t)g * p.sb_sg;
    }

    // ---------------------------------------------------------------- copies
    // Copy j of a wave brings tile rows 8 (wave + 4 j) + lane / 8; rows past the
    // tile repeat its last row, their outputs are not stored.
    uint32_t offA[kCopyA], offB[kCopyB];
    const int sub = lane >> 3, chunk = (lane & 7) ^ sub;
    const int ntail = p.K % BK / 16;                // chunks of the last slice, 0: all eight
    const int nk = (p.K + BK - 1) / BK;
#pragma unroll
    for (int j = 0; j < kCopyA; ++j) {
        int m = min(t.m0 + 8 * (wave + 4 * j) + sub, t.m1 - 1);
        if (GATHER) m = p.a_rows[m];
        offA[j] = (uint32_t)((int64_t)m * p.lda + chunk * 16);
    }
#pragma unroll
    for (int j = 0; j < kCopyB; ++j)
        offB[j] = (uint32_t)((int64_t)min(t.n0 + 8 * (wave + 4 * j) + sub, p.N - 1) * p.ldb + chunk * 16);
    const uint32_t lds0 = lds_addr(smem);
    auto copies = [&](int kb) {
        const uint32_t dst = lds0 + (kb & 1) * kBuf;
        // the last slice's missing chunks are read from its first one (in bounds)
        // and cleared in LDS
        const uint32_t back = kb == nk - 1 && ntail && chunk >= ntail ? (uint32_t)chunk * 16 : 0u;
#pragma unroll
        for (int j = 0; j < kCopyA; ++j)
            copy16(p.a + (int64_t)kb * BK, offA[j] - back, dst + (wave + 4 * j) * 8 * BK);
#pragma unroll
        for (int j = 0; j < kCopyB; ++j)
            copy16(t.b + (int64_t)kb * BK, offB[j] - back, dst + kABytes + (wave + 4 * j) * 8 * BK);
    };
    // slice kb has landed for every wave, and every wave has read slice kb - 1
    auto arrive = [&](int kb) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (kb == nk - 1 && ntail) {
            // zeros in the activations are enough: a zero times any code is zero
            for (int i = threadIdx.x; i < BM * 8; i += 256) {
                const int r = i >> 3, c = i & 7;
                if (c >= ntail) lds_write16(lds0 + (kb & 1) * kBuf + r * BK + ((c ^ (r & 7)) << 4), i32x4{0, 0, 0, 0});
            }
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
    };
    // Fragments of half h of slice kb: chunk q + 4 h of each row.
    auto read_half = [&](int kb, int h, i32x4 (&fa)[TM], i32x4 (&fb)[TN]) {
        const uint32_t at = lds0 + (kb & 1) * kBuf + r16 * BK + (((q + 4 * h) ^ (r16 & 7)) << 4);
        uint32_t aa = at + wm * 16 * TM * BK, bb = at + kABytes + wn * 16 * TN * BK;
        asm volatile("" : "+v"(aa), "+v"(bb));      // one address each, the tiles as offsets
#pragma unroll
        for (int i = 0; i < TN; ++i) fb[i] = lds_read16(bb + i * 16 * BK);
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[i] = lds_read16(aa + i * 16 * BK);
    };

    i32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    auto multiply = [&](const i32x4 (&fa)[TM], const i32x4 (&fb)[TN]) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = mfma(fb[i], fa[j], acc[i][j]);
    };

    if (nk > 0) {
        i32x4 fa0[TM], fb0[TN], fa1[TM], fb1[TN];
        copies(0);
        arrive(0);
        if (nk > 1) copies(1);
        read_half(0, 0, fa0, fb0);
        for (int kb = 0; kb < nk; ++kb) {
            read_half(kb, 1, fa1, fb1);
            multiply(fa0, fb0);
            if (kb + 1 < nk) {
                arrive(kb + 1);
                if (kb + 2 < nk) copies(kb + 2);
                read_half(kb + 1, 0, fa0, fb0);
            }
            multiply(fa1, fb1);
        }
    }

    // -------------------------------------------------------------- epilogue
    const int nw = t.n0 + wn * 16 * TN + 4 * q, mw = t.m0 + wm * 16 * TM + r16;
    float sam[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        int m = min(mw + 16 * j, t.m1 - 1);
        if (GATHER) m = p.a_rows[m];
        sam[j] = p.sa[m];
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        const int n = nw + 16 * i;
        float sbn[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) sbn[r] = t.sb[min(n + r, p.N - 1)];
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int m = mw + 16 * j;
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = (float)acc[i][j][r] * sam[j] * sbn[r];
            if (m < t.m1 && n < p.N) store4<OUT32>(p.c, (int64_t)m * p.ldc + n, v);
        }
    }
}

// Few rows (decode): the weights are read once, straight into registers, by waves
// that split K and meet in LDS.  A workgroup takes 16 NT weight rows; a wave
// takes every W-th run of 64 bytes of K and feeds it to NT x MT matrix
// instructions.  Grouped: grid row y is a group; its rows go in passes of 16 MT.
template <int MT, int NT, int W, bool GROUPED, bool GATHER, bool OUT32>
__global__ void __launch_bounds__(64 * W) k_i8_stream(I8Args p) {
    constexpr int kOut = NT * MT * 64;              // 16-byte pieces of a wave's partial sums
    __shared__ __attribute__((aligned(16))) i32x4 part[W][kOut];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, r16 = lane & 15;
    const int n0 = blockIdx.x * 16 * NT;
    int m0 = 0, m1 = p.M;
    const uint8_t* b = p.b;
    const float* sb = p.sb;
    if (GROUPED) {
        m0 = p.offsets[blockIdx.y];
        m1 = p.offsets[blockIdx.y + 1];
        b += (int64_t)blockIdx.y * p.b_sg;
        sb += (int64_t)blockIdx.y * p.sb_sg;
    }
    const uint8_t* brow[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) brow[i] = b + (int64_t)min(n0 + 16 * i + r16, p.N - 1) * p.ldb + 16 * q;
    const int steps = (p.K + 63) / 64;
    for (; m0 < m1; m0 += 16 * MT) {
        const uint8_t* arow[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            int m = min(m0 + 16 * j + r16, m1 - 1);
            if (GATHER) m = p.a_rows[m];
            arow[j] = p.a + (int64_t)m * p.lda + 16 * q;
        }
        i32x4 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
        constexpr int U = 4;                        // runs in flight
        for (int s = wave; s < steps; s += W * U) {
            i32x4 fb[U][NT], fa[U][MT];
            const i32x4 zero = {0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // past K: nothing is read, and zeros add nothing
                const int k = (s + u * W) * 64;
                const bool in = k + 16 * q < p.K;
#pragma unroll
                for (int i = 0; i < NT; ++i) fb[u][i] = in ? *reinterpret_cast<const i32x4*>(brow[i] + k) : zero;
#pragma unroll
                for (int j = 0; j < MT; ++j) fa[u][j] = in ? *reinterpret_cast<const i32x4*>(arow[j] + k) : zero;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < MT; ++j) acc[i][j] = mfma(fb[u][i], fa[u][j], acc[i][j]);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) part[wave][(i * MT + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        for (int o = threadIdx.x; o < kOut; o += 64 * W) {
            i32x4 v = part[0][o];
#pragma unroll
            for (int w = 1; w < W; ++w) v += part[w][o];
            const int l = o & 63, i = (o >> 6) / MT, j = (o >> 6) % MT;
            const int m = m0 + 16 * j + (l & 15), n = n0 + 16 * i + 4 * (l >> 4);
            if (m < m1 && n < p.N) {
                const float sam = p.sa[GATHER ? p.a_rows[m] : m];
                const float f[4] = {(float)v[0] * sam * sb[n], (float)v[1] * sam * sb[n + 1],
                                    (float)v[2] * sam * sb[n + 2], (float)v[3] * sam * sb[n + 3]};
                store4<OUT32>(p.c, (int64_t)m * p.ldc + n, f);
            }
        }
        __syncthreads();
    }
}

template <int TM, int TN, bool GROUPED, bool GATHER>
hipError_t tile(const I8Args& p, bool out32, hipStream_t st) {
    constexpr int BM = 32 * TM, BN = 32 * TN;
    const int64_t ntn = (p.N + BN - 1) / BN;
    int64_t blocks = ((int64_t)p.M + BM - 1) / BM * ntn;
    if (GROUPED) blocks = (((int64_t)p.M / BM + std::min<int64_t>(p.G, p.M)) * ntn + 7) / 8 * 8;   // at most this many tiles
    if (out32) hipLaunchKernelGGL((k_i8_tile<TM, TN, GROUPED, GATHER, true>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    else hipLaunchKernelGGL((k_i8_tile<TM, TN, GROUPED, GATHER, false>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    return hipGetLastError();
}

template <int MT, int NT, int W, bool GROUPED, bool GATHER>
hipError_t stream(const I8Args& p, bool out32, hipStream_t st) {
    const dim3 grid((unsigned)((p.N + 16 * NT - 1) / (16 * NT)), (unsigned)(GROUPED ? p.G : 1));
    if (out32) hipLaunchKernelGGL((k_i8_stream<MT, NT, W, GROUPED, GATHER, true>), grid, dim3(64 * W), 0, st, p);
    else hipLaunchKernelGGL((k_i8_stream<MT, NT, W, GROUPED, GATHER, false>), grid, dim3(64 * W), 0, st, p);
    return hipGetLastError();
}

template <bool GROUPED, bool GATHER>
hipError_t launch(const I8Args& p, bool out32, hipStream_t st) {
    // rows per product, or on average per group
    const int64_t rows = GROUPED ? ((int64_t)p.M + p.G - 1) / p.G : p.M;
    if (rows <= 16) return stream<1, 1, 8, GROUPED, GATHER>(p, out32, st);
    if (rows <= 64) return stream<4, 1, 8, GROUPED, GATHER>(p, out32, st);
    const int64_t big = ((int64_t)p.M + 255) / 256 * ((p.N + 255) / 256);
    if (big >= 128) return tile<8, 8, GROUPED, GATHER>(p, out32, st);
    return tile<4, 4, GROUPED, GATHER>(p, out32, st);
}

}  // namespace

hipError_t launch_i8_gemm(const I8GemmArgs& g, hipStream_t st) {
    if (g.M == 0 || g.N == 0) return hipSuccess;
    const I8Args p{(int32_t)g.M, (int32_t)g.N, (int32_t)g.K, g.a, g.lda, g.sa, g.b, g.ldb, g.b_sg, g.sb, g.sb_sg,
                   g.c, g.ldc, g.G, g.offsets, g.a_rows};
    if (g.G == 0) return launch<false, false>(p, g.out_f32, st);
    return g.a_rows ? launch<true, true>(p, g.out_f32, st) : launch<true, false>(p, g.out_f32, st);
}

}  // namespace fp8bs
