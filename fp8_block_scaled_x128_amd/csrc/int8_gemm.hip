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
// Tiles (k_i8_tile).  A workgroup of four waves, two by two, computes 64 TN weight
// rows (n) x 64 TM activation rows (m) with the 32 x 32 x 32 matrix instruction, which
// reaches 5.0 POPS on 256 units where 16 x 16 x 64 reaches 2.5 (3.8 on random codes:
// the clock falls with the power they draw).  K advances in slices of 128 bytes that
// global_load_lds copies straight into LDS, two slices of activations and three of
// weights resident.  LDS rows are 128 bytes with the 16-byte chunk c of row r at slot
// c ^ (r & 7), so that fragment reads hit all banks.  Weight rows are the matrix
// instruction's first operand: a lane's outputs are runs of four consecutive n of one
// m.  With TM = TN = 4 a wave holds 256 sums, 128 x 128 outputs: per slice a compute
// unit reads 128 KB of fragments and writes 64 KB of copies beside 2048 cycles of
// matrix work.  One such workgroup fills a unit's LDS, so nothing else hides a wave's
// latencies: it works a slice ahead of itself.  4096 x 2560 by 9728: 117 to 136 us by
// the card at hand, 1.5 to 1.7 POPS; 131072 expert rows of 2048 by 1536 495 to 531, 1.55
// to 1.67.  Counters of the former (608 tiles, 2.4 rounds of 256 units): 250000 cycles,
// on random codes at 2.1 GHz and on zeros at 2.5 (100 us), so power costs a sixth of the
// clock and nothing else; a tile takes 74000 of them, of which 41000 are matrix work and
// 30000 waits, and LDS is in use for 51000 of the 250000.  What bounds it are the waits of
// the one workgroup that a unit holds (a tile's first copies, its barriers, its epilogue)
// and the third round, not LDS bandwidth.  TM = TN = 2 puts two workgroups on a unit and
// takes products with fewer tiles; TM = 1, TN = 2 the K ranges and small groups.
// Few rows are bound by the weights' way from memory, see below.
#include <algorithm>
#include <utility>

#include "int8_common.h"
#include "internal.h"
#include "reduce.h"

namespace fp8bs {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int BK = 128;                 // K bytes per slice
constexpr int kCUs = 256;

struct I8Args {
    int32_t M, N, K;
    const uint8_t* a; int64_t lda; const float* sa;
    const uint8_t* b; int64_t ldb; int64_t b_sg; const float* sb; int64_t sb_sg;
    void* c; int64_t ldc;
    int32_t G; const int32_t* offsets; const int32_t* a_rows;
    int32_t splits;                     // dense: K ranges, one per grid row (OUT_SUMS)
};

// What a tile leaves: scaled outputs, or the sums themselves as [splits][M][N].
enum { OUT_BF16, OUT_FP32, OUT_SUMS };

__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) { return (uint32_t)(uintptr_t)(const lds_u8*)p; }
__device__ __forceinline__ i32x4 lds_read16(uint32_t addr) {
    return *reinterpret_cast<const __attribute__((address_space(3))) i32x4*>((uintptr_t)addr);
}
__device__ __forceinline__ void lds_write16(uint32_t addr, i32x4 v) {
    *reinterpret_cast<__attribute__((address_space(3))) i32x4*>((uintptr_t)addr) = v;
}

// Lane l's 16 bytes at base + off land at LDS address dst + AT + 16 l (dst
// wave-uniform).  Inline assembly, since the compiler cannot tell which slice a
// copy writes and would wait for all copies before each LDS read; the kernel
// waits itself: vmcnt on the issuing wave, then a barrier.
template <int AT>
__device__ __forceinline__ void copy16(const void* base, uint32_t off, uint32_t dst) {
    asm volatile("s_add_u32 m0, %0, %c3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(dst), "v"(off), "s"(base), "n"(AT) : "memory", "scc", "m0");
}
// The same where `go` (uniform) is not 0.  The branch is the assembly's own: a slice
// stays one basic block.
template <int AT>
__device__ __forceinline__ void copy16_if(uint32_t go, const void* base, uint32_t off, uint32_t dst) {
    asm volatile("s_cmp_eq_u32 %4, 0\n\ts_cbranch_scc1 .Lskip%=\n\ts_add_u32 m0, %0, %c3\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %1, %2\n.Lskip%=:"
                 :: "s"(dst), "v"(off), "s"(base), "n"(AT), "s"(go) : "memory", "scc", "m0");
}
// All but the last N1 + N2 copies of this wave have landed where `one` and `two` are
// not 0, the last N1 with `one` alone, all without.
template <int N1, int N2>
__device__ __forceinline__ void wait_copies(uint32_t one, uint32_t two) {
    asm volatile("s_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 .Lall%=\n\ts_cmp_eq_u32 %1, 0\n\ts_cbranch_scc1 .Lone%=\n\t"
                 "s_waitcnt vmcnt(%c3)\n\ts_branch .Ldone%=\n.Lone%=:\n\ts_waitcnt vmcnt(%c2)\n\ts_branch .Ldone%=\n"
                 ".Lall%=:\n\ts_waitcnt vmcnt(0)\n.Ldone%=:"
                 :: "s"(one), "s"(two), "n"(N1), "n"(N1 + N2) : "memory", "scc");
}

__device__ __forceinline__ i32x4 mfma(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// A wave's 256 sums in accumulation registers of our own choice, a0 to a255, which
// take one half of its registers whole.  The compiler is told that they are used
// (ACC_IN_USE), which reserves that half and keeps its values out of it at that point;
// that it puts none there later, values or spills, is no promise of the clobber list but
// of the 214 registers that the kernels need of the other half, and the build checks it
// on the listing.  Left to allocate the sums itself it copies them between the two halves
// of the register file, 388 copies beside 128 matrix instructions in two slices.  Only
// the functions below touch them; the waits that the compiler adds around matrix
// instructions are theirs.
#define FP8BS_ACC_IN_USE() asm volatile("" ::: \
        "a0", "a1", "a2", "a3", "a4", "a5", "a6", "a7", "a8", "a9", "a10", "a11", "a12", "a13", "a14", "a15", \
        "a16", "a17", "a18", "a19", "a20", "a21", "a22", "a23", "a24", "a25", "a26", "a27", "a28", "a29", "a30", "a31", \
        "a32", "a33", "a34", "a35", "a36", "a37", "a38", "a39", "a40", "a41", "a42", "a43", "a44", "a45", "a46", "a47", \
        "a48", "a49", "a50", "a51", "a52", "a53", "a54", "a55", "a56", "a57", "a58", "a59", "a60", "a61", "a62", "a63", \
        "a64", "a65", "a66", "a67", "a68", "a69", "a70", "a71", "a72", "a73", "a74", "a75", "a76", "a77", "a78", "a79", \
        "a80", "a81", "a82", "a83", "a84", "a85", "a86", "a87", "a88", "a89", "a90", "a91", "a92", "a93", "a94", "a95", \
        "a96", "a97", "a98", "a99", "a100", "a101", "a102", "a103", "a104", "a105", "a106", "a107", "a108", "a109", "a110", "a111", \
        "a112", "a113", "a114", "a115", "a116", "a117", "a118", "a119", "a120", "a121", "a122", "a123", "a124", "a125", "a126", "a127", \
        "a128", "a129", "a130", "a131", "a132", "a133", "a134", "a135", "a136", "a137", "a138", "a139", "a140", "a141", "a142", "a143", \
        "a144", "a145", "a146", "a147", "a148", "a149", "a150", "a151", "a152", "a153", "a154", "a155", "a156", "a157", "a158", "a159", \
        "a160", "a161", "a162", "a163", "a164", "a165", "a166", "a167", "a168", "a169", "a170", "a171", "a172", "a173", "a174", "a175", \
        "a176", "a177", "a178", "a179", "a180", "a181", "a182", "a183", "a184", "a185", "a186", "a187", "a188", "a189", "a190", "a191", \
        "a192", "a193", "a194", "a195", "a196", "a197", "a198", "a199", "a200", "a201", "a202", "a203", "a204", "a205", "a206", "a207", \
        "a208", "a209", "a210", "a211", "a212", "a213", "a214", "a215", "a216", "a217", "a218", "a219", "a220", "a221", "a222", "a223", \
        "a224", "a225", "a226", "a227", "a228", "a229", "a230", "a231", "a232", "a233", "a234", "a235", "a236", "a237", "a238", "a239", \
        "a240", "a241", "a242", "a243", "a244", "a245", "a246", "a247", "a248", "a249", "a250", "a251", "a252", "a253", "a254", "a255")
template <int I>
__device__ __forceinline__ void acc_mfma(i32x4 a, i32x4 b) {
    asm volatile("v_mfma_i32_32x32x32_i8 a[%c0:%c1], %2, %3, a[%c0:%c1]" :: "n"(I), "n"(I + 15), "v"(a), "v"(b));
}
template <int I>
__device__ __forceinline__ void acc_zero() {
    asm volatile("v_accvgpr_write_b32 a[%c0], 0" :: "n"(I));
}
template <int I>
__device__ __forceinline__ int acc_read() {
    int v;
    asm volatile("v_accvgpr_read_b32 %0, a[%c1]" : "=v"(v) : "n"(I));
    return v;
}
// Until the last matrix instruction's sums are there.
__device__ __forceinline__ void acc_wait() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

template <int N, class F, int... I>
__device__ __forceinline__ void unrolled(F f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unrolled(F f) { unrolled<N>(f, std::make_integer_sequence<int, N>{}); }

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

// Tile `bid` of a product, or K range blockIdx.y of it (OUT_SUMS).
template <int TM, int TN, bool GROUPED, bool GATHER, int OUT>
__device__ __forceinline__ void tile_product(const I8Args& p, const int bid, uint8_t* smem) {
    constexpr int BM = 64 * TM, BN = 64 * TN;
    constexpr int kABytes = BM * BK, kBBytes = BN * BK;
    int* s_found = reinterpret_cast<int*>(smem);    // before the first copy

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & 1, wm = wave >> 1;
    const int hi = lane >> 5, r32 = lane & 31;

    // ------------------------------------------------------------ which tile
    Tile t;
    const int ntn = (p.N + BN - 1) / BN;
    if (!GROUPED) {
        // consecutive tiles on one XCD (workgroups are dealt round-robin to the
        // eight), in groups of 8 row tiles that sweep n: the tiles an XCD runs at
        // a time share their panels in its L2
        const int ntm = (p.M + BM - 1) / BM, nblk = ntn * ntm, per = nblk / 8;
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
        __syncthreads();                            // s_found's place is copied to
    }

    // The output's scales, loaded ahead of everything: lane l has row l % 32 of each
    // activation tile and two of the wave's columns.
    const int mw = t.m0 + wm * 32 * TM + r32, nw = t.n0 + wn * 32 * TN;
    float sam[TM], sbv[TN / 2];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        int m = min(mw + 32 * j, t.m1 - 1);
        if (GATHER) m = p.a_rows[m];
        sam[j] = p.sa[m];
    }
#pragma unroll
    for (int i = 0; i < TN / 2; ++i) sbv[i] = t.sb[min(nw + 64 * i + lane, p.N - 1)];

    // ---------------------------------------------------------------- copies
    // Copy j of a wave brings rows 8 (wave + 4 j) + lane / 8 of a tile; rows past it
    // repeat its last row, their outputs are not stored.
    uint32_t offA[2 * TM], offB[2 * TN];
    const int sub = lane >> 3, chunk = (lane & 7) ^ sub;
    int ntail = p.K % BK / 16;                      // chunks of the last slice, 0: all eight
    int nk = (p.K + BK - 1) / BK;
    const uint8_t* pa = p.a;
    if (OUT == OUT_SUMS) {
        // this grid row's slices: the first nk % splits ranges have one more
        const int y = blockIdx.y, per = nk / p.splits, more = nk % p.splits, k0 = y * per + min(y, more);
        nk = per + (y < more);
        if (y != p.splits - 1) ntail = 0;
        pa += (int64_t)k0 * BK;
        t.b += (int64_t)k0 * BK;
    }
#pragma unroll
    for (int j = 0; j < 2 * TM; ++j) {
        int m = min(t.m0 + 8 * (wave + 4 * j) + sub, t.m1 - 1);
        if (GATHER) m = p.a_rows[m];
        offA[j] = (uint32_t)((int64_t)m * p.lda + chunk * 16);
    }
#pragma unroll
    for (int j = 0; j < 2 * TN; ++j)
        offB[j] = (uint32_t)((int64_t)min(t.n0 + 8 * (wave + 4 * j) + sub, p.N - 1) * p.ldb + chunk * 16);
    // activations of slice kb in one of two buffers, weights in one of three
    const uint32_t lds0 = lds_addr(smem);
    auto bufA = [&](int kb) { return lds0 + (uint32_t)(kb & 1) * kABytes; };
    auto bufB = [&](int kb) { return lds0 + 2 * kABytes + (uint32_t)(kb % 3) * kBBytes; };
    // The last slice's missing chunks are read from its first one (in bounds), by
    // offsets moved back before its copies, and cleared in LDS.
    const uint32_t back = ntail && chunk >= ntail ? (uint32_t)chunk * 16 : 0u;
    const uint32_t mine = (uint32_t)wave * 8 * BK;  // a wave's first copy in a buffer
    auto copies = [&](int kb, bool acts, bool weights) {
        if (kb == nk - 1 && ntail) {
#pragma unroll
            for (int j = 0; j < 2 * TM; ++j) offA[j] -= acts ? back : 0u;
#pragma unroll
            for (int j = 0; j < 2 * TN; ++j) offB[j] -= weights ? back : 0u;
        }
        unrolled<2 * TM>([&](auto j) {
            constexpr int J = decltype(j)::value;
            if (acts) copy16<32 * J * BK>(pa + (int64_t)kb * BK, offA[J], bufA(kb) + mine);
        });
        unrolled<2 * TN>([&](auto j) {
            constexpr int J = decltype(j)::value;
            if (weights) copy16<32 * J * BK>(t.b + (int64_t)kb * BK, offB[J], bufB(kb) + mine);
        });
    };
    // zeros in the last slice's missing activations are enough: zero times any code
    auto clear = [&](int kb) {
        for (int i = threadIdx.x; i < BM * 8; i += 256) {
            const int r = i >> 3, c = i & 7;
            if (c >= ntail) lds_write16(bufA(kb) + r * BK + ((c ^ (r & 7)) << 4), i32x4{0, 0, 0, 0});
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    // This lane's addresses of a wave's first 32 rows: the 16 bytes of matrix
    // instruction u (32 of the slice's 128) are chunk 2 u + lane / 32; later rows are
    // constant offsets.
    struct Frag { uint32_t at[4]; };
    auto frag = [&](uint32_t rows) {
        const uint32_t at = rows + r32 * BK;
        Frag f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            f.at[u] = at + (((2 * u + hi) ^ (r32 & 7)) << 4);
            asm volatile("" : "+v"(f.at[u]));
        }
        return f;
    };

    // sums of weight tile i and activation tile j (32 x 32): accumulation registers
    // from 16 (i TM + j) on, or the compiler's where two workgroups share a compute unit
    constexpr bool kAcc = TM * TN > 4;
    i32x16 own[kAcc ? 1 : TN * TM];
    if constexpr (kAcc) {
        FP8BS_ACC_IN_USE();
        unrolled<16 * TN * TM>([](auto i) { acc_zero<decltype(i)::value>(); });
    } else {
#pragma unroll
        for (int i = 0; i < TN * TM; ++i) own[i] = i32x16{};
    }
    auto add = [&](auto at, i32x4 b, i32x4 a) {
        constexpr int I = decltype(at)::value;
        if constexpr (kAcc) acc_mfma<16 * I>(b, a);
        else own[I] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, own[I], 0, 0, 0);
    };

    // One slice, in 2 TN steps of half a weight tile each (64 of its bytes): its
    // activations are in `fa`, the first step's weights in fb[0].  Meanwhile the next
    // slice's activations go to `na` (steps before kMid), the next step's weights to
    // the other fb, and the copies of the weights two and the activations three slices
    // ahead to LDS.  At kMid every wave has read the next activations,
    // so their buffer is free; before the last step the next slice's weights and the
    // activations after it have landed.
    // A wave alone on its SIMD issues an instruction every four cycles or so and a
    // matrix instruction runs for 32: whatever else there is stands between matrix
    // instructions, one thing after each (in one place per step it left the matrix
    // unit idle for a third of the time: 3240 cycles a slice, not 2048).
    constexpr int kSteps = 2 * TN, kMid = TN, kReads = 4, kSpan = 2 * TM;
    constexpr int kStepB = (2 * TN + kMid - 1) / kMid, kStepA = (2 * TM + kSteps - kMid - 2) / (kSteps - kMid - 1);
    static_assert(4 * TM <= kReads * kMid, "the next activations are read before kMid");
    i32x4 fb[2][2];
    uint32_t wb = 0, wb1 = 1, wb2 = 2;              // weight buffers of this slice and the next two
    auto slice = [&](int kb, const i32x4 (&fa)[4][TM], i32x4 (&na)[4][TM]) {
        const uint32_t two = __builtin_amdgcn_readfirstlane(max(nk - kb - 2, 0)), three = __builtin_amdgcn_readfirstlane(max(nk - kb - 3, 0));
        if (ntail) {
            if (kb + 2 == nk) clear(kb + 1);
            if (kb + 3 == nk) {
#pragma unroll
                for (int j = 0; j < 2 * TN; ++j) offB[j] -= back;
            }
            if (kb + 4 == nk) {
#pragma unroll
                for (int j = 0; j < 2 * TM; ++j) offA[j] -= back;
            }
        }
        const uint32_t rowsB = lds0 + 2 * kABytes + wn * 32 * TN * BK;
        const Frag ha = frag(bufA(kb + 1) + wm * 32 * TM * BK), hb = frag(rowsB + wb * kBBytes);
        const Frag hn = frag(rowsB + wb1 * kBBytes);
        const uint8_t* baseA = pa + (int64_t)(kb + 3) * BK;
        const uint8_t* baseB = t.b + (int64_t)(kb + 2) * BK;
        const uint32_t dstA = bufA(kb + 1) + mine, dstB = lds0 + 2 * kABytes + wb2 * kBBytes + mine;
        unrolled<kSteps>([&](auto step) {
            constexpr int i = decltype(step)::value;
            if constexpr (i == kMid) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            // copies of the next weights and of the activations after them are older
            // than the last 2 (TM + TN) or fewer
            if constexpr (i == kSteps - 1) {
                wait_copies<2 * TN, 2 * TM>(two, three);
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            }
            i32x4 (&nb)[2] = fb[(i + 1) & 1];
            unrolled<kSpan>([&](auto vv) {
                constexpr int v = decltype(vv)::value, u = v / TM;
                add(std::integral_constant<int, i / 2 * TM + v % TM>{}, fb[i & 1][u], fa[2 * (i % 2) + u][v % TM]);
                // reads spread over the span: the next weights, then the next activations
                constexpr int kAll = 2 + (i < kMid ? kReads : 0), kOver = kAll > kSpan ? kAll : kSpan;
                unrolled<kAll>([&](auto xx) {
                    constexpr int x = decltype(xx)::value, r = i * kReads + x - 2;
                    if constexpr (x * kSpan / kOver == v) {
                        if constexpr (x >= 2) {
                            if constexpr (r < 4 * TM) na[r / TM][r % TM] = lds_read16(ha.at[r / TM] + (r % TM) * 32 * BK);
                        } else if constexpr (i < kSteps - 1) {
                            nb[x] = lds_read16(hb.at[2 * ((i + 1) % 2) + x] + (i + 1) / 2 * 32 * BK);
                        } else {
                            nb[x] = lds_read16(hn.at[x]);    // (after the last slice: whatever is there, not used)
                        }
                    }
                });
                constexpr int c = kSpan - 1 - v;    // copies from the span's end on
                if constexpr (i < kMid && c < kStepB) {
                    constexpr int j = i * kStepB + c;
                    if constexpr (j < 2 * TN) copy16_if<32 * j * BK>(two, baseB, offB[j], dstB);
                }
                if constexpr (i >= kMid && i < kSteps - 1 && c < kStepA) {
                    constexpr int j = (i - kMid) * kStepA + c;
                    if constexpr (j < 2 * TM) copy16_if<32 * j * BK>(three, baseA, offA[j], dstA);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        });
        const uint32_t w = wb;
        wb = wb1;
        wb1 = wb2;
        wb2 = w;
    };

    if (nk > 0) {
        i32x4 fa[4][TM], na[4][TM];
        copies(0, true, true);
        if (nk > 1) {
            copies(1, true, true);
            asm volatile("s_waitcnt vmcnt(%c0)\n\ts_barrier" :: "n"(2 * TN) : "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        }
        if (ntail && nk == 1) clear(0);
        const Frag ha = frag(bufA(0) + wm * 32 * TM * BK), hb = frag(bufB(0) + wn * 32 * TN * BK);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (u < 2) fb[0][u] = lds_read16(hb.at[u]);
#pragma unroll
            for (int j = 0; j < TM; ++j) fa[u][j] = lds_read16(ha.at[u] + j * 32 * BK);
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (nk > 2) copies(2, true, false);
        for (int kb = 0;; kb += 2) {
            slice(kb, fa, na);
            if (kb + 1 >= nk) break;
            slice(kb + 1, na, fa);
            if (kb + 2 >= nk) break;
        }
    }

    // -------------------------------------------------------------- epilogue
    // Sum r of a 32 x 32 tile is column 8 (r / 4) + 4 (lane / 32) + r % 4.  The
    // columns' scales go through LDS, 32 TN floats of the wave's own (the last barrier
    // left every buffer free); of two runs of eight bf16 columns the lanes' halves
    // trade their halves, so that each lane stores sixteen bytes of its row.
    float* sbl = reinterpret_cast<float*>(smem) + wave * 32 * TN;
#pragma unroll
    for (int i = 0; i < TN / 2; ++i) sbl[64 * i + lane] = sbv[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if constexpr (kAcc) acc_wait();
    unrolled<2 * TN>([&](auto step) {
        constexpr int i = decltype(step)::value / 2, g = decltype(step)::value % 2 * 2;     // runs g, g + 1 of tile i
        const float4 s0 = *reinterpret_cast<const float4*>(sbl + 32 * i + 8 * g + 4 * hi);
        const float4 s1 = *reinterpret_cast<const float4*>(sbl + 32 * i + 8 * g + 8 + 4 * hi);
        const float sbn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
        unrolled<TM>([&](auto col) {
            constexpr int j = decltype(col)::value, at = i * TM + j;
            const int m = mw + 32 * j, n = nw + 32 * i + 8 * g;
            float v[8];
            int sum[8];
            unrolled<8>([&](auto rr) {
                constexpr int r = decltype(rr)::value;
                if constexpr (kAcc) sum[r] = acc_read<16 * at + 4 * g + r>();
                else sum[r] = own[at][4 * g + r];
                v[r] = (float)sum[r] * sam[j] * sbn[r];
            });
            if constexpr (OUT == OUT_SUMS) {
                int32_t* c = static_cast<int32_t*>(p.c) + ((int64_t)blockIdx.y * p.M + m) * p.N + n + 4 * hi;
                if (m < t.m1 && n < p.N) *reinterpret_cast<i32x4*>(c) = i32x4{sum[0], sum[1], sum[2], sum[3]};
                if (m < t.m1 && n + 8 < p.N) *reinterpret_cast<i32x4*>(c + 8) = i32x4{sum[4], sum[5], sum[6], sum[7]};
            } else if constexpr (OUT == OUT_FP32) {
                float* c = static_cast<float*>(p.c) + (int64_t)m * p.ldc + n + 4 * hi;
                if (m < t.m1 && n < p.N) *reinterpret_cast<float4*>(c) = make_float4(v[0], v[1], v[2], v[3]);
                if (m < t.m1 && n + 8 < p.N) *reinterpret_cast<float4*>(c + 8) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                const auto lo = __builtin_amdgcn_permlane32_swap(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[4], v[5]), false, false);
                const auto up = __builtin_amdgcn_permlane32_swap(pack_bf16x2(v[2], v[3]), pack_bf16x2(v[6], v[7]), false, false);
                if (m < t.m1 && n + 8 * hi < p.N)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.c) + (int64_t)m * p.ldc + n + 8 * hi) =
                        make_uint4(lo[0], up[0], lo[1], up[1]);
            }
        });
    });
}

template <int TM, int TN>
constexpr int kTileLds = (2 * TM + 3 * TN) * 64 * BK;
template <int TM, int TN, bool GROUPED, bool GATHER, int OUT>
__global__ void __launch_bounds__(256, (TM * TN > 4 ? 1 : 2)) k_i8_tile(I8Args p) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[kTileLds<TM, TN>];
    tile_product<TM, TN, GROUPED, GATHER, OUT>(p, blockIdx.x, smem);
}

// Two products in one launch, the first's tiles (blocks below `first`, the longer K)
// before the second's, so that the second's fill the units that the first leaves idle:
// the gradients of 4096 x 2560 by 9728, 160 tiles of 76 slices and 380 of 32 on 256
// units, 191 to 210 us where one after the other took 250.
struct I8Pair {
    I8Args p[2];
    int32_t first;
};
template <int TM, int TN>
__global__ void __launch_bounds__(256, (TM * TN > 4 ? 1 : 2)) k_i8_tile_pair(I8Pair g) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[kTileLds<TM, TN>];
    const bool b = (int)blockIdx.x >= g.first;
    const I8Args &u = g.p[0], &v = g.p[1];
    const I8Args p{b ? v.M : u.M, b ? v.N : u.N, b ? v.K : u.K, b ? v.a : u.a, b ? v.lda : u.lda, b ? v.sa : u.sa,
                   b ? v.b : u.b, b ? v.ldb : u.ldb, 0, b ? v.sb : u.sb, 0, b ? v.c : u.c, b ? v.ldc : u.ldc, 0,
                   nullptr, nullptr, 1};
    tile_product<TM, TN, false, false, OUT_FP32>(p, (int)blockIdx.x - (b ? g.first : 0), smem);
}

// Few rows (decode): the weights are read once, straight into registers, by waves
// that split K and meet in LDS.  A workgroup takes 16 weight rows; a wave takes every
// W-th run of 128 bytes of K, a whole cache line of each row, and feeds it to two
// matrix instructions per 16 activation rows.  Lane quarter q has bytes 32 q to
// 32 q + 31 of a run from both operands: any order of K will do for a sum of integers.
constexpr int kRun = 128;

struct Run {
    i32x4 lo, hi;
};
// A lane's 32 bytes at `row` + k (K % 16 == 0).  Past the end weights are those of the
// row's last 16 bytes, so that no load waits for a comparison, and activations zeros:
// zero times any code is zero.
__device__ __forceinline__ Run weight_run(const uint8_t* row, int k, int K, int q) {
    const int at = k + 32 * q;
    return {*reinterpret_cast<const i32x4*>(row + min(at, K - 16)), *reinterpret_cast<const i32x4*>(row + min(at + 16, K - 16))};
}
__device__ __forceinline__ Run act_run(const uint8_t* row, int k, int K, int q) {
    const int at = k + 32 * q;
    Run r = weight_run(row, k, K, q);
    const i32x4 zero = {0, 0, 0, 0};
    r.lo = at < K ? r.lo : zero;
    r.hi = at + 16 < K ? r.hi : zero;
    return r;
}

// The waves' partial sums of MT tiles, added in LDS, scaled and stored.
template <int MT, int W, bool GATHER, bool OUT32>
__device__ __forceinline__ void join_waves(const I8Args& p, const i32x4 (&acc)[MT], i32x4* part, int m0, int m1, int n0,
                                           const float* sa, const float* sb) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < MT; ++j) part[(wave * MT + j) * 64 + lane] = acc[j];
    __syncthreads();
    for (int o = threadIdx.x; o < MT * 64; o += 64 * W) {
        const int l = o & 63, m = m0 + 16 * (o >> 6) + (l & 15), n = n0 + 4 * (l >> 4);
        i32x4 v = part[o];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w * MT * 64 + o];
        if (m < m1 && n < p.N) {
            const float s = sa[GATHER ? p.a_rows[m] : m];
            const float f[4] = {(float)v[0] * s * sb[n], (float)v[1] * s * sb[n + 1], (float)v[2] * s * sb[n + 2],
                                (float)v[3] * s * sb[n + 3]};
            store4<OUT32>(p.c, (int64_t)m * p.ldc + n, f);
        }
    }
}

// Up to U runs in flight: passes of U, then one of the runs that are left, so that no
// load is made in vain (a kernel that read the last 16 bytes again instead took 91 us
// where this takes 63 on 110 groups of 1536 x 2048 weights).  Grouped: grid row y is a
// group, whose rows go in passes of 16 MT; dense: grid row y is such a pass.
template <int MT, int W, int U, bool GROUPED, bool GATHER, bool OUT32>
__global__ void __launch_bounds__(64 * W) k_i8_stream(I8Args p) {
    __shared__ __attribute__((aligned(16))) i32x4 part[W * MT * 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, r16 = lane & 15, n0 = blockIdx.x * 16;
    int m0 = 0, m1 = p.M;
    const uint8_t* b = p.b;
    const float* sb = p.sb;
    if (GROUPED) {
        m0 = p.offsets[blockIdx.y];
        m1 = p.offsets[blockIdx.y + 1];
        b += (int64_t)blockIdx.y * p.b_sg;
        sb += (int64_t)blockIdx.y * p.sb_sg;
    } else {
        m0 = blockIdx.y * 16 * MT;
        m1 = min(m1, m0 + 16 * MT);
    }
    const uint8_t* brow = b + (int64_t)min(n0 + r16, p.N - 1) * p.ldb;
    for (; m0 < m1; m0 += 16 * MT) {
        const uint8_t* arow[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            int m = min(m0 + 16 * j + r16, m1 - 1);
            if (GATHER) m = p.a_rows[m];
            arow[j] = p.a + (int64_t)m * p.lda;
        }
        i32x4 acc[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[j] = i32x4{0, 0, 0, 0};
        auto pass = [&](auto count, int k) {
            constexpr int C = decltype(count)::value;
            Run fb[C], fa[C][MT];
#pragma unroll
            for (int u = 0; u < C; ++u) {
                fb[u] = weight_run(brow, k + u * W * kRun, p.K, q);
#pragma unroll
                for (int j = 0; j < MT; ++j) fa[u][j] = act_run(arow[j], k + u * W * kRun, p.K, q);
            }
#pragma unroll
            for (int u = 0; u < C; ++u)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[j] = mfma(fb[u].hi, fa[u][j].hi, mfma(fb[u].lo, fa[u][j].lo, acc[j]));
        };
        int k = wave * kRun, left = ((p.K + kRun - 1) / kRun - wave + W - 1) / W;
        for (; left >= U; left -= U, k += U * W * kRun) pass(std::integral_constant<int, U>{}, k);
        unrolled<U - 1>([&](auto c) {
            if (left == decltype(c)::value + 1) pass(std::integral_constant<int, decltype(c)::value + 1>{}, k);
        });
        join_waves<MT, W, GATHER, OUT32>(p, acc, part, m0, m1, n0, p.sa, sb);
        __syncthreads();
    }
}

// One or two rows (decode).  A wave takes R whole rows of weights, a kilobyte of each
// at a time and up to P in flight, and multiplies them by every activation row with
// v_dot4: reading whole rows is what pays (25 MB cold: 5.3 us, in the fragments of a
// matrix instruction 7.4), and 16 cycles per kilobyte and row hide behind the reads.
// FUSED: one row that comes in bf16 and that every workgroup quantizes for itself into
// LDS (kFusedCodes at most) in the shadow of its first weights, which saves a launch.
constexpr int kFusedCodes = 16384;
template <int MT, int R, int P, int W, bool FUSED, bool OUT32>
__global__ void __launch_bounds__(64 * W) k_i8_dot(I8Args p, const uint16_t* x, int32_t cols) {
    static_assert(MT == 1 || !FUSED, "one row");
    constexpr int kChunks = FUSED ? kFusedCodes / 8 / (64 * W) : 1;     // chunks of eight values per thread
    __shared__ __attribute__((aligned(16))) uint8_t codes[FUSED ? kFusedCodes : 16];
    __shared__ uint32_t top[W];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = (blockIdx.x * W + wave) * R;
    const uint8_t* brow = p.b + (int64_t)min(n0, p.N - R) * p.ldb;
    i32x4 w[R][P];
    int pieces = (p.K + 1023) / 1024;
    auto load = [&](int k) {
        unrolled<P>([&](auto c) {
            constexpr int i = decltype(c)::value;
            if (i < pieces)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    w[r][i] = *reinterpret_cast<const i32x4*>(brow + r * p.ldb + min(k + 1024 * i + 16 * lane, p.K - 16));
        });
    };
    load(0);
    float scale = 0;
    if constexpr (FUSED) {
        const int chunks = cols / 8;
        uint4 v[kChunks];
        u16x2 m = {0, 0};
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            const int c = threadIdx.x + i * 64 * W;
            if (c < chunks) v[i] = *reinterpret_cast<const uint4*>(x + c * 8);
            m = absmax_bits(m, v[i]);
        }
        const uint32_t mine = lanes_umax<64>(max((uint32_t)m.x, (uint32_t)m.y));
        if (lane == 0) top[wave] = mine;
        __syncthreads();
        uint32_t all = top[0];
#pragma unroll
        for (int i = 1; i < W; ++i) all = max(all, top[i]);
        scale = i8_scale_of(all);
        const I8Scale sc = i8_scale(scale);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = threadIdx.x + i * 64 * W;
            if (c >= p.K / 8) break;                            // past cols: zeros
            float f[8];
            unpack8(v[i], f);
            *reinterpret_cast<uint2*>(codes + c * 8) = i8_codes8<0>(f, &sc);
        }
        __syncthreads();
    }
    int acc[R][MT] = {};
    for (int k = 0;;) {
        unrolled<P>([&](auto c) {
            constexpr int i = decltype(c)::value;
            if (i >= pieces) return;
            const int at = k + 1024 * i + 16 * lane;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint8_t* row = FUSED ? codes : p.a + m * p.lda;
                i32x4 a = *reinterpret_cast<const i32x4*>(row + min(at, p.K - 16));
                if (at >= p.K) a = i32x4{0, 0, 0, 0};
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int b = 0; b < 4; ++b) acc[r][m] = __builtin_amdgcn_sdot4(w[r][i][b], a[b], acc[r][m], false);
            }
        });
        pieces -= P;
        if (pieces <= 0) break;
        k += 1024 * P;
        load(k);
    }
    // output m * R + r on lane m * R + r
    int sum = 0;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int v = (int)lanes_usum((uint32_t)acc[r][m]);
            sum = lane == m * R + r ? v : sum;
        }
    const int m = lane / R, n = n0 + lane % R;
    if (m < MT && n < p.N) {
        const float f = (float)sum * (FUSED ? scale : p.sa[m]) * p.sb[n];
        if (OUT32) static_cast<float*>(p.c)[m * p.ldc + n] = f;
        else static_cast<uint16_t*>(p.c)[m * p.ldc + n] = (uint16_t)pack_bf16x2(f, f);
    }
}

// The K ranges' sums [splits][M][N], added, scaled and stored: four outputs a thread.
template <bool OUT32>
__global__ void __launch_bounds__(256) k_i8_join(I8Args p, const i32x4* sums, int64_t quads) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= quads) return;
    const int64_t m = i * 4 / p.N;
    const int n = (int)(i * 4 - m * p.N);
    i32x4 v = sums[i];
#pragma unroll 4
    for (int s = 1; s < p.splits; ++s) v += sums[s * quads + i];
    const float sa = p.sa[m];
    const float f[4] = {(float)v[0] * sa * p.sb[n], (float)v[1] * sa * p.sb[n + 1], (float)v[2] * sa * p.sb[n + 2],
                        (float)v[3] * sa * p.sb[n + 3]};
    store4<OUT32>(p.c, m * p.ldc + n, f);
}

// Workgroups of a launch of tiles; grouped: as many as there can be tiles.
template <int TM, int TN>
int64_t tile_blocks(int64_t M, int64_t N, int64_t G) {
    constexpr int BM = 64 * TM, BN = 64 * TN;
    const int64_t ntn = (N + BN - 1) / BN;
    return G == 0 ? (M + BM - 1) / BM * ntn : ((M / BM + std::min(G, M)) * ntn + 7) / 8 * 8;
}

template <int TM, int TN, bool GROUPED, bool GATHER>
hipError_t tile(const I8Args& p, bool out32, hipStream_t st) {
    const int64_t blocks = tile_blocks<TM, TN>(p.M, p.N, GROUPED ? p.G : 0);
    if (out32) hipLaunchKernelGGL((k_i8_tile<TM, TN, GROUPED, GATHER, OUT_FP32>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    else hipLaunchKernelGGL((k_i8_tile<TM, TN, GROUPED, GATHER, OUT_BF16>), dim3((unsigned)blocks), dim3(256), 0, st, p);
    return hipGetLastError();
}

// Products of so little work (M N K) that tiles of 128 x 128 leave most compute units
// idle, or wait for each slice: 205 x 1008 by 1512 6.0 us in the waves' K ranges and 8.6
// in tiles, 32 x 4096 by 4096 8.4 and 11.7 (K split).  Just past the limit both ways win
// somewhere: ranges at 128 x 2048 by 2560 (10.7 us, K split 11.2, tiles 12.0) and 64 x
// 2560 by 4096 (8.4, 11.2, 14.1), tiles at 256 x 1024 by 2560 (8.2, ranges 11.0), 64 x
// 1024 by 10240 (8.3, 9.6) and 205 x 1280 by 2560 (9.2, 11.2), K split at 32 x 8192 by
// 2560 (12.2, 13.2) and 17 x 4096 by 9728 (14.4, 17.2); further on the ranges lose: 205 x
// 2048 by 2560 14 and 12.2, 32 x 2560 by 9728 16.0 and 12.9.  Eight waves need a run each.
bool little(int64_t M, int64_t N, int64_t K) { return K > 7 * kRun && M * N * K <= 640000000; }

// K ranges for products with few tiles and a long K: tiles of 64 x 128, about one for
// each compute unit (64 x 9728 by 2560 14.6 us, two for each 16.4; 128 x 9728 16.8 and
// 18.3), or two where one would keep more than 32 slices (333 x 9728 by 2560 26.3, one
// 28.4); of four slices at least.  The join and the sums' way through memory cost as
// much as some 12 slices, so as many are to be saved: 64 x 9728 by 2560 takes 45 us
// whole; 333 x 2048 by 2560 would take 17.2 for 12.4.
int split_count(int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = (M + 63) / 64 * ((N + 127) / 128), nk = (K + BK - 1) / BK;
    if (M <= 16 || M > 512 || tiles >= kCUs || little(M, N, K)) return 1;
    const int64_t one = kCUs / tiles, n = std::min<int64_t>(nk > 32 * one ? 2 * kCUs / tiles : one, nk / 4);
    return n > 1 && nk - nk / n >= 12 ? (int)n : 1;
}

hipError_t split(I8Args p, bool out32, int splits, void* ws, hipStream_t st) {
    I8Args q = p;
    q.c = ws;
    q.splits = p.splits = splits;
    const dim3 grid((unsigned)((p.M + 63) / 64 * ((p.N + 127) / 128)), (unsigned)splits);
    hipLaunchKernelGGL((k_i8_tile<1, 2, false, false, OUT_SUMS>), grid, dim3(256), 0, st, q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t quads = (int64_t)p.M * p.N / 4;
    const dim3 join((unsigned)((quads + 255) / 256));
    const i32x4* sums = static_cast<const i32x4*>(ws);
    if (out32) hipLaunchKernelGGL(k_i8_join<true>, join, dim3(256), 0, st, p, sums, quads);
    else hipLaunchKernelGGL(k_i8_join<false>, join, dim3(256), 0, st, p, sums, quads);
    return hipGetLastError();
}

template <int MT, int W, int U, bool GROUPED, bool GATHER>
hipError_t stream(const I8Args& p, bool out32, hipStream_t st) {
    const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)(GROUPED ? p.G : (p.M + 16 * MT - 1) / (16 * MT)));
    if (out32) hipLaunchKernelGGL((k_i8_stream<MT, W, U, GROUPED, GATHER, true>), grid, dim3(64 * W), 0, st, p);
    else hipLaunchKernelGGL((k_i8_stream<MT, W, U, GROUPED, GATHER, false>), grid, dim3(64 * W), 0, st, p);
    return hipGetLastError();
}

template <int MT, int R, int P, int W, bool FUSED>
hipError_t dot(const I8Args& p, bool out32, const uint16_t* x, int64_t cols, hipStream_t st) {
    const dim3 grid((unsigned)((p.N + W * R - 1) / (W * R)));
    if (out32) hipLaunchKernelGGL((k_i8_dot<MT, R, P, W, FUSED, true>), grid, dim3(64 * W), 0, st, p, x, (int32_t)cols);
    else hipLaunchKernelGGL((k_i8_dot<MT, R, P, W, FUSED, false>), grid, dim3(64 * W), 0, st, p, x, (int32_t)cols);
    return hipGetLastError();
}
template <int MT, int W, bool FUSED>
hipError_t dot(const I8Args& p, bool out32, const uint16_t* x, int64_t cols, hipStream_t st) {
    if (p.K > 5120) return dot<MT, 1, 10, W, FUSED>(p, out32, x, cols, st);
    return dot<MT, 2, 5, W, FUSED>(p, out32, x, cols, st);
}

hipError_t launch_dense(const I8Args& p, bool out32, hipStream_t st) {
    if (p.M == 1) return dot<1, 4, false>(p, out32, nullptr, 0, st);
    if (p.M == 2) return dot<2, 4, false>(p, out32, nullptr, 0, st);
    if (p.M <= 16)      // four waves where they have all their runs in flight at once
        return p.K <= 2560 ? stream<1, 4, 5, false, false>(p, out32, st) : stream<1, 16, 5, false, false>(p, out32, st);
    if (little(p.M, p.N, p.K))      // passes of 32 rows, or of 64 where one holds all (64 x 2048 by 2560 7.2 us, 8.2)
        return p.M > 32 && p.M <= 64 ? stream<4, 8, 2, false, false>(p, out32, st) : stream<2, 8, 3, false, false>(p, out32, st);
    // tiles of 256 x 256 where half of the compute units have one
    const int64_t big = ((int64_t)p.M + 255) / 256 * ((p.N + 255) / 256);
    return big >= 128 ? tile<4, 4, false, false>(p, out32, st) : tile<2, 2, false, false>(p, out32, st);
}

// By the rows of a group on average.  128 groups of 1536 x 2048 weights, in us:
//   rows per group     1    2    4    8   16   32   64  128  256
//   stream            38   58   72   90  124  209
//   tile 64 x 128     38   66   73   74   78   79  104  142  232
//   tile 128 x 128    41   73   77   82   82   81   90  122  203
//   tile 256 x 256    59  102  106  102  103  108  113  122  178
enum class Grouped { STREAM, TILE64, TILE128, TILE256 };
Grouped grouped_way(int64_t M, int64_t G) {
    const int64_t rows = (M + G - 1) / G;
    return rows <= 4 ? Grouped::STREAM : rows <= 32 ? Grouped::TILE64 : rows < 128 ? Grouped::TILE128 : Grouped::TILE256;
}
template <bool GATHER>
hipError_t launch_grouped(const I8Args& p, bool out32, hipStream_t st) {
    switch (grouped_way(p.M, p.G)) {
        case Grouped::STREAM: return stream<1, 4, 4, true, GATHER>(p, out32, st);
        case Grouped::TILE64: return tile<1, 2, true, GATHER>(p, out32, st);
        case Grouped::TILE128: return tile<2, 2, true, GATHER>(p, out32, st);
        default: return tile<4, 4, true, GATHER>(p, out32, st);
    }
}

}  // namespace

bool i8_grouped_fits(int64_t M, int64_t N, int64_t G) {
    constexpr int64_t kMost = 1ll << 24;            // 256 threads each
    switch (grouped_way(M, G)) {
        case Grouped::STREAM: return (N + 15) / 16 < kMost;
        case Grouped::TILE64: return tile_blocks<1, 2>(M, N, G) < kMost;
        case Grouped::TILE128: return tile_blocks<2, 2>(M, N, G) < kMost;
        default: return tile_blocks<4, 4>(M, N, G) < kMost;
    }
}

size_t i8_gemm_ws_bytes(int64_t M, int64_t N, int64_t K) {
    const int n = M == 0 || N == 0 ? 1 : split_count(M, N, K);
    return n > 1 ? (size_t)n * (size_t)M * (size_t)N * 4 : 0;
}

hipError_t launch_i8_gemm(const I8GemmArgs& g, void* ws, hipStream_t st) {
    if (g.M == 0 || g.N == 0) return hipSuccess;
    const I8Args p{(int32_t)g.M, (int32_t)g.N, (int32_t)g.K, g.a, g.lda, g.sa, g.b, g.ldb, g.b_sg, g.sb, g.sb_sg,
                   g.c, g.ldc, g.G, g.offsets, g.a_rows, 1};
    if (g.G == 0) {
        const int n = ws ? split_count(g.M, g.N, g.K) : 1;
        return n > 1 ? split(p, g.out_f32, n, ws, st) : launch_dense(p, g.out_f32, st);
    }
    return g.a_rows ? launch_grouped<true>(p, g.out_f32, st) : launch_grouped<false>(p, g.out_f32, st);
}

hipError_t launch_i8_gemm_pair(const I8GemmArgs& g, const I8GemmArgs& h, void* ws, hipStream_t st) {
    const auto tiles = [](const I8GemmArgs& x) { return (x.M + 255) / 256 * ((x.N + 255) / 256); };
    // together they fill the units, and neither is a product of few rows, which the
    // ways of launch_dense read faster
    if (tiles(g) + tiles(h) < kCUs || std::min(g.M, h.M) < 256) {
        const hipError_t e = launch_i8_gemm(g, ws, st);
        return e != hipSuccess ? e : launch_i8_gemm(h, ws, st);
    }
    const auto args = [](const I8GemmArgs& x) {
        return I8Args{(int32_t)x.M, (int32_t)x.N, (int32_t)x.K, x.a, x.lda, x.sa, x.b, x.ldb, 0, x.sb, 0, x.c, x.ldc, 0,
                      nullptr, nullptr, 1};
    };
    const bool swap = h.K > g.K;
    const I8Pair p{{args(swap ? h : g), args(swap ? g : h)}, (int32_t)tiles(swap ? h : g)};
    hipLaunchKernelGGL((k_i8_tile_pair<4, 4>), dim3((unsigned)(tiles(g) + tiles(h))), dim3(256), 0, st, p);
    return hipGetLastError();
}

bool i8_linear_fused(int64_t rows, int64_t cols) { return rows == 1 && cols <= kFusedCodes && cols > 0; }

hipError_t launch_i8_linear_fused(const I8GemmArgs& g, const uint16_t* x, int64_t cols, hipStream_t st) {
    const I8Args p{(int32_t)g.M, (int32_t)g.N, (int32_t)g.K, nullptr, 0, nullptr, g.b, g.ldb, 0, g.sb, 0, g.c, g.ldc, 0,
                   nullptr, nullptr, 1};
    return dot<1, 8, true>(p, g.out_f32, x, cols, st);
}

}  // namespace fp8bs
