// Quantization to 8-bit integers with one scale per row (token) or per column
// (channel), and SiLU*mul followed by the row form: the operands of int8_gemm.
// Rowwise and columnwise are the granularities of scaled 8-bit products ("Towards
// Full Pipeline FP8 Reinforcement Learning for LLMs" compares rowwise scaling with
// the block-wise one for FP8 codes; here the codes are integers).
//
// Bound by HBM: 2 bytes read and 1 written per value, once for rows; columns
// need their maximum over all rows before the first code, so a long tensor is read
// twice (the second time mostly from the last-level cache).  Rows: 4096 x 2560 9 us,
// 4096 x 9728 21 (5.7 TB/s); columns of 4096 x 9728 44 in three launches (26 and 23 in a
// trace; two reads and the writes at 5.5 TB/s are 36), of 9728 x 2560 30, of 4096 x 2560
// 14.5, of 205 x 1512 5.5, one launch.  SiLU*mul codes: 131072 rows of 768 120 us (4.2
// TB/s), 4096 of 9728 44 (4.6), 256 of 768 3.2.
#include "int8_common.h"
#include "internal.h"
#include "reduce.h"

namespace fp8bs {
namespace {

struct RowArgs {
    const uint16_t* x; int64_t rows; int32_t cols; int64_t ld_x;
    uint8_t* q; int64_t ld_q; float* s;
    const int32_t* live;                    // nullable: rows from *live on are left alone
    uint16_t* h; int64_t ld_h;              // SILU: nullable
};

// Eight values of a row as packed bf16: x itself, or h = bf16(silu(gate) * up)
// with the up projection's columns behind the gate's.
template <bool SILU>
__device__ __forceinline__ uint4 row_chunk(const RowArgs& p, const uint16_t* x, int at) {
    const uint4 a = load_nt16(x + at);
    if (!SILU) return a;
    const uint4 u = load_nt16(x + p.cols + at);
    uint32_t hb[8];
    silu_mul8_bf16(a, u, hb);
    return make_uint4(hb[0] | hb[1] << 16, hb[2] | hb[3] << 16, hb[4] | hb[5] << 16, hb[6] | hb[7] << 16);
}

__device__ __forceinline__ void store_codes(const RowArgs& p, uint8_t* q, int at, const uint4 w, const I8Scale& sc) {
    float v[8];
    unpack8(w, v);
    *reinterpret_cast<uint2*>(q + at) = i8_codes8<0>(v, &sc);
}

// L lanes (a wave or the workgroup) hold a row, C chunks of eight columns each,
// from the one read to the codes.  A wave per row serves many rows of up to 4096
// columns; few rows, and longer ones, take a workgroup each.
template <int L, int C, bool SILU>
__global__ void __launch_bounds__(256) k_i8_rows(RowArgs p) {
    __shared__ uint32_t part[4];
    const int l = threadIdx.x % L;
    const int64_t row = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const int64_t end = p.live ? min(p.rows, (int64_t)*p.live) : p.rows;
    if (row >= end) return;                 // whole waves (L 64) or workgroups (L 256)
    const uint16_t* x = p.x + row * p.ld_x;
    uint4 w[C];
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int at = (l + i * L) * 8;
        w[i] = make_uint4(0, 0, 0, 0);
        if (at < p.cols) w[i] = row_chunk<SILU>(p, x, at);
        m = absmax_bits(m, w[i]);
    }
    uint32_t top = lanes_umax<64>(max((uint32_t)m.x, (uint32_t)m.y));
    if (L == 256) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
        __syncthreads();
        top = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    const float s = i8_scale_of(top);
    const I8Scale sc = i8_scale(s);
    if (l == 0) p.s[row] = s;
    uint8_t* q = p.q + row * p.ld_q;
    const int padded = (p.cols + 15) & ~15;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int at = (l + i * L) * 8;
        if (at < padded) store_codes(p, q, at, w[i], sc);       // behind cols: zeros
        if (SILU && p.h && at < p.cols) store_nt16(p.h + row * p.ld_h + at, w[i]);
    }
}

// Rows past 16384 columns: the row is read twice.
template <bool SILU>
__global__ void __launch_bounds__(256) k_i8_rows_long(RowArgs p) {
    __shared__ uint32_t part[4];
    const int64_t row = blockIdx.x;
    if (p.live && row >= *p.live) return;
    const uint16_t* x = p.x + row * p.ld_x;
    u16x2 m = {0, 0};
    for (int64_t at = threadIdx.x * 8; at < p.cols; at += 2048) m = absmax_bits(m, row_chunk<SILU>(p, x, (int)at));
    const uint32_t mine = lanes_umax<64>(max((uint32_t)m.x, (uint32_t)m.y));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = mine;
    __syncthreads();
    const float s = i8_scale_of(max(max(part[0], part[1]), max(part[2], part[3])));
    const I8Scale sc = i8_scale(s);
    if (threadIdx.x == 0) p.s[row] = s;
    const int64_t padded = ((int64_t)p.cols + 15) & ~15ll;
    for (int64_t at = threadIdx.x * 8; at < padded; at += 2048) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (at < p.cols) w = row_chunk<SILU>(p, x, (int)at);
        store_codes(p, p.q + row * p.ld_q, (int)at, w, sc);
        if (SILU && p.h && at < p.cols) store_nt16(p.h + row * p.ld_h + at, w);
    }
}

template <bool SILU>
hipError_t launch_rows(const RowArgs& p, hipStream_t st) {
    const int chunks = (p.cols + 7) / 8;
    // a workgroup per row while a wave per row would leave compute units idle
    const bool wide = chunks > 512 || p.rows < 1024;
    const dim3 grid((unsigned)(wide ? p.rows : (p.rows + 3) / 4));
#define FP8BS_ROWS(L, C) hipLaunchKernelGGL((k_i8_rows<L, C, SILU>), grid, dim3(256), 0, st, p)
    if (wide) {
        if (chunks <= 256) FP8BS_ROWS(256, 1);
        else if (chunks <= 512) FP8BS_ROWS(256, 2);
        else if (chunks <= 1024) FP8BS_ROWS(256, 4);
        else if (chunks <= 1280) FP8BS_ROWS(256, 5);
        else if (chunks <= 2048) FP8BS_ROWS(256, 8);
        else hipLaunchKernelGGL(k_i8_rows_long<SILU>, grid, dim3(256), 0, st, p);
    } else {
        if (chunks <= 64) FP8BS_ROWS(64, 1);
        else if (chunks <= 128) FP8BS_ROWS(64, 2);
        else if (chunks <= 256) FP8BS_ROWS(64, 4);
        else if (chunks <= 320) FP8BS_ROWS(64, 5);
        else FP8BS_ROWS(64, 8);
    }
#undef FP8BS_ROWS
    return hipGetLastError();
}

// ------------------------------------------------------------------ columns
// A thread takes eight columns of four consecutive rows, so that a column's four
// codes are one word of an LDS tile of 64 columns (column stride odd: the 64 writes of
// a wave hit 64 banks), which leaves for memory as whole lines per column.
constexpr int kTileCols = 64;

struct ColArgs {
    const uint16_t* x; int64_t rows; int32_t cols; int64_t ld_x;
    uint8_t* q; int64_t ld_q; float* s;
};

__device__ __forceinline__ uint4 col_chunk(const ColArgs& p, int64_t row, int col) {
    if (row < p.rows && col < p.cols) return load_nt16(p.x + row * p.ld_x + col);
    return make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void max_words(uint32_t (&m)[4], const uint4 w) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m[i]),
                                                                       __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu)));
}

// Codes of 4 ROWQ rows x 64 columns, whose values are in w (rows row0 + 4 (t / 8) + j,
// columns col0 + 8 (t % 8)), through the tile.
template <int ROWQ>
__device__ __forceinline__ void encode_tile(const ColArgs& p, int64_t row0, int col0, const uint4 (&w)[4],
                                            const I8Scale (&sc)[8], uint32_t* tile) {
    constexpr int kStride = ROWQ + 1, kThreads = 8 * ROWQ;
    const int c = threadIdx.x & 7, rq = threadIdx.x >> 3;
    uint2 b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[8];
        unpack8(w[j], v);
        b[j] = i8_codes8<1>(v, sc);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t sel = (uint32_t)(i & 3) | (uint32_t)(4 + (i & 3)) << 8 | 0x0c0c0000u;
        const uint32_t lo = __builtin_amdgcn_perm(i < 4 ? b[1].x : b[1].y, i < 4 ? b[0].x : b[0].y, sel);
        const uint32_t hi = __builtin_amdgcn_perm(i < 4 ? b[3].x : b[3].y, i < 4 ? b[2].x : b[2].y, sel);
        tile[(8 * c + i) * kStride + rq] = lo | hi << 16;
    }
    __syncthreads();
    const int64_t padded = (p.rows + 15) & ~15ll;
    constexpr int kPieces = ROWQ / 4;               // of sixteen rows, per column
#pragma unroll
    for (int u = 0; u < kTileCols * kPieces / kThreads; ++u) {
        const int piece = threadIdx.x + u * kThreads, col = piece / kPieces, at = piece % kPieces;
        const uint32_t* t = tile + col * kStride + 4 * at;
        if (col0 + col < p.cols && row0 + 16 * at < padded)
            *reinterpret_cast<uint4*>(p.q + (int64_t)(col0 + col) * p.ld_q + row0 + 16 * at) = make_uint4(t[0], t[1], t[2], t[3]);
    }
}

// Maxima m of a thread's eight columns, joined over the row lanes t / LC of a
// workgroup of WAVES waves: the pattern of column t (t < 8 LC).
template <int LC, int WAVES>
__device__ __forceinline__ uint32_t join_maxima(uint32_t (&m)[4], uint32_t* lds) {
    // row lanes of a wave first
#pragma unroll
    for (int d = LC; d < 64; d <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m[i]),
                                                                           __builtin_bit_cast(u16x2, (uint32_t)__shfl_xor((int)m[i], d, 64))));
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane < LC) {
#pragma unroll
        for (int i = 0; i < 4; ++i) lds[wave * 4 * LC + 4 * lane + i] = m[i];
    }
    __syncthreads();
    uint32_t top = 0;
    if (threadIdx.x < 8 * LC) {
#pragma unroll
        for (int r = 0; r < WAVES; ++r) {
            const uint32_t w = lds[r * 4 * LC + (threadIdx.x >> 1)];
            top = max(top, (threadIdx.x & 1) ? w >> 16 : w & 0xffffu);
        }
    }
    return top;
}

// Up to 512 rows: a workgroup holds 64 columns whole, from the one read to the codes.
constexpr int kFewRows = 512;
__global__ void __launch_bounds__(1024) k_i8_cols(ColArgs p) {
    __shared__ uint32_t tile[kTileCols * (kFewRows / 4 + 1)];
    __shared__ uint32_t part[16 * 32];
    __shared__ float scale[kTileCols];
    const int col0 = blockIdx.x * kTileCols, c = threadIdx.x & 7, rq = threadIdx.x >> 3;
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = col_chunk(p, 4 * rq + j, col0 + 8 * c);
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) max_words(m, w[j]);
    const uint32_t top = join_maxima<8, 16>(m, part);
    if (threadIdx.x < kTileCols) {
        const float s = i8_scale_of(top);
        scale[threadIdx.x] = s;
        if (col0 + (int)threadIdx.x < p.cols) p.s[col0 + threadIdx.x] = s;
    }
    __syncthreads();
    I8Scale sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sc[i] = i8_scale(scale[8 * c + i]);
    encode_tile<kFewRows / 4>(p, 0, col0, w, sc, tile);
}

// More rows: zeros into s; the maxima of runs of kMaxRows rows, joined by integer
// atomics on the scales' patterns (the division is monotone, so the largest run's
// scale is the scale of the maximum, and the order of the joins does not matter; NaN's
// pattern is above infinity's); the codes.  One workgroup of 1024 per strip of columns
// without atomics and zeros was slower (4096 x 9728: 33 against 25 + 4 us; 9728 x 2560:
// 37 against 18 + 4).
constexpr int kMaxRows = 256;
__global__ void __launch_bounds__(256) k_i8_zero(float* s, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) s[i] = 0.0f;
}
__global__ void __launch_bounds__(256) k_i8_col_max(ColArgs p) {
    __shared__ uint32_t part[4 * 32];
    const int col0 = blockIdx.x * kTileCols, col = col0 + 8 * (threadIdx.x & 7);
    const int64_t r0 = (int64_t)blockIdx.y * kMaxRows + (threadIdx.x >> 3);
    uint4 w[kMaxRows / 32];
#pragma unroll
    for (int u = 0; u < kMaxRows / 32; ++u) {       // past the last row or column: those again
        w[u] = *reinterpret_cast<const uint4*>(p.x + min(r0 + 32 * u, p.rows - 1) * p.ld_x + min(col, p.cols - 8));
    }
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < kMaxRows / 32; ++u) max_words(m, w[u]);
    const uint32_t top = join_maxima<8, 4>(m, part);
    if (threadIdx.x < kTileCols && col0 + (int)threadIdx.x < p.cols)
        atomicMax(reinterpret_cast<uint32_t*>(p.s) + col0 + threadIdx.x, __float_as_uint(i8_scale_of(top)));
}

// Last launch: the codes, 128 rows x 64 columns per workgroup.
__global__ void __launch_bounds__(256) k_i8_col_codes(ColArgs p) {
    __shared__ uint32_t tile[kTileCols * 33];
    const int col0 = blockIdx.x * kTileCols, c = threadIdx.x & 7, rq = threadIdx.x >> 3;
    const int64_t row0 = (int64_t)blockIdx.y * 128;
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = col_chunk(p, row0 + 4 * rq + j, col0 + 8 * c);
    I8Scale sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sc[i] = i8_scale(p.s[min(col0 + 8 * c + i, p.cols - 1)]);
    encode_tile<32>(p, row0, col0, w, sc, tile);
}

// Several tensors' columns at once, with a workspace: the maxima of runs of rows to
// memory, then the codes, whose workgroups join the runs: no zeros, no atomics, two
// launches for all (dY, W and X of 4096 x 2560 by 9728: 47 us for the maxima, 3.5 TB/s
// where dirty lines of the products before leave the cache, and 55 for the codes).
constexpr int kRuns = 32;               // runs per tensor at most
__host__ __device__ inline int64_t run_rows(int64_t rows) {
    return kMaxRows * ((rows + (int64_t)kMaxRows * kRuns - 1) / ((int64_t)kMaxRows * kRuns));
}
struct ColsArgs {
    ColArgs t[kI8ColTensors];
    uint16_t* part[kI8ColTensors];      // [runs][cols]
    int32_t strips[kI8ColTensors];
    int32_t end[kI8ColTensors];         // workgroups up to and with this tensor
};
// This workgroup's tensor, strip of columns and block of rows.
struct ColsWork {
    ColArgs p;
    uint16_t* part;
    int32_t strip, block;
};
__device__ __forceinline__ ColsWork cols_work(const ColsArgs& a) {
    static_assert(kI8ColTensors == 3, "written out for three");
    const int b = blockIdx.x;
    const bool one = b >= a.end[0], two = b >= a.end[1];
    const ColArgs &x = a.t[0], &y = a.t[1], &z = a.t[2];
    ColsWork w;
    w.p = {two ? z.x : one ? y.x : x.x, two ? z.rows : one ? y.rows : x.rows, two ? z.cols : one ? y.cols : x.cols,
           two ? z.ld_x : one ? y.ld_x : x.ld_x, two ? z.q : one ? y.q : x.q, two ? z.ld_q : one ? y.ld_q : x.ld_q,
           two ? z.s : one ? y.s : x.s};
    w.part = two ? a.part[2] : one ? a.part[1] : a.part[0];
    const int at = b - (two ? a.end[1] : one ? a.end[0] : 0), strips = two ? a.strips[2] : one ? a.strips[1] : a.strips[0];
    w.block = at / strips;
    w.strip = at - w.block * strips;
    return w;
}
// (Strips of 512 columns, a kilobyte of a row per load, were no faster: 46 us for 47.)
__global__ void __launch_bounds__(256) k_i8_cols_max(ColsArgs a) {
    __shared__ uint32_t lds[4 * 32];
    const ColsWork k = cols_work(a);
    const ColArgs& p = k.p;
    const int col0 = k.strip * kTileCols, col = col0 + 8 * (threadIdx.x & 7);
    const int64_t len = run_rows(p.rows), r0 = k.block * len, r1 = min(r0 + len, p.rows);
    uint32_t m[4] = {0, 0, 0, 0};
    for (int64_t r = r0; r < r1; r += kMaxRows) {
        uint4 w[kMaxRows / 32];
#pragma unroll
        for (int u = 0; u < kMaxRows / 32; ++u)     // past the last row or column: those again
            w[u] = *reinterpret_cast<const uint4*>(p.x + min(r + (threadIdx.x >> 3) + 32 * u, r1 - 1) * p.ld_x + min(col, p.cols - 8));
#pragma unroll
        for (int u = 0; u < kMaxRows / 32; ++u) max_words(m, w[u]);
    }
    const uint32_t top = join_maxima<8, 4>(m, lds);
    if (threadIdx.x < kTileCols && col0 + (int)threadIdx.x < p.cols)
        k.part[(int64_t)k.block * p.cols + col0 + threadIdx.x] = (uint16_t)top;
}
__global__ void __launch_bounds__(256) k_i8_cols_codes(ColsArgs a) {
    __shared__ uint32_t tile[kTileCols * 33];
    __shared__ uint32_t top[4][kTileCols];
    const ColsWork k = cols_work(a);
    const ColArgs& p = k.p;
    const int col0 = k.strip * kTileCols, c = threadIdx.x & 7, rq = threadIdx.x >> 3;
    const int64_t row0 = (int64_t)k.block * 128;
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = col_chunk(p, row0 + 4 * rq + j, col0 + 8 * c);
    const int runs = (int)((p.rows + run_rows(p.rows) - 1) / run_rows(p.rows)), mine = min(col0 + (int)(threadIdx.x & 63), p.cols - 1);
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < kRuns / 4; ++u) {
        const int r = (threadIdx.x >> 6) + 4 * u;
        if (r < runs) m = max(m, (uint32_t)k.part[(int64_t)r * p.cols + mine]);
    }
    top[threadIdx.x >> 6][threadIdx.x & 63] = m;
    __syncthreads();
    I8Scale sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = 8 * c + i;
        const float s = i8_scale_of(max(max(top[0][at], top[1][at]), max(top[2][at], top[3][at])));
        sc[i] = i8_scale(s);
        if (k.block == 0 && rq == 0 && col0 + at < p.cols) p.s[col0 + at] = s;
    }
    encode_tile<32>(p, row0, col0, w, sc, tile);
}

}  // namespace

size_t i8_cols_part_bytes(int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    return (size_t)((rows + run_rows(rows) - 1) / run_rows(rows)) * (size_t)cols * 2;
}

hipError_t launch_i8_quant_cols3(const I8Cols (&t)[kI8ColTensors], hipStream_t st) {
    ColsArgs a;
    int64_t runs = 0, blocks = 0;
    int32_t run_end[kI8ColTensors];
    for (int i = 0; i < kI8ColTensors; ++i) {
        a.t[i] = {t[i].x, t[i].rows, (int32_t)t[i].cols, t[i].ld_x, t[i].q, t[i].ld_q, t[i].s};
        a.part[i] = t[i].part;
        a.strips[i] = (int32_t)((t[i].cols + kTileCols - 1) / kTileCols);
        runs += a.strips[i] * ((t[i].rows + run_rows(t[i].rows) - 1) / run_rows(t[i].rows));
        run_end[i] = (int32_t)runs;
        blocks += a.strips[i] * ((t[i].rows + 127) / 128);
        a.end[i] = (int32_t)blocks;
    }
    ColsArgs m = a;
    for (int i = 0; i < kI8ColTensors; ++i) m.end[i] = run_end[i];
    hipLaunchKernelGGL(k_i8_cols_max, dim3((unsigned)runs), dim3(256), 0, st, m);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_i8_cols_codes, dim3((unsigned)blocks), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_i8_quant_rows(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* q, int64_t ld_q,
                                float* s, hipStream_t st) {
    return launch_rows<false>(RowArgs{x, rows, (int32_t)cols, ld_x, q, ld_q, s, nullptr, nullptr, 0}, st);
}

hipError_t launch_i8_silu_mul_quant(const uint16_t* gu, int64_t rows, int64_t I, int64_t ld_in, const int32_t* live,
                                    uint8_t* q, int64_t ld_q, float* s, uint16_t* h, int64_t ld_h, hipStream_t st) {
    return launch_rows<true>(RowArgs{gu, rows, (int32_t)I, ld_in, q, ld_q, s, live, h, ld_h}, st);
}

hipError_t launch_i8_quant_cols(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* q, int64_t ld_q,
                                float* s, hipStream_t st) {
    const ColArgs p{x, rows, (int32_t)cols, ld_x, q, ld_q, s};
    const unsigned strips = (unsigned)((cols + kTileCols - 1) / kTileCols);
    if (rows <= kFewRows) {
        hipLaunchKernelGGL(k_i8_cols, dim3(strips), dim3(1024), 0, st, p);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(k_i8_zero, dim3((unsigned)((cols + 255) / 256)), dim3(256), 0, st, s, cols);
    hipLaunchKernelGGL(k_i8_col_max, dim3(strips, (unsigned)((rows + kMaxRows - 1) / kMaxRows)), dim3(256), 0, st, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_i8_col_codes, dim3(strips, (unsigned)((rows + 127) / 128)), dim3(256), 0, st, p);
    return hipGetLastError();
}

}  // namespace fp8bs
