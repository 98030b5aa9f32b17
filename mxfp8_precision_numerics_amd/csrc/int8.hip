// 8-bit integer operands for gfx950: quantization of each token (or output channel) to int8, and the product of two such
// operands with a scale for each token and each output channel, dense or over ragged expert row groups.
//
//   quantize:  s_r = max_c |x_rc| / 127,  q_rc = rint(127 x_rc / max_c |x_rc|)          ties to even, -127 .. 127
//   product:   C[m][n] = bf16( (sum_k a[m][k] b[n][k]) sa[m] sb[n] ),  the sum exact in 32-bit integers
//   SwiGLU:    B holds F gate rows, then F up rows:  C[m][f] = bf16( silu(G[m][f]) U[m][f] ) from the products in fp32
#pragma clang fp contract(off)
#include <type_traits>

#include "gemm_tile.h"
#include "launch.h"
#include "mx_block.h"

namespace mxq {

// ------------------------------------------------------------------------------------------------ quantization
// One row's factors. 127 / amax may leave fp32's range where amax is tiny, so values are first scaled by a power of two.
struct Int8Row {
    float scale;        // amax / 127
    float pre, inv;     // code = rint((x pre) inv), inv = 127 / (amax pre)
};

// amax as a bf16 pattern. A NaN or an infinity in the row (0x7F80 and above) gives the scale NaN and zero codes, so that
// every product with the row is NaN.
__device__ __forceinline__ Int8Row int8_row(uint32_t amax_bits) {
    Int8Row r;
    const float amax = __uint_as_float(amax_bits << 16);
    const bool tiny = amax_bits < 0x1000u;                       // below 2^-95
    r.pre = tiny ? 0x1p100f : 1.0f;
    r.inv = 127.0f / (amax * r.pre);
    r.scale = amax / 127.0f;
    if (amax_bits == 0u || amax_bits >= 0x7F80u) {
        r.pre = 0.0f;
        r.inv = 0.0f;
        r.scale = amax_bits ? __uint_as_float(0x7FC00000u) : 0.0f;
    }
    return r;
}

// The code of x in the low byte. t = x inv is within 2^-23 t of 127 x / amax. That quotient of two 8-bit significands is
// either exactly halfway between two codes or at least 2^-15 t away from it, so t rounded to 18 significant bits falls on
// the half exactly where the quotient does, and on the quotient's side of it elsewhere: the code is the quotient's own,
// without a division. Adding 1.5 2^23 rounds to the integer, ties to even, and leaves it in the low bits.
__device__ __forceinline__ uint32_t int8_code(float x, const Int8Row& r) {
    const float t = (x * r.pre) * r.inv;
    const float u = __uint_as_float((__float_as_uint(t) + 0x20u) & ~0x3Fu);
    return __float_as_uint(u + 12582912.0f);
}

__device__ __forceinline__ uint2 int8_codes8(uint4 v, const Int8Row& r, bool finite) {
    float x[8];
    unpack8(v, x);
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = int8_code(x[e], r);
    const uint32_t lo = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0C0C0400u),
                                              __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u), 0x05040100u);
    const uint32_t hi = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[7], c[6], 0x0C0C0400u),
                                              __builtin_amdgcn_perm(c[5], c[4], 0x0C0C0400u), 0x05040100u);
    return finite ? make_uint2(lo, hi) : make_uint2(0u, 0u);     // 0 times an infinity is no code
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    return v;
}

// W waves per row, NCH chunks of 8 values per lane, the row held in registers between the maximum and the codes (NCH = 0:
// a row of any length, read twice). Bound by memory: 3 bytes a value.
template <int W, int NCH>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void int8_quantize_kernel(const uint16_t* __restrict__ x,
                                                                            int64_t rows, int64_t cols,
                                                                            int8_t* __restrict__ q,
                                                                            float* __restrict__ scale) {
    constexpr int ROWS = W < 4 ? 4 / W : 1;
    __shared__ uint32_t part[W > 1 ? ROWS * W : 1];
    const int t = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W);
    const int64_t row = (int64_t)blockIdx.x * ROWS + sub;
    const bool ok = row < rows;
    const int64_t chunks = cols / 8;
    const uint16_t* xr = x + row * cols;
    uint4 v[NCH ? NCH : 1];
    uint32_t m = 0;
    if constexpr (NCH > 0) {
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int64_t ch = t + 64 * W * j;
            v[j] = (ok && ch < chunks) ? ldnt16(xr + 8 * ch) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < NCH; ++j) m = max(m, amax_bits8(v[j]));
    } else {
        if (ok)
            for (int64_t ch = t; ch < chunks; ch += 64 * W) m = max(m, amax_bits8(*reinterpret_cast<const uint4*>(xr + 8 * ch)));
    }
    m = wave_max_u32(m);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) m = max(m, part[sub * W + w]);
    }
    if (!ok) return;
    const Int8Row r = int8_row(m);
    const bool finite = m < 0x7F80u;
    if (t == 0) scale[row] = r.scale;
    int8_t* qr = q + row * cols;
    if constexpr (NCH > 0) {
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int64_t ch = t + 64 * W * j;
            if (ch < chunks) *reinterpret_cast<uint2*>(qr + 8 * ch) = int8_codes8(v[j], r, finite);
        }
    } else {
        for (int64_t ch = t; ch < chunks; ch += 64 * W)
            *reinterpret_cast<uint2*>(qr + 8 * ch) =
                int8_codes8(*reinterpret_cast<const uint4*>(xr + 8 * ch), r, finite);
    }
}

int64_t int8_quantize_max_rows(int64_t cols) {
    return cols <= 2048 ? kMaxThreads / 64 : cols <= 8192 ? kMaxThreads / 256 : kMaxThreads / 1024;
}

hipError_t launch_int8_quantize(const uint16_t* x, int64_t rows, int64_t cols, int8_t* q, float* scale,
                                hipStream_t stream) {
    const dim3 four((unsigned)((rows + 3) / 4)), one((unsigned)rows);
    if (cols <= 512) hipLaunchKernelGGL((int8_quantize_kernel<1, 1>), four, dim3(256), 0, stream, x, rows, cols, q, scale);
    else if (cols <= 1024) hipLaunchKernelGGL((int8_quantize_kernel<1, 2>), four, dim3(256), 0, stream, x, rows, cols, q, scale);
    else if (cols <= 2048) hipLaunchKernelGGL((int8_quantize_kernel<1, 4>), four, dim3(256), 0, stream, x, rows, cols, q, scale);
    else if (cols <= 8192) hipLaunchKernelGGL((int8_quantize_kernel<4, 4>), one, dim3(256), 0, stream, x, rows, cols, q, scale);
    else if (cols <= 32768) hipLaunchKernelGGL((int8_quantize_kernel<16, 4>), one, dim3(1024), 0, stream, x, rows, cols, q, scale);
    else hipLaunchKernelGGL((int8_quantize_kernel<16, 0>), one, dim3(1024), 0, stream, x, rows, cols, q, scale);
    return hipGetLastError();
}

// ------------------------------------------------------------------------------------------------ products
struct Int8Gemm {
    const int8_t* a;        // [M][K]
    const int8_t* b;        // [N][K], for each expert
    const float* sa;        // [M]
    const float* sb;        // [N], for each expert
    uint16_t* c;
    int64_t M, N, K, ldc;   // N: rows of b (SwiGLU: gate rows, then up rows)
    const int64_t* offsets; // grouped: [G + 1]
    int64_t G;
};

// One output from its integer sum. The product is scaled by the token first: sa sb alone could leave fp32's range.
__device__ __forceinline__ float int8_value(int acc, float sa, float sb) { return ((float)acc * sa) * sb; }

// silu(g) u. The exponential and the quotient are the hardware's (v_exp_f32 and v_rcp_f32, an ulp each), 8 operations of
// which two take four times as long; the fixed sequence of the MXFP8 path with its division takes about 60, which would cost
// a 256 x 128 tile more than its matrix instructions at K = 2048. Relative error below (13 + 4.3 |g|) 2^-24, of which
// 3 (1 + |g|) is g's own; the result is rounded to bf16.
__device__ __forceinline__ float silu_times(float g, float u) {
    const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
    return (g * __builtin_amdgcn_rcpf(1.0f + e)) * u;
}

// Rows of B in a tile of TN of them. Plain: TN consecutive rows, TN output columns. SwiGLU: blocks of BLK rows alternate
// between gate and up rows of the same BLK output columns, so a wave holds both factors of an output in two accumulators.
template <bool SWIGLU, int BLK>
__device__ __forceinline__ int64_t b_row(int64_t n0, int r, int64_t F) {
    if constexpr (!SWIGLU) return n0 + r;
    else return n0 + (r / (2 * BLK)) * BLK + r % BLK + ((r / BLK) & 1) * F;
}

// 128 x 128 rows of A and B per workgroup (4 waves, 2 x 2, each 64 x 64 as 4 x 4 v_mfma_i32_16x16x64_i8). K advances 128
// bytes per stage, staged through registers into two LDS buffers of 128-byte rows whose 16-byte chunks are XOR-swizzled by
// the row. B is the instruction's first operand: lane l, register e hold output row l % 16, column 4 (l / 16) + e.
constexpr int QT = 128, QK = 128;
__device__ __forceinline__ int q_swz(int row, int chunk) { return row * QK + ((chunk ^ (row & 7)) << 4); }

template <bool GROUPED, bool SWIGLU>
__global__ __launch_bounds__(256) void int8_gemm_kernel(Int8Gemm g) {
    __shared__ __attribute__((aligned(16))) uint8_t sA[2][QT * QK];
    __shared__ __attribute__((aligned(16))) uint8_t sB[2][QT * QK];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave & 1, wn = wave >> 1;
    const int64_t cols = SWIGLU ? g.N / 2 : g.N;                 // output columns
    constexpr int TC = SWIGLU ? QT / 2 : QT;                     // of a tile
    const int64_t tiles_n = (cols + TC - 1) / TC;
    int64_t m0, m_end, grp = 0;
    const int64_t n0 = (blockIdx.x % tiles_n) * TC;
    if constexpr (GROUPED) {
        const RowTile rt = find_row_tile<QT>(g.offsets, g.G, g.M, blockIdx.x / tiles_n);
        if (rt.grp < 0) return;
        grp = rt.grp;
        m0 = rt.lo;
        m_end = rt.lo + QT < rt.hi ? rt.lo + QT : rt.hi;
    } else {
        m0 = (blockIdx.x / tiles_n) * QT;
        m_end = m0 + QT < g.M ? m0 + QT : g.M;
    }
    const int8_t* B = g.b + grp * g.N * g.K;
    const float* sb = g.sb + grp * g.N;

    uint4 ra[4], rb[4];
    auto load_stage = [&](int64_t k0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = (tid >> 3) + 32 * j;
            const int64_t kk = k0 + 16 * (tid & 7), ar = m0 + row, br = b_row<SWIGLU, 16>(n0, row, cols);
            const bool b_ok = SWIGLU ? n0 + (row / 32) * 16 + row % 16 < cols : br < cols;
            ra[j] = (ar < m_end && kk < g.K) ? *reinterpret_cast<const uint4*>(g.a + ar * g.K + kk) : make_uint4(0, 0, 0, 0);
            rb[j] = (b_ok && kk < g.K) ? *reinterpret_cast<const uint4*>(B + br * g.K + kk) : make_uint4(0, 0, 0, 0);
        }
    };
    auto store_stage = [&](int buf) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = (tid >> 3) + 32 * j;
            *reinterpret_cast<uint4*>(&sA[buf][q_swz(row, tid & 7)]) = ra[j];
            *reinterpret_cast<uint4*>(&sB[buf][q_swz(row, tid & 7)]) = rb[j];
        }
    };
    v4i acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    const int r16 = lane & 15, q16 = lane >> 4;
    const int nk = (int)((g.K + QK - 1) / QK);
    load_stage(0);
    store_stage(0);
    __syncthreads();
    for (int kt = 0; kt < nk; ++kt) {
        const int buf = kt & 1;
        if (kt + 1 < nk) load_stage((int64_t)(kt + 1) * QK);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v4i fa[4], fb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                fa[j] = *reinterpret_cast<const v4i*>(&sA[buf][q_swz(wm * 64 + j * 16 + r16, 4 * h + q16)]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                fb[i] = *reinterpret_cast<const v4i*>(&sB[buf][q_swz(wn * 64 + i * 16 + r16, 4 * h + q16)]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[i], fa[j], acc[i][j], 0, 0, 0);
        }
        if (kt + 1 < nk) store_stage(buf ^ 1);
        __syncthreads();
    }

    const bool vec_ok = (g.ldc & 3) == 0 && (reinterpret_cast<uintptr_t>(g.c) & 7) == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + wm * 64 + j * 16 + r16;
        if (m >= m_end) continue;
        const float s = g.sa[m];
#pragma unroll
        for (int i = 0; i < 4; i += SWIGLU ? 2 : 1) {
            const int64_t n = SWIGLU ? n0 + wn * 32 + (i / 2) * 16 + 4 * q16 : n0 + wn * 64 + i * 16 + 4 * q16;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n + e >= cols) {
                    v[e] = 0.0f;
                } else if constexpr (SWIGLU) {
                    v[e] = silu_times(int8_value(acc[i][j][e], s, sb[n + e]),
                                      int8_value(acc[i + 1][j][e], s, sb[cols + n + e]));
                } else {
                    v[e] = int8_value(acc[i][j][e], s, sb[n + e]);
                }
            }
            uint16_t* dst = g.c + m * g.ldc + n;
            if (vec_ok && n + 4 <= cols) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < cols) dst[e] = (uint16_t)pack_bf16(v[e], 0.0f);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------------------
// Large tiles: 256 x 256 rows of A and B per workgroup, one workgroup per CU; 4 waves, 2 x 2, each 128 x 128 as 8 x 8
// accumulators of 16 x 16 (256 registers). K advances 64 bytes per stage: one v_mfma_i32_16x16x64_i8 per accumulator.
// (The chip is held back by its power here: from registers alone, on normally distributed codes, this instruction runs
// at 4.2 POP/s and the 32 x 32 x 32 form at 3.4; on zeros both reach 4.9.) Operand of lane l: row l % 16, bytes 16 (l / 16)
// .. + 15; B is the first operand, so register e of lane l holds output row l % 16, column 4 (l / 16) + e.
//
// K advances in pairs of stages, 128 bytes, so that a copy instruction (global to LDS, no registers) takes whole lines: 8
// rows of 128 bytes. (16 rows of 64 bytes a copy, twice the requests to the L2, cost 1.13 times the time at
// 4096 x 36864 x 12288.) LDS holds three pairs of A and two of B, 32 KiB each, as rows of 128 bytes whose 16-byte chunk c
// lies at position c ^ (row / 2 % 8): the fragment reads of 16 consecutive rows fall on all banks once.
// Trip t multiplies stage t from registers and reads stage t + 1's fragments into a second set; the one barrier of a pair
// lies behind its first trip, where every wave has read the whole pair p: trip 2p + 1 then copies B's pair p + 2 into B's
// region of p, trip 2p + 2 A's pair p + 3 into A's region of p. At the next barrier, behind trip 2p + 2, all but that last
// pair of A must have landed: B has one to two trips to arrive, A three to four.
constexpr int LT = 256, LK = 64, LPAIR = 2 * LK, LREGION = LT * LPAIR, LREGIONS_A = 3;
constexpr int LGROUP_M = 4;            // row tiles that an XCD's workgroups walk together
constexpr int64_t LXCD = 32;           // workgroups of one XCD at a time

// acc += b a. Written as assembly so that the sum stays in its registers: left to itself the compiler gives the instruction
// another destination and copies results about in the loop. The operands' loads are waited for by the compiler; nothing
// else may write an operand or read a sum within 19 wait states (the kernel has 64 instructions between two uses of a
// sum, and waits of its own around the last stage).
__device__ __forceinline__ void mfma_in_place(v4i& acc, v4i b, v4i a) {
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}

template <bool GROUPED, bool SWIGLU>
__global__ __launch_bounds__(256, 1) void int8_gemm_large_kernel(Int8Gemm g) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[(LREGIONS_A + 2) * LREGION];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int64_t cols = SWIGLU ? g.N / 2 : g.N;
    constexpr int TC = SWIGLU ? LT / 2 : LT;
    const int tiles_n = (int)((cols + TC - 1) / TC);

    // ------------------------------------------------------------------ tile
    int64_t m0, m_end, n0, grp = 0;
    if constexpr (GROUPED) {
        // each XCD (every eighth workgroup) takes chunks of LXCD consecutive tiles, which share an expert's weights
        const int64_t nb = gridDim.x, b = blockIdx.x, round = 8 * LXCD;
        const int64_t t = b < (nb / round) * round ? (b >> 3) / LXCD * round + (b & 7) * LXCD + (b >> 3) % LXCD : b;
        n0 = (t % tiles_n) * TC;
        const RowTile rt = find_row_tile<LT>(g.offsets, g.G, g.M, t / tiles_n);
        if (rt.grp < 0) return;
        grp = rt.grp;
        m0 = rt.lo;
        m_end = rt.lo + LT < rt.hi ? rt.lo + LT : rt.hi;
    } else {
        // each XCD walks a contiguous run of an order in groups of LGROUP_M row tiles
        const int tiles_m = (int)((g.M + LT - 1) / LT);
        const int T = tiles_m * tiles_n, T8 = T & ~7, b = blockIdx.x;
        const int v = b < T8 ? (b & 7) * (T8 >> 3) + (b >> 3) : b;
        const int per_group = LGROUP_M * tiles_n, first_m = (v / per_group) * LGROUP_M;
        const int gm = min(LGROUP_M, tiles_m - first_m), r = v % per_group;
        m0 = (int64_t)(first_m + r % gm) * LT;
        n0 = (int64_t)(r / gm) * TC;
        m_end = m0 + LT < g.M ? m0 + LT : g.M;
    }
    const int8_t* A = g.a + m0 * g.K;
    const int8_t* B = g.b + (grp * g.N + n0) * g.K;             // SwiGLU: the gate rows; the up rows are cols rows further
    const int64_t n_end = n0 + TC < cols ? n0 + TC : cols;

    // ------------------------------------------------------------------ scales of the wave's rows and columns
    // Read here, ahead of the copies, so that the epilogue begins with them in registers.
    const int r16 = lane & 15, q16 = lane >> 4;
    constexpr int NB = SWIGLU ? 4 : 8;                          // 16-column output blocks of a wave
    const float* sb = g.sb + grp * g.N;
    float sa[8], s_gate[NB][4], s_up[SWIGLU ? NB : 1][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t m = m0 + wm * 128 + j * 16 + r16;
        sa[j] = g.sa[m < m_end ? m : m_end - 1];
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t n = n0 + wn * (TC / 2) + 16 * b + 4 * q16 + e, nc = n < cols ? n : cols - 1;
            s_gate[b][e] = sb[nc];
            if constexpr (SWIGLU) s_up[b][e] = sb[cols + nc];
        }

    // ------------------------------------------------------------------ copies
    // Copy c (0 .. 7) of a wave fills rows 32c + 8 wave .. + 7 of a region: lane l brings row l / 8 of them, the chunk that
    // belongs at position l % 8. The resources end with the operand: rows behind its end are zeros, rows of A behind the
    // group's are the next group's, and what a last pair asks for past the end of K is a part of the next row (their
    // outputs are never stored, and the last is masked).
    auto bytes = [&](int64_t rows) { return (uint32_t)(rows * g.K < 0x7FFFFFFF ? rows * g.K : 0x7FFFFFFF); };
    const v4i rA = buffer_rsrc(A, bytes(g.M - m0));
    const v4i rB = buffer_rsrc(SWIGLU && wave >= 2 ? B + cols * g.K : B, bytes(cols - n0));   // waves 2, 3 bring up rows
    const int brow = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
    const int K = (int)g.K;
    const int a_off = brow * K + 16 * chunk, b_off = (SWIGLU ? brow & 15 : brow) * K + 16 * chunk;
    const int a_step = 32 * K, b_step = SWIGLU ? 16 * K : 32 * K;
    const uint32_t lds0 = lds_offset(&lds[1024 * wave]);
    // copy c of pair p into the region at byte `into`
    auto copy_a = [&](int p, uint32_t into, int c) { dma_to_lds<16>(rA, lds0 + into + 4096 * c, a_off + c * a_step, p * LPAIR); };
    auto copy_b = [&](int p, uint32_t into, int c) { dma_to_lds<16>(rB, lds0 + into + 4096 * c, b_off + c * b_step, p * LPAIR); };
    constexpr uint32_t B0 = LREGIONS_A * LREGION;               // B's regions

    // ------------------------------------------------------------------ fragments and matrix instructions
    const int in_row[2] = {r16 * LPAIR + 16 * (q16 ^ (r16 >> 1)), r16 * LPAIR + 16 * ((4 + q16) ^ (r16 >> 1))};
    // fragment f (0 .. 7: A rows 16f .., 8 .. 15: B rows 16 (f - 8) .. of the wave) of half h of the pair in regions a and b
    auto frag = [&](uint32_t a, uint32_t b, int h, int f) {
        const uint32_t at = f < 8 ? a + wm * 128 * LPAIR + f * 16 * LPAIR : b + wn * 128 * LPAIR + (f - 8) * 16 * LPAIR;
        return *reinterpret_cast<const v4i*>(&lds[at + in_row[h]]);
    };
    v4i acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    // Everything that writes the sums before this statement has been issued, and nothing that reads them has.
    auto settle = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm volatile("" : "+a"(acc[i][0]), "+a"(acc[i][1]), "+a"(acc[i][2]), "+a"(acc[i][3]), "+a"(acc[i][4]),
                              "+a"(acc[i][5]), "+a"(acc[i][6]), "+a"(acc[i][7]));
    };
    v4i F[2][16];                                               // two sets of fragments

    // One trip in 16 steps of 4 instructions: set P is multiplied; with READ, half P ^ 1 of the pair in regions (a, b) is read
    // into the other set, two fragments in each of the first 8 steps; a copy (copy(c), c = 0 .. 7) goes in every other step.
    auto trip = [&](auto p_c, auto read_c, uint32_t a, uint32_t b, auto&& copy) {
        constexpr int P = decltype(p_c)::value;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int i = q >> 1;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = 4 * (q & 1) + x;
                mfma_in_place(acc[i][j], F[P][8 + i], F[P][j]);
            }
            if constexpr (decltype(read_c)::value) {
                if (q < 8) {
                    F[P ^ 1][2 * q] = frag(a, b, P ^ 1, 2 * q);
                    F[P ^ 1][2 * q + 1] = frag(a, b, P ^ 1, 2 * q + 1);
                }
            }
            if (q & 1) copy(q >> 1);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using T0 = std::integral_constant<int, 0>;
    using T1 = std::integral_constant<int, 1>;
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    auto none = [](int) {};
    // What a last pair holds past K becomes zero in A (selects: the sums keep one path).
    const int rem = (int)(g.K % LPAIR);                         // 0, 32, 64 or 96
    auto mask = [&](auto p_c) {
        constexpr int P = decltype(p_c)::value;
        const int keep = rem == 0 || 16 * (4 * P + q16) < rem ? -1 : 0;
#pragma unroll
        for (int f = 0; f < 8; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e) F[P][f][e] &= keep;
        // the selects' results to the matrix instructions
        asm volatile("s_nop 7" : "+v"(F[P][0]), "+v"(F[P][1]), "+v"(F[P][2]), "+v"(F[P][3]), "+v"(F[P][4]), "+v"(F[P][5]),
                                 "+v"(F[P][6]), "+v"(F[P][7]));
    };

    // ------------------------------------------------------------------ prologue: pairs 0 and 1, and A's pair 2
    const int np = (int)((g.K + LPAIR - 1) / LPAIR);
#pragma unroll
    for (int c = 0; c < 8; ++c) copy_a(0, 0, c);
#pragma unroll
    for (int c = 0; c < 8; ++c) copy_b(0, B0, c);
    if (np > 1) {
#pragma unroll
        for (int c = 0; c < 8; ++c) copy_a(1, LREGION, c);
#pragma unroll
        for (int c = 0; c < 8; ++c) copy_b(1, B0 + LREGION, c);
    }
    if (np > 2) {
#pragma unroll
        for (int c = 0; c < 8; ++c) copy_a(2, 2 * LREGION, c);
    }
    settle();                                                   // the zeros are written while the first pairs are on their way
    if (np > 2) wait_copies_barrier<24>();
    else if (np > 1) wait_copies_barrier<16>();
    else wait_copies_barrier<0>();
#pragma unroll
    for (int f = 0; f < 16; ++f) F[0][f] = frag(0, B0, 0, f);
    if (np == 1) mask(T0{});
    trip(T0{}, yes, 0, B0, none);
    if (np > 2) wait_copies_barrier<8>();
    else wait_copies_barrier<0>();
    __builtin_amdgcn_s_waitcnt(0xC07F);                         // the compiler's own view of that wait

    // ------------------------------------------------------------------ pairs
    int p = 0;
    uint32_t a0 = 0, a1 = LREGION, b0 = B0, b1 = B0 + LREGION;  // regions of pairs p and p + 1
    auto next = [&]() {
        a0 = a1;
        a1 = a1 == 2 * LREGION ? 0u : a1 + LREGION;
        const uint32_t x = b0;
        b0 = b1;
        b1 = x;
        ++p;
    };
    while (p + 3 < np) {
        trip(T1{}, yes, a1, b1, [&](int c) { copy_b(p + 2, b0, c); });
        trip(T0{}, yes, a1, b1, [&](int c) { copy_a(p + 3, a0, c); });
        wait_copies_barrier<8>();
        __builtin_amdgcn_s_waitcnt(0xC07F);
        next();
    }
    while (p + 1 < np) {                                        // at most B's pair p + 2 is still to be copied
        if (p + 2 < np) {
#pragma unroll
            for (int c = 0; c < 8; ++c) copy_b(p + 2, b0, c);
        }
        trip(T1{}, yes, a1, b1, none);
        if (p + 2 == np && rem) mask(T0{});
        trip(T0{}, yes, a1, b1, none);
        wait_copies_barrier<0>();
        __builtin_amdgcn_s_waitcnt(0xC07F);
        next();
    }
    if (rem == 0 || rem > LK) {                                 // the last half, if K reaches into it
        if (rem) mask(T1{});
        trip(T1{}, no, 0, 0, none);
    }
    asm volatile("s_nop 15\n\ts_nop 15");                       // the matrix instructions' results to what reads them
    settle();

    // ------------------------------------------------------------------ epilogue
    // Lane l holds columns 4 (l / 16) .. + 3 of row l % 16 of each 16 x 16 block. Two blocks side by side swap every other
    // 16-lane row (v_permlane16_swap), which leaves a lane with 8 consecutive columns of one of them: lanes of row R hold
    // columns 16 (R % 2) + 8 (R / 2) .. of the pair's 32, and a 16-byte store writes 64 contiguous bytes into each of 16
    // rows.
    const bool vec_ok = (g.ldc & 7) == 0 && (reinterpret_cast<uintptr_t>(g.c) & 15) == 0;
#pragma unroll
    for (int p = 0; p < NB / 2; ++p) {
        const int64_t n = n0 + wn * (TC / 2) + p * 32 + 16 * (q16 & 1) + 8 * (q16 >> 1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t w[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int b = 2 * p + h;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (SWIGLU)
                        v[e] = silu_times(int8_value(acc[2 * b][j][e], sa[j], s_gate[b][e]),
                                          int8_value(acc[2 * b + 1][j][e], sa[j], s_up[b][e]));
                    else
                        v[e] = int8_value(acc[b][j][e], sa[j], s_gate[b][e]);
                }
                w[h][0] = pack_bf16(v[0], v[1]);
                w[h][1] = pack_bf16(v[2], v[3]);
            }
            const auto x = __builtin_amdgcn_permlane16_swap(w[0][0], w[1][0], false, false);
            const auto y = __builtin_amdgcn_permlane16_swap(w[0][1], w[1][1], false, false);
            const int64_t m = m0 + wm * 128 + j * 16 + r16;
            if (m >= m_end) continue;
            uint16_t* dst = g.c + m * g.ldc + n;
            const uint32_t d[4] = {(uint32_t)x[0], (uint32_t)y[0], (uint32_t)x[1], (uint32_t)y[1]};
            if (vec_ok && n + 8 <= n_end) {
                *reinterpret_cast<uint4*>(dst) = make_uint4(d[0], d[1], d[2], d[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < n_end) dst[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
}

// Upper bound of the row tiles of TH rows over ragged groups: every group with rows adds at most one partial tile.
static int64_t most_row_tiles(int64_t rows, int64_t G, int64_t TH) { return (rows + TH - 1) / TH + (G < rows ? G : rows); }

// Large tiles where they fill the chip: at least 512 rows and output columns (grouped: 512 rows an expert on average).
static bool large_tiles(int64_t M, int64_t cols, int64_t G) { return cols >= 512 && M >= 512 * (G ? G : 1); }

int64_t int8_gemm_blocks(int64_t M, int64_t cols, int64_t G, int swiglu) {
    const int64_t tile = large_tiles(M, cols, G) ? LT : QT, tc = swiglu ? tile / 2 : tile;
    const int64_t tiles_n = (cols + tc - 1) / tc, tiles_m = G ? most_row_tiles(M, G, tile) : (M + tile - 1) / tile;
    return tiles_n > 0 && tiles_m > INT64_MAX / tiles_n ? INT64_MAX : tiles_m * tiles_n;
}

template <bool GROUPED, bool SWIGLU>
static void launch_products(const Int8Gemm& g, int64_t cols, hipStream_t stream) {
    const dim3 blocks((unsigned)int8_gemm_blocks(g.M, cols, g.G, SWIGLU));
    if (large_tiles(g.M, cols, g.G))
        hipLaunchKernelGGL((int8_gemm_large_kernel<GROUPED, SWIGLU>), blocks, dim3(256), 0, stream, g);
    else
        hipLaunchKernelGGL((int8_gemm_kernel<GROUPED, SWIGLU>), blocks, dim3(256), 0, stream, g);
}

hipError_t launch_int8_gemm(const int8_t* a_q, const float* a_scale, const int64_t* offsets, int64_t G, int64_t M,
                            const int8_t* b_q, const float* b_scale, int64_t N, int64_t K, int swiglu, uint16_t* c,
                            int64_t ldc, hipStream_t stream) {
    const Int8Gemm g{a_q, b_q, a_scale, b_scale, c, M, N, K, ldc, offsets, G};
    if (G) {
        if (swiglu) launch_products<true, true>(g, N / 2, stream);
        else launch_products<true, false>(g, N, stream);
    } else {
        if (swiglu) launch_products<false, true>(g, N / 2, stream);
        else launch_products<false, false>(g, N, stream);
    }
    return hipGetLastError();
}

}  // namespace mxq
