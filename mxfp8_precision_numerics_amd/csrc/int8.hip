// 8-bit integer operands for gfx950: quantization of each token (or output channel) to int8, and the product of two such
// operands with a scale for each token and each output channel, dense or over ragged expert row groups.
//
//   quantize:  s_r = max_c |x_rc| / 127,  q_rc = rint(127 x_rc / max_c |x_rc|)          ties to even, -127 .. 127
//   product:   C[m][n] = bf16( (sum_k a[m][k] b[n][k]) sa[m] sb[n] ),  the sum exact in 32-bit integers
//   SwiGLU:    B holds F gate rows, then F up rows:  C[m][f] = bf16( silu(G[m][f]) U[m][f] ) from the products in fp32
#pragma clang fp contract(off)
#include <type_traits>

#include "gemm_tile.h"
#include "int8_plan.h"
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

// The code of x in the low byte. t = x inv is within 2^-23 t of 127 x / amax. With 8-bit significands X and A, that quotient and a
// half between two codes differ by a whole multiple of 1 / 2A in the binade of x, or not at all: by at least t / (254 X) > 2^-16 t.
// t rounded to 18 significant bits moves by at most 2^-18 t, so it falls on the half exactly where the quotient does, and on the
// quotient's side of it elsewhere: the code is the quotient's own, without a division. Adding 1.5 2^23 rounds to the integer,
// ties to even, and leaves it in the low bits.
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
// a row of any length, read twice). Bound by memory, 3 bytes a value: 16384 x 8192 60.6 us, 6.6 TB/s.
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
// a 256 x 128 tile more than its matrix instructions at K = 2048. For g >= -87 the relative error is below (13 + 4.3 |g|) 2^-24, of
// which 3 (1 + |g|) is g's own; the result is rounded to bf16. Below that 1 + e passes 2^126, v_rcp_f32 gives 0 for what would be
// subnormal, and silu, at most 2^-119, is lost: a denominator held in range by a power of two for far gates cost 131072 routed
// rows up 491 -> 502 us and 16384 x 4096 x 1024 69 -> 75.
__device__ __forceinline__ float silu_times(float g, float u) {
    const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
    return (g * __builtin_amdgcn_rcpf(1.0f + e)) * u;
}

// Rows of B in a tile with SwiGLU: blocks of 16 alternate between gate rows and the up rows of the same 16 output columns, so a
// wave holds both factors of an output in two accumulators.

// The tile of a workgroup: TM rows of A within one group, and the index of its column tile.
struct Int8Tile {
    int64_t m0, m_end, grp, n;      // grp < 0: none
};
constexpr int GROUP_M = 4;              // row tiles that an XCD's workgroups walk together
constexpr int64_t XCD_CHUNK = 32;       // consecutive tiles that an XCD takes at a time (grouped)

template <int TM, bool GROUPED>
__device__ __forceinline__ Int8Tile tile_of(const Int8Gemm& g, int tiles_n) {
    Int8Tile r;
    r.grp = 0;
    if constexpr (GROUPED) {
        // each XCD (every eighth workgroup) takes chunks of consecutive tiles, which share an expert's weights
        const int64_t nb = gridDim.x, b = blockIdx.x, round = 8 * XCD_CHUNK;
        const int64_t t = b < (nb / round) * round ? (b >> 3) / XCD_CHUNK * round + (b & 7) * XCD_CHUNK + (b >> 3) % XCD_CHUNK : b;
        r.n = t % tiles_n;
        const RowTile rt = find_row_tile<TM>(g.offsets, g.G, g.M, t / tiles_n);
        r.grp = rt.grp;
        r.m0 = rt.lo;
        r.m_end = rt.lo + TM < rt.hi ? rt.lo + TM : rt.hi;
    } else {
        // each XCD walks a contiguous run of an order in groups of GROUP_M row tiles
        const int tiles_m = (int)((g.M + TM - 1) / TM);
        const int T = tiles_m * tiles_n, T8 = T & ~7, b = blockIdx.x;
        const int v = b < T8 ? (b & 7) * (T8 >> 3) + (b >> 3) : b;
        const int per_group = GROUP_M * tiles_n, first_m = (v / per_group) * GROUP_M;
        const int gm = min(GROUP_M, tiles_m - first_m), x = v % per_group;
        r.m0 = (int64_t)(first_m + x % gm) * TM;
        r.n = x / gm;
        r.m_end = r.m0 + TM < g.M ? r.m0 + TM : g.M;
    }
    return r;
}

// Where in its contraction a workgroup begins (of n steps, then around): spread evenly over consecutive tiles. Workgroups that
// walk rows of the same length in step would ask the same few memory channels at any time; the order of an exact sum is free.
__device__ __forceinline__ int first_step(uint32_t tile, int n) {
    return __builtin_amdgcn_readfirstlane((int)(((uint64_t)(tile * 0x9E3779B9u) * (uint32_t)n) >> 32));
}

// Resource of an operand's rows from `p` on, `rows` of them to the operand's end (a tile takes at most 256, and K is below
// 2^17): what lies behind reads as zeros.
__device__ __forceinline__ v4i rows_rsrc(const int8_t* p, int64_t rows, int64_t K) {
    return buffer_rsrc(p, (uint32_t)(rows < 256 ? rows : 256) * (uint32_t)K);
}

// Middle tiles: 64 rows of A by 128 rows of B per workgroup; 4 waves side by side, each 64 x 32, as 16 x 16 accumulators of
// v_mfma_i32_16x16x64_i8. K advances 128 bytes per stage; a ring of DEPTH stages in LDS, filled by copies of whole lines, rows
// of 128 bytes whose 16-byte chunk c lies at position c ^ (row / 2 % 8). One barrier a stage: behind it the stage has landed for
// every wave and the one before it has been read, so its place is filled with the stage DEPTH - 1 ahead. B is the instruction's
// first operand: lane l, register e hold output row l % 16, column 4 (l / 16) + e. (128 x 128 tiles, two to a CU, were within
// 5% of the better of these and the large ones, or behind, at 130 to 2048 rows.)
template <int DEPTH, bool GROUPED, bool SWIGLU>
__global__ __launch_bounds__(256) void int8_gemm_kernel(Int8Gemm g) {
    constexpr int STAGE = (MT_M + MT_N) * 128, COPIES = STAGE / 4096;            // copies of a wave
    constexpr int NI = 2;                                                        // 16-row blocks of B a wave
    __shared__ __attribute__((aligned(16))) uint8_t lds[DEPTH * STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t cols = SWIGLU ? g.N / 2 : g.N;
    constexpr int TC = SWIGLU ? MT_N / 2 : MT_N;                                     // output columns of a tile
    const Int8Tile tile = tile_of<MT_M, GROUPED>(g, (int)((cols + TC - 1) / TC));
    if (tile.grp < 0) return;
    const int64_t n0 = tile.n * TC;
    const int8_t* B = g.b + (tile.grp * g.N + n0) * g.K;

    // Copy c of a wave fills rows 32c + 8 wave .. + 7 of a stage (A's rows, then B's): lane l brings row l / 8 of them, the
    // chunk that belongs at position l % 8. Rows of A behind the group's and bytes past K are a neighbour's or zeros: the
    // outputs of the first are not stored, the second are masked in A.
    const int K = (int)g.K;
    const v4i rA = rows_rsrc(g.a + tile.m0 * g.K, g.M - tile.m0, g.K);
    const v4i rB = rows_rsrc(SWIGLU && wave >= 2 ? B + cols * g.K : B, cols - n0, g.K);        // waves 2, 3 bring up rows
    const int row = 8 * wave + (lane >> 3), chunk = 16 * ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
    const int a_off = row * K + chunk, b_off = (SWIGLU ? row & 15 : row) * K + chunk;
    const uint32_t lds0 = lds_offset(&lds[1024 * wave]);
    const int nk = (K + 127) / 128, begin = GROUPED ? 0 : first_step((uint32_t)tile.n, nk);
    auto stage = [&](int s) { return s + begin < nk ? s + begin : s + begin - nk; };
    auto copy = [&](int s, uint32_t slot) {
#pragma unroll
        for (int c = 0; c < COPIES; ++c) {
            if (32 * c < MT_M) dma_to_lds<16>(rA, lds0 + slot + 4096 * c, a_off + 32 * c * K, stage(s) * 128);
            else dma_to_lds<16>(rB, lds0 + slot + 4096 * c, b_off + (SWIGLU ? 16 : 32) * (c - MT_M / 32) * K, stage(s) * 128);
        }
    };
    v4i acc[NI][4];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    const int r16 = lane & 15, q16 = lane >> 4;
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d)
        if (d < nk) copy(d, d * STAGE);
    uint32_t slot = 0;
    for (int s = 0; s < nk; ++s) {
        if (s + DEPTH - 2 < nk) wait_copies_barrier<(DEPTH - 2) * COPIES>();
        else wait_copies_barrier<0>();
        const uint32_t before = slot == 0 ? (DEPTH - 1) * STAGE : slot - STAGE;
        if (s + DEPTH - 1 < nk) copy(s + DEPTH - 1, before);
        const int left = K - 128 * stage(s);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int in_row = r16 * 128 + 16 * ((4 * u + q16) ^ (r16 >> 1));
            v4i fa[4], fb[NI];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                fa[j] = *reinterpret_cast<const v4i*>(&lds[slot + 16 * j * 128 + in_row]);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                fb[i] = *reinterpret_cast<const v4i*>(&lds[slot + (MT_M + 32 * wave + 16 * i) * 128 + in_row]);
            if (left < 128) {
                const int keep = 64 * u + 16 * q16 < left ? -1 : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) fa[j][e] &= keep;
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[i], fa[j], acc[i][j], 0, 0, 0);
        }
        slot = slot == (DEPTH - 1) * STAGE ? 0u : slot + STAGE;
    }

    const float* sb = g.sb + tile.grp * g.N;
    const bool vec_ok = (g.ldc & 3) == 0 && (reinterpret_cast<uintptr_t>(g.c) & 7) == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t m = tile.m0 + j * 16 + r16;
        if (m >= tile.m_end) continue;
        const float sa = g.sa[m];
#pragma unroll
        for (int i = 0; i < NI; i += SWIGLU ? 2 : 1) {
            const int64_t n = n0 + (SWIGLU ? 16 * wave : 32 * wave + 16 * i) + 4 * q16;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n + e >= cols) {
                    v[e] = 0.0f;
                } else if constexpr (SWIGLU) {
                    v[e] = silu_times(int8_value(acc[i][j][e], sa, sb[n + e]),
                                      int8_value(acc[i + 1][j][e], sa, sb[cols + n + e]));
                } else {
                    v[e] = int8_value(acc[i][j][e], sa, sb[n + e]);
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
// One tile a CU: up to 16 MA tokens against `blocks` (at most MOST) 16-row blocks of B, a number that the host chooses so that the
// workgroups are one for each CU, or as near to whole rounds of that as N allows: what a CU copies into LDS takes its time
// whatever asks for it, so the CU with the most bytes decides. Stages of 128 bytes of K in a ring of DEPTH, rows of 128 bytes
// swizzled as in the middle tiles, one barrier for PER stages. The waves share the tile's blocks (SwiGLU: its pairs of a gate
// and an up block) in turn: all four a stage (PER = 1), or waves 0 and 1 the first of two stages and waves 2 and 3 the second,
// and these hand their sums to the former at the end (PER = 2: a barrier's and the fragments' latency for twice the bytes, but
// the ring runs two stages shorter: for tiles of few blocks, which leave room for a long ring; 61 tokens at 8192 x 8192 take
// 20.7 us so and 34.7 with PER = 1, at 36864 x 12288 96 and 88). Every wave issues the same number of copies a stage, those
// past the tile's blocks or past K for a place behind the operand, so that one count serves all waits.
template <int MA, int MOST, int PER, int DEPTH, bool SWIGLU>
__global__ __launch_bounds__(256) void int8_wide_kernel(Int8Gemm g, int blocks) {
    constexpr int COPIES = (MA + MOST + 1) / 2, STAGE = 4096 * COPIES;
    constexpr int SHARE = 4 / PER;                              // waves that share a stage's blocks
    constexpr int NI = SWIGLU ? (MOST / 2 + SHARE - 1) / SHARE * 2 : MOST / SHARE;      // blocks of a wave
    static_assert(PER == 1 || DEPTH * STAGE >= 2 * 64 * NI * MA * 16, "the ring holds two waves' sums");
    __shared__ __attribute__((aligned(16))) uint8_t lds[DEPTH * STAGE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t cols = SWIGLU ? g.N / 2 : g.N;
    const int tc = SWIGLU ? 8 * blocks : 16 * blocks;           // output columns of a tile
    const int tiles_m = (int)((g.M + 16 * MA - 1) / (16 * MA));
    const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * (16 * MA), n0 = (int64_t)(blockIdx.x / tiles_m) * tc;
    const int64_t m_end = m0 + 16 * MA < g.M ? m0 + 16 * MA : g.M;
    const int8_t* B = g.b + n0 * g.K;
    const int K = (int)g.K, nk = (K + 127) / 128;
    const int begin = first_step((uint32_t)(n0 / tc), nk);
    auto stage = [&](int s) { return s + begin < nk ? s + begin : s + begin - nk; };

    // Copy j of a wave fills the 8 rows wave + 4j of a stage: A's 2 MA, then two for each block of B.
    const bool up = SWIGLU && (((wave >> 1) + MA) & 1);         // whether the wave's B rows are up rows
    const v4i rA = rows_rsrc(g.a + m0 * g.K, m_end - m0, g.K);
    const v4i rB = rows_rsrc(up ? B + cols * g.K : B, cols - n0, g.K);
    const uint32_t lds0 = lds_offset(&lds[1024 * wave]);
    int off[COPIES];
#pragma unroll
    for (int j = 0; j < COPIES; ++j) {
        const int e = wave + 4 * j, b = (e - 2 * MA) >> 1;      // eight rows, block of B
        const int row = e < 2 * MA ? 8 * e : 16 * (SWIGLU ? b / 2 : b) + 8 * (e & 1);
        off[j] = (row + (lane >> 3)) * K + 16 * ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
        if (e >= 2 * MA && b >= blocks) off[j] = 0x7FFFFFF0;
    }
    auto copy = [&](int s, uint32_t slot) {
#pragma unroll
        for (int j = 0; j < COPIES; ++j)
            dma_to_lds<16>(wave + 4 * j < 2 * MA ? rA : rB, lds0 + slot + 4096 * j, s < nk ? off[j] : 0x7FFFFFF0,
                           s < nk ? stage(s) * 128 : 0);
    };
    auto next = [](uint32_t slot) { return slot == (DEPTH - 1) * STAGE ? 0u : slot + STAGE; };
    const int part = wave % SHARE, which = wave / SHARE;        // of the blocks, of a barrier's stages
    auto block_of = [&](int x) { return SWIGLU ? 2 * (part + SHARE * (x >> 1)) + (x & 1) : part + SHARE * x; };
    v4i acc[NI][MA];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MA; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    const int r16 = lane & 15, q16 = lane >> 4;
#pragma unroll
    for (int d = 0; d < DEPTH - PER; ++d) copy(d, d * STAGE);
    uint32_t slot = 0, into = (DEPTH - PER) * STAGE;
    for (int s = 0; s < nk; s += PER) {
        // the next PER stages have landed for every wave, and the PER before them have been read
        wait_copies_barrier<(DEPTH - 2 * PER) * COPIES>();
#pragma unroll
        for (int d = 0; d < PER; ++d) {
            copy(s + DEPTH - PER + d, into);
            into = next(into);
        }
        const int mine = s + which;
        const uint32_t at = which ? next(slot) : slot;
        if (mine < nk) {
            const int left = K - 128 * stage(mine);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int in_row = r16 * 128 + 16 * ((4 * u + q16) ^ (r16 >> 1));
                v4i fa[MA];
#pragma unroll
                for (int j = 0; j < MA; ++j) fa[j] = *reinterpret_cast<const v4i*>(&lds[at + 16 * j * 128 + in_row]);
                if (left < 128) {
                    const int keep = 64 * u + 16 * q16 < left ? -1 : 0;
#pragma unroll
                    for (int j = 0; j < MA; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) fa[j][e] &= keep;
                }
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    if (block_of(i) < blocks) {
                        const v4i fb = *reinterpret_cast<const v4i*>(&lds[at + 16 * (MA + block_of(i)) * 128 + in_row]);
#pragma unroll
                        for (int j = 0; j < MA; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb, fa[j], acc[i][j], 0, 0, 0);
                    }
                }
            }
        }
        slot = PER == 2 ? next(next(slot)) : next(slot);
    }
    wait_copies_barrier<0>();                                   // no copy outlives the workgroup's LDS
    if constexpr (PER == 2) {                                   // the second pair's sums, by way of the ring
        v4i* sums = reinterpret_cast<v4i*>(lds) + part * (64 * NI * MA) + lane;
        if (which) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < MA; ++j) sums[64 * (i * MA + j)] = acc[i][j];
        }
        __syncthreads();
        if (which) return;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < MA; ++j) acc[i][j] += sums[64 * (i * MA + j)];
    }
    const bool vec_ok = (g.ldc & 3) == 0 && (reinterpret_cast<uintptr_t>(g.c) & 7) == 0;
#pragma unroll
    for (int i = 0; i < NI; i += SWIGLU ? 2 : 1) {
        if (block_of(i) >= blocks) continue;
        const int64_t n = n0 + (SWIGLU ? 8 : 16) * block_of(i) + 4 * q16;
#pragma unroll
        for (int j = 0; j < MA; ++j) {
            const int64_t m = m0 + 16 * j + r16;
            if (m >= m_end) continue;
            const float sa = g.sa[m];
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n + e >= cols) v[e] = 0.0f;
                else if constexpr (SWIGLU) v[e] = silu_times(int8_value(acc[i][j][e], sa, g.sb[n + e]), int8_value(acc[i + 1][j][e], sa, g.sb[cols + n + e]));
                else v[e] = int8_value(acc[i][j][e], sa, g.sb[n + e]);
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
// Large tiles: 256 x 256 rows of A and B, one workgroup per CU, which takes its tiles in turn (LargeTiles); 4 waves, 2 x 2, each
// 128 x 128 as 8 x 8 accumulators of 16 x 16 (256 registers). K advances 64 bytes per stage: one v_mfma_i32_16x16x64_i8 per
// accumulator. (The chip is held back by its power here: from registers alone, on normally distributed codes, this instruction
// runs at 4.2 POP/s and the 32 x 32 x 32 form at 3.4; on zeros both reach 4.9.) Operand of lane l: row l % 16, bytes 16 (l / 16)
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
// The pairs of a workgroup's tiles are one sequence: while a tile's last pairs are multiplied the next tile's first are copied,
// and they land while its outputs are computed and stored. (With a workgroup for each tile, the search for the tile, the first
// pairs and the scales took 11,000 of 44,000 cycles at K = 1024, where the trips take 23,000.)
// Measured, over calls, boxes and what ran before (the chip's power): 4096 x 36864 x 12288 1.20 to 1.28 ms, 2.9 to 3.1 POP/s (1.22 to
// 1.26 with a workgroup for each tile where these took 1.20); 131072 rows of 64 experts, K = 2048 to 2 x 1024 with SwiGLU 473 to 536
// us, 2.1 to 2.3 POP/s (522 where these took 473), K = 1024 to 2048 307 to 320 us, 1.7 to 1.8 POP/s (357 against 307). What
// is left of a tile beside its trips is mostly the arithmetic on the sums, 8,000 cycles (with SwiGLU 10,000), for which the
// matrix unit waits.
constexpr int LPAIR = 128, LREGION = LT * LPAIR, LREGIONS_A = 3;

typedef float f32x4a __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The same kind of resource as buffer_rsrc's, for loads and stores that the compiler issues and waits for.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int records) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, records, 0x00020000);
}

// acc += b a, and acc = b a. Written as assembly so that the sum stays in its registers: left to itself the compiler gives the
// instruction another destination and copies results about in the loop. The operands' loads are waited for by the compiler; nothing
// else may write an operand or read a sum within 19 wait states (the kernel has 64 instructions between two uses of a
// sum, and waits of its own around the last stage).
__device__ __forceinline__ void mfma_in_place(v4i& acc, v4i b, v4i a) {
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}

__device__ __forceinline__ void mfma_from_zero(v4i& acc, v4i b, v4i a) {
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, 0" : "+a"(acc) : "v"(b), "v"(a));
}

// The tiles that one workgroup takes in turn: every gridDim.x-th of an order in which each XCD (every eighth workgroup) walks a
// contiguous run, so that the workgroups of an XCD share rows and weights in its L2. Grouped: a wave holds the rows of 64 groups
// and the number of row tiles before each, a group a lane, and the next tile costs no memory access until one lies behind those.
// The walk over the groups goes forward only, so a workgroup's tiles must not decrease: int8_plan.h says why they do not.
template <bool GROUPED>
struct LargeTiles {
    const Int8Gemm& g;
    const int tiles_n;
    int tiles_m, T, b = blockIdx.x;     // tiles_m: dense only
    int64_t base = 0, lo = 0, hi = 0;   // lane l: rows of group base + l
    int before = 0, excl = 0, total = 0;

    __device__ __forceinline__ LargeTiles(const Int8Gemm& g_, int tn, int most) : g(g_), tiles_n(tn) {
        if constexpr (GROUPED) {
            load();
            int64_t rows = total;
            if (g.G > 64) {
                for (base = 64; base < g.G; base += 64) {
                    load();
                    rows += total;
                }
                base = 0;
                load();
            }
            T = large_tiles(rows, tiles_n, most);
        } else {
            tiles_m = (int)((g.M + LT - 1) / LT);
            T = tiles_m * tiles_n;
        }
    }
    __device__ __forceinline__ void load() {
        const int lane = threadIdx.x & 63;
        const int64_t q = base + lane;
        lo = hi = 0;
        if (q < g.G) {
            lo = g.offsets[q];
            hi = g.offsets[q + 1];
            lo = lo < 0 ? 0 : (lo > g.M ? g.M : lo);
            hi = hi < lo ? lo : (hi > g.M ? g.M : hi);
        }
        const int nt = (int)((hi - lo + LT - 1) / LT);
        int incl = nt;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(incl, off, 64);
            if (lane >= off) incl += v;
        }
        excl = incl - nt;
        total = __builtin_amdgcn_readlane(incl, 63);
    }
    __device__ __forceinline__ static int64_t lane_value(int64_t v, int lane) {
        return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)v, lane) |
                         (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32);
    }
    __device__ __forceinline__ Int8Tile next() {
        Int8Tile r{0, 0, -1, 0};
        if (b >= T) return r;
        const int v = large_tile(b, T);
        b += (int)gridDim.x;
        if constexpr (GROUPED) {
            const int row = v / tiles_n;
            while (row - before >= total) {
                if (base + 64 >= g.G) return r;
                base += 64;
                before += total;
                load();
            }
            const int at = row - before;
            const int L = 63 - __builtin_clzll(__ballot(excl <= at));     // the last group with that many tiles before it
            r.grp = base + L;
            r.m0 = lane_value(lo, L) + (int64_t)(at - __builtin_amdgcn_readlane(excl, L)) * LT;
            const int64_t end = lane_value(hi, L);
            r.m_end = r.m0 + LT < end ? r.m0 + LT : end;
            r.n = v - row * tiles_n;
        } else {
            // in groups of GROUP_M row tiles
            const int per_group = GROUP_M * tiles_n, first_m = (v / per_group) * GROUP_M;
            const int gm = min(GROUP_M, tiles_m - first_m), x = v % per_group;
            r.grp = 0;
            r.m0 = (int64_t)(first_m + x % gm) * LT;
            r.n = x / gm;
            r.m_end = r.m0 + LT < g.M ? r.m0 + LT : g.M;
        }
        return r;
    }
};

template <bool GROUPED, bool SWIGLU, bool ALIGNED>
__global__ __launch_bounds__(256, 1) void int8_gemm_large_kernel(Int8Gemm g, int most) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[(LREGIONS_A + 2) * LREGION];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int64_t cols = SWIGLU ? g.N / 2 : g.N;
    constexpr int TC = SWIGLU ? LT / 2 : LT;
    LargeTiles<GROUPED> tiles(g, (int)((cols + TC - 1) / TC), most);
    Int8Tile tile = tiles.next();
    if (tile.grp < 0) return;
    const int r16 = lane & 15, q16 = lane >> 4;

    // ------------------------------------------------------------------ copies
    // Copy c (0 .. 7) of a wave fills rows 32c + 8 wave .. + 7 of a region: lane l brings row l / 8 of them, the chunk that
    // belongs at position l % 8. The resources end with the operand: rows behind its end are zeros, rows of A behind the
    // group's are the next group's (their outputs are never stored).
    auto a_rows = [&](const Int8Tile& t) {
        return t.grp < 0 ? buffer_rsrc(g.a, 0) : rows_rsrc(g.a + t.m0 * g.K, g.M - t.m0, g.K);
    };
    auto b_rows = [&](const Int8Tile& t) {                      // SwiGLU: waves 0, 1 bring gate rows, waves 2, 3 up rows
        const int64_t n0 = t.n * TC, row = t.grp * g.N + n0 + (SWIGLU && wave >= 2 ? cols : 0);
        return t.grp < 0 ? buffer_rsrc(g.b, 0) : rows_rsrc(g.b + row * g.K, cols - n0, g.K);
    };
    const int brow = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
    const int K = (int)g.K;
    const int a_off = brow * K + 16 * chunk, b_off = (SWIGLU ? brow & 15 : brow) * K + 16 * chunk;
    const int a_step = 32 * K, b_step = SWIGLU ? 16 * K : 32 * K;
    const uint32_t lds0 = lds_offset(&lds[1024 * wave]);
    constexpr uint32_t B0 = LREGIONS_A * LREGION;               // B's regions
    // Pairs of a tile: at least three, so that copies reach no further ahead than the next tile; a shorter contraction is filled up
    // with pairs whose A is zeros. What the last pair holds past the end of K is zeros in A too (an offset out of range).
    const int pairs = (K + LPAIR - 1) / LPAIR, np = max(pairs, 3), fill = np - pairs;
    const int a_none = 0x70000000, a_last = 16 * chunk < K - LPAIR * (pairs - 1) ? a_off : a_none;
    const int a_first = pairs == 1 ? a_last : a_off;
    // The pairs of one operand in the order they are copied: a tile's, then the next tile's. Behind the last tile an empty operand.
    struct Stream {
        v4i rows;
        int k, step, left, off;                                 // byte of K, what a pair advances it by, pairs left of the tile
    };
    Stream in_a{a_rows(tile), 0, LPAIR, np, a_first}, in_b{b_rows(tile), 0, LPAIR, np, b_off};
    v4i next_a = in_a.rows, next_b = in_b.rows;
    int next_step = 0;
    auto turn = [&](Stream& s, const v4i& next, int off) {      // before a pair's copies
        if (s.left == 0) s = Stream{next, 0, next_step, np, off};
    };
    auto done = [&](Stream& s) {                                // behind them
        s.k += s.step;
        if (--s.left == fill) s.k = s.step = 0;                 // an offset of K past the operand's end would wrap around
    };
    auto aim_a = [&]() { in_a.off = in_a.left > fill + 1 ? a_off : in_a.left == fill + 1 ? a_last : a_none; };
    auto done_a = [&]() {
        done(in_a);
        aim_a();
    };
    auto copy_a = [&](uint32_t into, int c) { dma_to_lds<16>(in_a.rows, lds0 + into + 4096 * c, in_a.off + c * a_step, in_a.k); };
    auto copy_b = [&](uint32_t into, int c) { dma_to_lds<16>(in_b.rows, lds0 + into + 4096 * c, b_off + c * b_step, in_b.k); };

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
        for (int j = 0; j < 8; ++j) asm volatile("" : "=a"(acc[i][j]));        // written by a tile's first trip
    // Everything that writes the sums before this statement has been issued, and nothing that reads them has.
    auto settle = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm volatile("" : "+a"(acc[i][0]), "+a"(acc[i][1]), "+a"(acc[i][2]), "+a"(acc[i][3]), "+a"(acc[i][4]),
                              "+a"(acc[i][5]), "+a"(acc[i][6]), "+a"(acc[i][7]));
    };
    v4i F[2][16];                                               // two sets of fragments

    // One trip in 16 steps of 4 instructions: set P is multiplied (a tile's first trip begins the sums); half P ^ 1 of the pair in
    // regions (a, b) is read into the other set, two fragments in each of the first 8 steps; a copy (copy(c), c = 0 .. 7) goes in
    // every other step.
    auto trip = [&](auto p_c, auto first_c, uint32_t a, uint32_t b, auto&& copy) {
        constexpr int P = decltype(p_c)::value;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int i = q >> 1;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = 4 * (q & 1) + x;
                if constexpr (decltype(first_c)::value) mfma_from_zero(acc[i][j], F[P][8 + i], F[P][j]);
                else mfma_in_place(acc[i][j], F[P][8 + i], F[P][j]);
            }
            if (q < 8) {
                F[P ^ 1][2 * q] = frag(a, b, P ^ 1, 2 * q);
                F[P ^ 1][2 * q + 1] = frag(a, b, P ^ 1, 2 * q + 1);
            }
            if (!(q & 1)) copy(q >> 1);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using T0 = std::integral_constant<int, 0>;
    using T1 = std::integral_constant<int, 1>;
    constexpr std::true_type yes{};
    constexpr std::false_type no{};

    // ------------------------------------------------------------------ prologue: the first tile's pairs 0 and 1
#pragma unroll
    for (int c = 0; c < 8; ++c) copy_a(0, c);
#pragma unroll
    for (int c = 0; c < 8; ++c) copy_b(B0, c);
    done_a();
    done(in_b);
#pragma unroll
    for (int c = 0; c < 8; ++c) copy_a(LREGION, c);
#pragma unroll
    for (int c = 0; c < 8; ++c) copy_b(B0 + LREGION, c);
    done_a();
    done(in_b);
    wait_copies_barrier<16>();
#pragma unroll
    for (int f = 0; f < 16; ++f) F[0][f] = frag(0, B0, 0, f);

    uint32_t a0 = 2 * LREGION, a1 = 0, b0 = B0 + LREGION, b1 = B0;      // regions of the pair before and the next one
    auto next = [&]() {
        a0 = a1;
        a1 = a1 == 2 * LREGION ? 0u : a1 + LREGION;
        const uint32_t x = b0;
        b0 = b1;
        b1 = x;
    };
    auto pair_end = [&]() {
        wait_copies_barrier<8>();
        __builtin_amdgcn_s_waitcnt(0xC07F);                     // the compiler's own view of that wait
        next();
    };
    const int inner = max(np - 4, 0);                           // iterations whose copies are neither a tile's first nor its last pair
    for (;;) {
        trip(T0{}, yes, a1, b1, [&](int c) { copy_a(a0, c); });
        done_a();
        pair_end();
        const Int8Tile after = tiles.next();
        next_a = a_rows(after);
        next_b = b_rows(after);
        next_step = after.grp < 0 ? 0 : LPAIR;
        int p = 0;
        for (; p < inner; ++p) {                                // pairs p + 2 of B, p + 3 of A
            trip(T1{}, no, a1, b1, [&](int c) { copy_b(b0, c); });
            in_b.k += LPAIR;
            trip(T0{}, no, a1, b1, [&](int c) { copy_a(a0, c); });
            in_a.k += LPAIR;
            pair_end();
        }
        in_b.left -= inner;
        in_a.left -= inner;
        aim_a();
        for (; p + 1 < np; ++p) {
            turn(in_b, next_b, b_off);
            trip(T1{}, no, a1, b1, [&](int c) { copy_b(b0, c); });
            done(in_b);
            turn(in_a, next_a, a_first);
            trip(T0{}, no, a1, b1, [&](int c) { copy_a(a0, c); });
            done_a();
            pair_end();
        }

        // -------------------------------------------------------------- scales of the wave's rows and columns
        // Read ahead of the last trip, at addresses that differ by constants: an address, a clamp and a check for each cost more
        // than the arithmetic on the sums (a wave is alone on its SIMD here, four cycles an instruction).
        const int64_t m0 = tile.m0, m_end = tile.m_end, n0 = tile.n * TC, grp = tile.grp;
        const int64_t n_end = n0 + TC < cols ? n0 + TC : cols;
        constexpr int NB = SWIGLU ? 4 : 8;                      // 16-column output blocks of a wave
        const float* sb = g.sb + grp * g.N + n0 + wn * (TC / 2);
        const float* sm = g.sa + m0 + wm * 128;
        float sa[8];
        f32x4a s_gate[NB], s_up[SWIGLU ? NB : 1];
        const int rows_left = (int)(m_end - m0) - wm * 128, cols_left = (int)(n_end - n0) - wn * (TC / 2);    // of the wave
        if constexpr (ALIGNED) {
            // those behind a tile's last row or column are out of the buffer's range and read as zeros
            const auto ra = buffer_of(sm, 4 * max(rows_left, 0)), rg = buffer_of(sb, 4 * max(cols_left, 0));
            const auto ru = buffer_of(sb + cols, SWIGLU ? 4 * max(cols_left, 0) : 0);
#pragma unroll
            for (int j = 0; j < 8; ++j) sa[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ra, 4 * r16 + 64 * j, 0, 0));
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                s_gate[b] = __builtin_bit_cast(f32x4a, __builtin_amdgcn_raw_buffer_load_b128(rg, 16 * q16 + 64 * b, 0, 0));
                if constexpr (SWIGLU)
                    s_up[b] = __builtin_bit_cast(f32x4a, __builtin_amdgcn_raw_buffer_load_b128(ru, 16 * q16 + 64 * b, 0, 0));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) sa[j] = sm[min(16 * j + r16, rows_left - 1)];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s_gate[b][e] = sb[min(16 * b + 4 * q16 + e, cols_left - 1)];
                    if constexpr (SWIGLU) s_up[b][e] = sb[cols + min(16 * b + 4 * q16 + e, cols_left - 1)];
                }
        }
        turn(in_b, next_b, b_off);
        trip(T1{}, no, a1, b1, [&](int c) { copy_b(b0, c); });
        asm volatile("s_nop 15\n\ts_nop 15");                   // the matrix instructions' results to what reads them
        settle();

        // ------------------------------------------------------------------ epilogue
        // Lane l holds columns 4 (l / 16) .. + 3 of row l % 16 of each 16 x 16 block. Two blocks side by side swap every other
        // 16-lane row (v_permlane16_swap), which leaves a lane with 8 consecutive columns of one of them: lanes of row R hold
        // columns 16 (R % 2) + 8 (R / 2) .. of the pair's 32, and a 16-byte store writes 64 contiguous bytes into each of 16
        // rows.
        // output columns 32p .. of the wave, row block j: 8 consecutive ones of its row for each lane
        auto outputs = [&](int p, int j) {
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
            return u32x4{(uint32_t)x[0], (uint32_t)y[0], (uint32_t)x[1], (uint32_t)y[1]};
        };
        const int col0 = 16 * (q16 & 1) + 8 * (q16 >> 1);                               // of the lane, within the wave's
        uint16_t* dst = g.c + (m0 + wm * 128) * g.ldc + n0 + wn * (TC / 2);
        if constexpr (ALIGNED) {
            const uint32_t row_bytes = 2 * (uint32_t)g.ldc;
            const auto rc = buffer_of(dst, (int)(max(rows_left, 0) * row_bytes));      // rows behind the last stay as they were
            uint32_t at[NB / 2];
#pragma unroll
            for (int p = 0; p < NB / 2; ++p) at[p] = col0 + 32 * p < cols_left ? r16 * row_bytes + 2 * (col0 + 32 * p) : 0x7F000000u;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int p = 0; p < NB / 2; ++p)
                    __builtin_amdgcn_raw_buffer_store_b128(outputs(p, j), rc, (int)(at[p] + 16 * j * row_bytes), 0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint16_t* row = dst + (r16 + 16 * j) * g.ldc + col0;
#pragma unroll
                for (int p = 0; p < NB / 2; ++p) {
                    const u32x4 d = outputs(p, j);
                    const int left = r16 + 16 * j < rows_left ? cols_left - col0 - 32 * p : 0;   // columns from this lane's first on
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < left) row[32 * p + e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
        done(in_b);
        if (after.grp < 0) break;
        tile = after;
        settle();
    }
    wait_copies_barrier<0>();                                   // no copy may arrive behind the workgroup's end
}

// ---------------------------------------------------------------------------------------------------------------
// Few tokens: the work is reading the weights once. A workgroup takes 16 NT rows of B (SwiGLU: 16 gate rows and the up rows
// of the same columns) for up to 16 MT tokens; its 4 waves share the contraction, 128 bytes of every row at a time, and each
// runs on its own: a ring of DEPTH such steps in LDS, filled past the registers by copies of whole lines (8 rows of 128 bytes
// an instruction; loads of 16 rows of 64 bytes, as the matrix instruction wants them, read at 3.5 to 4.8 TB/s where these
// read at 5.7 to 6.5), rows of 128 bytes swizzled as in the large tiles. The waves' sums meet in LDS by integer additions,
// whose order does not matter. Measured: 1 x 6144 x 2048 5.2 us; 16 tokens through 8 of 64 experts each, K = 2048 to 2 x 1024
// with SwiGLU, 43.6 us (the chosen experts' weights at 5.4 TB/s).
constexpr int FEW_W = 4;
template <int MT, int NT, int DEPTH, bool GROUPED, bool SWIGLU>
__global__ __launch_bounds__(64 * FEW_W) void int8_few_kernel(Int8Gemm g) {
    constexpr int W = FEW_W;
    constexpr int STEP = 16 * (NT + MT) * 128, COPIES = STEP / 1024;
    constexpr int PITCH = 16 * MT + 4;                          // words: the four row groups of a wave on banks of their own
    __shared__ __attribute__((aligned(16))) uint8_t ring[W][DEPTH][STEP];
    __shared__ int sums[16 * NT][PITCH];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t cols = SWIGLU ? g.N / 2 : g.N;
    constexpr int TC = SWIGLU ? 8 * NT : 16 * NT;               // output columns of a workgroup
    const int64_t tiles_n = (cols + TC - 1) / TC;
    const int64_t n0 = (blockIdx.x % tiles_n) * TC;
    int64_t m0, m_end, grp = 0;
    if constexpr (GROUPED) {
        const RowTile rt = find_row_tile<16 * MT>(g.offsets, g.G, g.M, blockIdx.x / tiles_n);
        if (rt.grp < 0) return;
        grp = rt.grp;
        m0 = rt.lo;
        m_end = rt.lo + 16 * MT < rt.hi ? rt.lo + 16 * MT : rt.hi;
    } else {
        m0 = (blockIdx.x / tiles_n) * (16 * MT);
        m_end = m0 + 16 * MT < g.M ? m0 + 16 * MT : g.M;
    }
    const int rows = (int)(m_end - m0), K = (int)g.K;
    const int r16 = lane & 15, q16 = lane >> 4;
    for (int i = tid; i < 16 * NT * PITCH; i += 64 * W) (&sums[0][0])[i] = 0;

    // The wave's steps are its pieces wave + W i of 128 bytes, from a place of the workgroup's own on. Copies of steps past the
    // last ask for a place behind the operands.
    // Rows behind an operand's end, and bytes past K, are zeros or a neighbour's: the sums of the first are not stored, the
    // second are masked in A.
    const int8_t* B = g.b + (grp * g.N + n0) * g.K;
    const v4i rA = rows_rsrc(g.a + m0 * g.K, rows, g.K);
    const v4i rB = rows_rsrc(B, cols - n0, g.K);
    const v4i rU = SWIGLU ? rows_rsrc(B + cols * g.K, cols - n0, g.K) : rB;
    const int pieces = (K + 127) / 128, steps = (pieces + W - 1 - wave) / W;
    const int begin = GROUPED ? 0 : first_step((uint32_t)(n0 / TC), steps);
    auto piece = [&](int s) { return wave + W * (s + begin < steps ? s + begin : s + begin - steps); };
    const int at[2] = {(lane >> 3) * K + 16 * ((lane & 7) ^ (lane >> 4)), (lane >> 3) * K + 16 * ((lane & 7) ^ 4 ^ (lane >> 4))};
    const uint32_t lds0 = lds_offset(&ring[wave][0][0]);
    auto copy = [&](int s, uint32_t slot) {
        const int k = s < steps ? 128 * piece(s) : 0x7F000000;
#pragma unroll
        for (int c = 0; c < COPIES; ++c) {
            const int row = 8 * c;                              // of the ring: B's 16 NT, then A's
            const bool b = row < 16 * NT;
            const int r = !b ? row - 16 * NT : SWIGLU ? 16 * (row / 32) + row % 16 : row;
            dma_to_lds<16>(!b ? rA : SWIGLU && (row & 16) ? rU : rB, lds0 + slot + 1024 * c, at[c & 1] + r * K + k, 0);
        }
    };
    v4i acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = v4i{0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) copy(d, d * STEP);
    uint32_t slot = 0;
    for (int s = 0; s < steps; ++s) {
        asm volatile("s_waitcnt vmcnt(%0)" :: "n"((DEPTH - 1) * COPIES) : "memory");    // step s has landed
        v4i f[2][NT + MT];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < NT + MT; ++i)
                f[u][i] = *reinterpret_cast<const v4i*>(&ring[wave][0][slot + (16 * i + r16) * 128 + 16 * ((4 * u + q16) ^ (r16 >> 1))]);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");                              // and has been read
        copy(s + DEPTH, slot);
        slot = slot == (DEPTH - 1) * STEP ? 0u : slot + STEP;
        const int left = K - 128 * piece(s);
        if (left < 128) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int keep = 64 * u + 16 * q16 < left ? -1 : 0;
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[u][NT + j][e] &= keep;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f[u][i], f[u][NT + j], acc[i][j], 0, 0, 0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");            // no copy outlives the workgroup's LDS
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) atomicAdd(&sums[16 * i + 4 * q16 + e][16 * j + r16], acc[i][j][e]);
    __syncthreads();
    const float* sb = g.sb + grp * g.N;
    for (int i = tid; i < TC * rows; i += 64 * W) {
        const int c = i % TC, m = i / TC;
        if (n0 + c >= cols) continue;
        const float sa = g.sa[m0 + m];
        float v;
        if constexpr (SWIGLU) {
            const int r = 32 * (c / 16) + c % 16;
            v = silu_times(int8_value(sums[r][m], sa, sb[n0 + c]), int8_value(sums[r + 16][m], sa, sb[cols + n0 + c]));
        } else {
            v = int8_value(sums[c][m], sa, sb[n0 + c]);
        }
        g.c[(m0 + m) * g.ldc + n0 + c] = (uint16_t)pack_bf16(v, 0.0f);
    }
}

bool int8_gemm_fits(int64_t M, int64_t cols, int64_t K, int64_t G, int swiglu) {
    return int8_plan(M, cols, K, G, swiglu != 0).blocks <= kMaxThreads / 256;
}

template <int MOST, bool SWIGLU>
static void launch_wide(const Int8Gemm& g, const Int8Plan& p, hipStream_t stream) {
    const dim3 blocks((unsigned)p.blocks), threads(256);
    constexpr bool S = MOST == 4;
    constexpr int PER = S ? 2 : 1;
    if (p.rows == 16) hipLaunchKernelGGL((int8_wide_kernel<1, MOST, PER, S ? 12 : 5, SWIGLU>), blocks, threads, 0, stream, g, p.wide);
    else if (p.rows == 32) hipLaunchKernelGGL((int8_wide_kernel<2, MOST, PER, S ? 12 : 5, SWIGLU>), blocks, threads, 0, stream, g, p.wide);
    else if (p.rows == 64) hipLaunchKernelGGL((int8_wide_kernel<4, MOST, PER, S ? 10 : 5, SWIGLU>), blocks, threads, 0, stream, g, p.wide);
    else hipLaunchKernelGGL((int8_wide_kernel<8, MOST, PER, S ? 6 : 4, SWIGLU>), blocks, threads, 0, stream, g, p.wide);
}

template <bool GROUPED, bool SWIGLU>
static void launch_products(const Int8Gemm& g, int64_t cols, hipStream_t stream) {
    const Int8Plan p = int8_plan(g.M, cols, g.K, g.G, SWIGLU);
    const dim3 blocks((unsigned)p.blocks), threads(256);
    // 16-byte stores by 32-bit offsets within a tile
    const bool aligned = cols % 8 == 0 && g.ldc % 8 == 0 && g.ldc < (1 << 21) && (reinterpret_cast<uintptr_t>(g.c) & 15) == 0;
    const dim3 cus((unsigned)large_groups(p.blocks));
    if (p.kind == INT8_LARGE && aligned) hipLaunchKernelGGL((int8_gemm_large_kernel<GROUPED, SWIGLU, true>), cus, threads, 0, stream, g, (int)p.blocks);
    else if (p.kind == INT8_LARGE) hipLaunchKernelGGL((int8_gemm_large_kernel<GROUPED, SWIGLU, false>), cus, threads, 0, stream, g, (int)p.blocks);
    else if (p.kind == INT8_MIDDLE && p.deep) hipLaunchKernelGGL((int8_gemm_kernel<3, GROUPED, SWIGLU>), blocks, threads, 0, stream, g);
    else if (p.kind == INT8_MIDDLE) hipLaunchKernelGGL((int8_gemm_kernel<2, GROUPED, SWIGLU>), blocks, threads, 0, stream, g);
    else if (p.kind == INT8_WIDE && p.wide <= 4) launch_wide<4, SWIGLU>(g, p, stream);
    else if (p.kind == INT8_WIDE) launch_wide<12, SWIGLU>(g, p, stream);
    else if (p.rows == 16) hipLaunchKernelGGL((int8_few_kernel<1, SWIGLU ? 2 : 1, 2, GROUPED, SWIGLU>), blocks, threads, 0, stream, g);
    else if (p.rows == 32) hipLaunchKernelGGL((int8_few_kernel<2, 2, 2, GROUPED, SWIGLU>), blocks, threads, 0, stream, g);
    else hipLaunchKernelGGL((int8_few_kernel<4, 2, 3, GROUPED, SWIGLU>), blocks, threads, 0, stream, g);
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
