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
                    v[e] = swiglu_f32(int8_value(acc[i][j][e], s, sb[n + e]),
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

// Upper bound of the row tiles of TH rows over ragged groups: every group with rows adds at most one partial tile.
static int64_t most_row_tiles(int64_t rows, int64_t G, int64_t TH) { return (rows + TH - 1) / TH + (G < rows ? G : rows); }

int64_t int8_gemm_blocks(int64_t M, int64_t cols, int64_t G, int swiglu) {
    const int64_t tc = swiglu ? QT / 2 : QT;
    const int64_t tiles_n = (cols + tc - 1) / tc, tiles_m = G ? most_row_tiles(M, G, QT) : (M + QT - 1) / QT;
    return tiles_n > 0 && tiles_m > INT64_MAX / tiles_n ? INT64_MAX : tiles_m * tiles_n;
}

hipError_t launch_int8_gemm(const int8_t* a_q, const float* a_scale, const int64_t* offsets, int64_t G, int64_t M,
                            const int8_t* b_q, const float* b_scale, int64_t N, int64_t K, int swiglu, uint16_t* c,
                            int64_t ldc, hipStream_t stream) {
    const Int8Gemm g{a_q, b_q, a_scale, b_scale, c, M, N, K, ldc, offsets, G};
    const dim3 blocks((unsigned)int8_gemm_blocks(M, swiglu ? N / 2 : N, G, swiglu));
    if (G) {
        if (swiglu) hipLaunchKernelGGL((int8_gemm_kernel<true, true>), blocks, dim3(256), 0, stream, g);
        else hipLaunchKernelGGL((int8_gemm_kernel<true, false>), blocks, dim3(256), 0, stream, g);
    } else {
        if (swiglu) hipLaunchKernelGGL((int8_gemm_kernel<false, true>), blocks, dim3(256), 0, stream, g);
        else hipLaunchKernelGGL((int8_gemm_kernel<false, false>), blocks, dim3(256), 0, stream, g);
    }
    return hipGetLastError();
}

}  // namespace mxq
