// RMSNorm with the residual's addition and an MXFP8 output, and its backward from an 8-bit checkpoint, for gfx950.
//
// Forward:   h = bf16(x + r)   (h = x without a residual)
//            rstd = 1 / sqrt(sum_c h^2 / cols + eps)
//            y = (h rstd) gamma                             each operation rounded to fp32 on its own
//            MXFP8 of y along rows and / or down columns; MXFP8 of h along rows (the 8-bit checkpoint)
// Backward:  xh = h^ rstd with h^ the checkpoint's values, g = dy gamma, m = sum_c(g xh) / cols
//            dx = bf16(dr + rstd (g - xh m)),  dgamma[c] = sum_rows dy xh
#pragma clang fp contract(off)
#include "launch.h"
#include "mx_block.h"

namespace mxq {

struct NormArgs {
    const uint16_t* x;
    const uint16_t* res;
    const float* gamma;
    int64_t rows, cols;
    float eps;
    uint16_t* sum;              // may be x or res: a lane writes the values it has read
    float* rstd;
    uint8_t *q_row, *s_row, *q_col, *s_col, *ck_q, *ck_s;
};

// ---------------------------------------------------------------------------------------- forward, row form
// W waves per row, NCH chunks of 8 values per lane: chunk j of lane l of the row's waves is l + 64 W j, so a wave's
// loads are contiguous and a 32-value block is one quad of lanes. W < 4 packs 4 / W rows into a workgroup.
template <int RULE, int W, int NCH>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void norm_row_kernel(NormArgs a) {
    constexpr int ROWS = W < 4 ? 4 / W : 1;              // rows per workgroup
    __shared__ float part[W > 1 ? ROWS * W : 1];
    const int t = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W);
    const int64_t row = (int64_t)blockIdx.x * ROWS + sub;
    const bool row_ok = row < a.rows;
    const int chunks = (int)(a.cols / 8);
    uint4 h[NCH];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int ch = t + 64 * W * j;
        h[j] = make_uint4(0u, 0u, 0u, 0u);
        if (row_ok && ch < chunks) {
            const int64_t at = row * a.cols + 8 * ch;
            h[j] = ldnt16(a.x + at);
            if (a.res) {
                const uint4 r = ldnt16(a.res + at);
                float u[8], v[8];
                unpack8(h[j], u);
                unpack8(r, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = u[e] + v[e];
                h[j] = pack8(u);
                *reinterpret_cast<uint4*>(a.sum + at) = h[j];
            }
        }
        float v[8];
        unpack8(h[j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
    }
    ss = wave_sum(ss);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
        __syncthreads();
        ss = part[sub * W];
#pragma unroll
        for (int w = 1; w < W; ++w) ss += part[sub * W + w];
    }
    const float rstd = 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);
    if (row_ok && t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int ch = t + 64 * W * j;
        if (!(row_ok && ch < chunks)) continue;          // whole quads: cols is a multiple of 32
        const int64_t at = row * a.cols + 8 * ch;
        const int64_t sat = row * (a.cols / 32) + ch / 4;
        uint32_t byte;
        if (a.ck_q) {
            stnt8(a.ck_q + at, encode_row8_bf16<RULE>(h[j], byte));
            if ((ch & 3) == 0) a.ck_s[sat] = (uint8_t)byte;
        }
        if (a.q_row) {
            const float4 g0 = *reinterpret_cast<const float4*>(a.gamma + 8 * ch);
            const float4 g1 = *reinterpret_cast<const float4*>(a.gamma + 8 * ch + 4);
            const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
            float y[8];
            unpack8(h[j], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = (y[e] * rstd) * g[e];
            stnt8(a.q_row + at, encode_row8<RULE>(y, byte));
            if ((ch & 3) == 0) a.s_row[sat] = (uint8_t)byte;
        }
    }
}

// ---------------------------------------------------------------------------------------- forward, column form
// A 128 x 128 tile of h per 256-thread workgroup, through LDS: thread (p, b) reads the column pair 2p, 2p + 1 of rows
// 32 b .. 32 b + 31 and forms y twice (for the block maximum, then for the codes) rather than keep 64 fp32 values.
// The codes pass through LDS once more so that each column's 128 codes leave as 16-byte pieces of whole lines.
constexpr int NT = 128;

template <int RULE>
__global__ __launch_bounds__(256) void norm_col_kernel(const uint16_t* h, const float* gamma, const float* rstd,
                                                      int64_t rows, int64_t cols, uint8_t* q_col, uint8_t* s_col) {
    __shared__ __attribute__((aligned(16))) uint32_t lds[NT * NT / 2];
    __shared__ __attribute__((aligned(16))) float rs[NT];
    const int tid = threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.y * NT, c0 = (int64_t)blockIdx.x * NT;
    const int ch = tid & 15;
    const int64_t gc = c0 + 8 * ch;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int lr = (tid >> 4) + 16 * j;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (gc < cols && r0 + lr < rows) v = *reinterpret_cast<const uint4*>(h + (r0 + lr) * cols + gc);
        *reinterpret_cast<uint4*>(&lds[lr * (NT / 2) + 4 * ch]) = v;
    }
    if (tid < NT) rs[tid] = r0 + tid < rows ? rstd[r0 + tid] : 0.0f;
    const int p = tid & 63, b = tid >> 6;
    float g0 = 0.0f, g1 = 0.0f;
    if (c0 + 2 * p < cols) {                                     // cols is even
        g0 = gamma[c0 + 2 * p];
        g1 = gamma[c0 + 2 * p + 1];
    }
    __syncthreads();
    uint32_t d[32];
    float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; r += 2) {
        d[r] = lds[(32 * b + r) * (NT / 2) + p];
        d[r + 1] = lds[(32 * b + r + 1) * (NT / 2) + p];
        const float2 k = *reinterpret_cast<const float2*>(&rs[32 * b + r]);
        t0 = amax3(t0, (bf16_lo(d[r]) * k.x) * g0, (bf16_lo(d[r + 1]) * k.y) * g0);
        t1 = amax3(t1, (bf16_hi(d[r]) * k.x) * g1, (bf16_hi(d[r + 1]) * k.y) * g1);
    }
    const uint32_t m0 = __float_as_uint(t0) & 0x7FFFFFFFu, m1 = __float_as_uint(t1) & 0x7FFFFFFFu;
    const uint32_t b0 = mx_scale_byte_f32(m0, RULE), b1 = mx_scale_byte_f32(m1, RULE);
    uint32_t o0[8], o1[8];
    const bool plain = block_is_plain<RULE>(m0) && block_is_plain<RULE>(m1);
    const float s0 = plain ? scale_operand(b0) : mx_inv_scale_f32(b0), s1 = plain ? scale_operand(b1) : mx_inv_scale_f32(b1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 k = *reinterpret_cast<const float4*>(&rs[32 * b + 4 * i]);
        const uint32_t* q = d + 4 * i;
        const float y0 = (bf16_lo(q[0]) * k.x) * g0, y1 = (bf16_lo(q[1]) * k.y) * g0, y2 = (bf16_lo(q[2]) * k.z) * g0,
                    y3 = (bf16_lo(q[3]) * k.w) * g0;
        const float z0 = (bf16_hi(q[0]) * k.x) * g1, z1 = (bf16_hi(q[1]) * k.y) * g1, z2 = (bf16_hi(q[2]) * k.z) * g1,
                    z3 = (bf16_hi(q[3]) * k.w) * g1;
        if (plain) {
            o0[i] = encode4_plain(y0, y1, y2, y3, s0);
            o1[i] = encode4_plain(z0, z1, z2, z3, s1);
        } else {
            o0[i] = encode4(y0, y1, y2, y3, s0);
            o1[i] = encode4(z0, z1, z2, z3, s1);
        }
    }
    __syncthreads();                                             // every column pair has been read
    uint8_t* ob = reinterpret_cast<uint8_t*>(lds);               // 128 x 128 codes, then 128 x 4 scale bytes
    const int ce = 2 * p, co = 2 * p + 1, sw = p & 7;            // 16-byte piece k of column c sits at k ^ (c/2 % 8)
    uint4* e = reinterpret_cast<uint4*>(ob + ce * NT);
    uint4* o = reinterpret_cast<uint4*>(ob + co * NT);
    e[(2 * b) ^ sw] = make_uint4(o0[0], o0[1], o0[2], o0[3]);
    e[(2 * b + 1) ^ sw] = make_uint4(o0[4], o0[5], o0[6], o0[7]);
    o[(2 * b) ^ sw] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
    o[(2 * b + 1) ^ sw] = make_uint4(o1[4], o1[5], o1[6], o1[7]);
    ob[NT * NT + 4 * ce + b] = (uint8_t)b0;
    ob[NT * NT + 4 * co + b] = (uint8_t)b1;
    __syncthreads();
    const int k = tid & 7;
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        const int c = 32 * pass + (tid >> 3);
        if (c0 + c < cols && r0 + 16 * k < rows)                 // rows % 32 == 0: a 16-row piece is whole
            *reinterpret_cast<uint4*>(q_col + (c0 + c) * rows + r0 + 16 * k) =
                *reinterpret_cast<const uint4*>(ob + c * NT + 16 * (k ^ ((c >> 1) & 7)));
    }
    if (tid < NT && c0 + tid < cols) {
        uint8_t* dst = s_col + (c0 + tid) * (rows / 32) + r0 / 32;
        for (int q = 0; q < 4 && r0 + 32 * q < rows; ++q) dst[q] = ob[NT * NT + 4 * tid + q];
    }
}

// ---------------------------------------------------------------------------------------- backward
// A workgroup walks rows blockIdx.x, blockIdx.x + gridDim.x, ... with the row split over W waves as in the forward;
// each lane keeps gamma and its columns' dgamma sums in registers over all its rows and writes one partial row of
// dgamma at the end. norm_dgamma_kernel adds the partial rows in a fixed order, so the result does not depend on timing.
template <int W, int NCH>
__global__ __launch_bounds__(64 * W) void norm_bwd_kernel(const uint16_t* dy, const uint16_t* dres, const uint8_t* ck_q,
                                                        const uint8_t* ck_s, const float* rstd, const float* gamma,
                                                        int64_t rows, int64_t cols, uint16_t* dx, float* partial) {
    __shared__ float part[2][W];
    const int t = threadIdx.x;
    const int chunks = (int)(cols / 8);
    float g[NCH][8], acc[NCH][8];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int ch = t + 64 * W * j;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[j][e] = 0.0f;
            g[j][e] = ch < chunks ? gamma[8 * ch + e] : 0.0f;
        }
    }
    int par = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, par ^= 1) {
        const float rs = rstd[row];
        float xh[NCH][8];
        uint4 d[NCH];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int ch = t + 64 * W * j;
            if (ch < chunks) {
                const int64_t at = row * cols + 8 * ch;
                d[j] = ldnt16(dy + at);
                dequant8(ldnt8(ck_q + at), e8m0_value(ck_s[row * (cols / 32) + ch / 4]), xh[j]);
            } else {
                d[j] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int e = 0; e < 8; ++e) xh[j][e] = 0.0f;
            }
            float v[8];
            unpack8(d[j], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[j][e] = xh[j][e] * rs;
                acc[j][e] += v[e] * xh[j][e];
                dot += (v[e] * g[j][e]) * xh[j][e];
            }
        }
        dot = wave_sum(dot);
        if constexpr (W > 1) {
            if ((t & 63) == 0) part[par][t >> 6] = dot;          // two buffers: one barrier per row suffices
            __syncthreads();
            dot = part[par][0];
#pragma unroll
            for (int w = 1; w < W; ++w) dot += part[par][w];
        }
        const float m = dot / (float)cols;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int ch = t + 64 * W * j;
            if (ch >= chunks) continue;
            const int64_t at = row * cols + 8 * ch;
            float v[8], r[8];
            unpack8(d[j], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = rs * (v[e] * g[j][e] - xh[j][e] * m);
            if (dres) {
                unpack8(ldnt16(dres + at), r);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = r[e] + v[e];
            }
            stnt16(dx + at, pack8(v));
        }
    }
    if (partial) {
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int ch = t + 64 * W * j;
            if (ch >= chunks) continue;
            float* o = partial + (int64_t)blockIdx.x * cols + 8 * ch;
            *reinterpret_cast<float4*>(o) = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
            *reinterpret_cast<float4*>(o + 4) = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
        }
    }
}

// dgamma[c] = (accumulate ? dgamma[c] : 0) + sum of the partial rows: 32 columns x 8 slices of the rows per workgroup.
__global__ __launch_bounds__(256) void norm_dgamma_kernel(const float* partial, int parts, int64_t cols, float* dgamma,
                                                         int accumulate) {
    __shared__ float s[8][32];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + c;            // cols % 32 == 0
    float v = 0.0f;
    for (int p = k; p < parts; p += 8) v += partial[(int64_t)p * cols + col];
    s[k][c] = v;
    __syncthreads();
    if (k == 0) {
#pragma unroll
        for (int q = 1; q < 8; ++q) v += s[q][c];
        dgamma[col] = accumulate ? dgamma[col] + v : v;
    }
}

// ---------------------------------------------------------------------------------------- launchers
template <int RULE, int W, int NCH>
static void run_row(const NormArgs& a, hipStream_t stream) {
    constexpr int ROWS = W < 4 ? 4 / W : 1;
    hipLaunchKernelGGL((norm_row_kernel<RULE, W, NCH>), dim3((unsigned)((a.rows + ROWS - 1) / ROWS)),
                       dim3(W < 4 ? 256 : 64 * W), 0, stream, a);
}

template <int RULE>
static void run_norm(const NormArgs& a, hipStream_t stream) {
    if (a.cols <= 512) run_row<RULE, 1, 1>(a, stream);
    else if (a.cols <= 1024) run_row<RULE, 1, 2>(a, stream);
    else if (a.cols <= 2048) run_row<RULE, 1, 4>(a, stream);
    else if (a.cols <= 4096) run_row<RULE, 4, 2>(a, stream);
    else if (a.cols <= 8192) run_row<RULE, 4, 4>(a, stream);
    else if (a.cols <= 12288) run_row<RULE, 8, 3>(a, stream);
    else run_row<RULE, 16, 4>(a, stream);
    if (a.q_col) {
        const dim3 grid((unsigned)((a.cols + NT - 1) / NT), (unsigned)((a.rows + NT - 1) / NT));
        hipLaunchKernelGGL((norm_col_kernel<RULE>), grid, dim3(256), 0, stream, a.res ? a.sum : a.x, a.gamma, a.rstd,
                           a.rows, a.cols, a.q_col, a.s_col);
    }
}

hipError_t launch_rmsnorm_mx_quantize(const uint16_t* x, const uint16_t* res, const float* gamma, int64_t rows,
                                      int64_t cols, float eps, uint16_t* sum, float* rstd, uint8_t* q_row,
                                      uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, uint8_t* ck_q, uint8_t* ck_s,
                                      int rule, hipStream_t stream) {
    const NormArgs a{x, res, gamma, rows, cols, eps, sum, rstd, q_row, s_row, q_col, s_col, ck_q, ck_s};
    if (rule == RULE_FLOOR) run_norm<RULE_FLOOR>(a, stream);
    else run_norm<RULE_RCEIL>(a, stream);
    return hipGetLastError();
}

int rmsnorm_backward_parts(int64_t rows) { return (int)(rows < kNormBwdParts ? rows : kNormBwdParts); }

hipError_t launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* dres, const uint8_t* ck_q, const uint8_t* ck_s,
                                   const float* rstd, const float* gamma, int64_t rows, int64_t cols, uint16_t* dx,
                                   float* dgamma, int accumulate, float* partial, hipStream_t stream) {
    const int parts = rmsnorm_backward_parts(rows);
    float* part = dgamma ? partial : nullptr;
#define MXQ_NORM_BWD(W, N)                                                                                          \
    hipLaunchKernelGGL((norm_bwd_kernel<W, N>), dim3((unsigned)parts), dim3(64 * W), 0, stream, dy, dres, ck_q, ck_s, \
                       rstd, gamma, rows, cols, dx, part)
    if (rows > 0) {
        if (cols <= 512) MXQ_NORM_BWD(1, 1);
        else if (cols <= 1024) MXQ_NORM_BWD(2, 1);
        else if (cols <= 2048) MXQ_NORM_BWD(4, 1);
        else if (cols <= 4096) MXQ_NORM_BWD(4, 2);
        else if (cols <= 8192) MXQ_NORM_BWD(8, 2);
        else if (cols <= 12288) MXQ_NORM_BWD(8, 3);
        else if (cols <= 16384) MXQ_NORM_BWD(16, 2);
        else MXQ_NORM_BWD(16, 4);
    }
#undef MXQ_NORM_BWD
    if (dgamma)
        hipLaunchKernelGGL(norm_dgamma_kernel, dim3((unsigned)(cols / 32)), dim3(256), 0, stream, partial, parts, cols,
                           dgamma, accumulate);
    return hipGetLastError();
}

}  // namespace mxq
