// SwiGLU with an 8-bit checkpoint of its input, and its backward from that checkpoint, for gfx950.
//
// Forward:   c = (g | u), h = silu(g) u in fp32 (swiglu_f32: one rounding per operation)
//            MXFP8 of h along rows (the down projection's operand) and MXFP8 of c along rows (the checkpoint, 33/32
//            bytes a value instead of c's 2)
// Backward:  from c^ = (g^ | u^), the checkpoint's values, and dh:
//            dc = ((dh u^) silu'(g^) | dh silu(g^)) in MXFP8, both orientations, and h^ = silu(g^) u^ in MXFP8 down
//            columns (the down projection's Wgrad operand), which the forward therefore need not keep.
#pragma clang fp contract(off)
#include "launch.h"
#include "mx_block.h"

namespace mxq {

// ---------------------------------------------------------------------------------------- forward
// One 8-value chunk of g and of u per thread; a quad of lanes holds a 32-value block of each (F % 32 == 0).
template <int RULE>
__global__ __launch_bounds__(256) void swiglu_ck_fwd_kernel(const uint16_t* __restrict__ c, int64_t rows, int64_t F,
                                                          uint8_t* __restrict__ q, uint8_t* __restrict__ s,
                                                          uint8_t* __restrict__ ck_q, uint8_t* __restrict__ ck_s) {
    const uint32_t per_row = (uint32_t)(F / 8);
    const int64_t base = (int64_t)blockIdx.x * 256;
    const int64_t row0 = base / per_row;                         // uniform over the workgroup
    const uint32_t local = (uint32_t)(base - row0 * per_row) + threadIdx.x;
    const uint32_t dr = local / per_row;
    const int64_t r = row0 + dr, j = 8 * (int64_t)(local - dr * per_row);
    if (r >= rows) return;
    const uint4 gv = ldnt16(c + r * 2 * F + j);
    const uint4 uv = ldnt16(c + r * 2 * F + F + j);
    float g[8], u[8], h[8];
    unpack8(gv, g);
    unpack8(uv, u);
    float sig[8];
    silu8(g, h, sig);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = h[e] * u[e];
    uint32_t bh, bg, bu;
    stnt8(q + r * F + j, encode_row8<RULE>(h, bh));
    stnt8(ck_q + r * 2 * F + j, encode_row8_bf16<RULE>(gv, bg));
    stnt8(ck_q + r * 2 * F + F + j, encode_row8_bf16<RULE>(uv, bu));
    if ((threadIdx.x & 3) == 0) {
        s[r * (F / 32) + j / 32] = (uint8_t)bh;
        ck_s[r * (F / 16) + j / 32] = (uint8_t)bg;
        ck_s[r * (F / 16) + F / 32 + j / 32] = (uint8_t)bu;
    }
}

// ---------------------------------------------------------------------------------------- backward
constexpr int CT_ROWS = 64, CT_COLS = 128;

// Column form of one fp32 tile held as x[j][e] (row tid / 16 + 16 j, column 8 (tid % 16) + e): through LDS to a thread
// per column and 32-row block.
template <int RULE>
__device__ __forceinline__ void ck_col_out(const float (&x)[4][8], float* tile, int64_t r0, int64_t c0, int64_t climit,
                                           int64_t oc0, int64_t rows, uint8_t* __restrict__ q_col,
                                           uint8_t* __restrict__ s_col) {
    const int tid = threadIdx.x, ch = tid & 15, rr = tid >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float* dst = &tile[(rr + 16 * j) * CT_COLS + 8 * ch];
        *reinterpret_cast<float4*>(dst) = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(x[j][4], x[j][5], x[j][6], x[j][7]);
    }
    __syncthreads();
    const int c = tid & (CT_COLS - 1), b = tid >> 7;
    float d[32], top = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; r += 2) {
        d[r] = tile[(32 * b + r) * CT_COLS + c];
        d[r + 1] = tile[(32 * b + r + 1) * CT_COLS + c];
        top = amax3(top, d[r], d[r + 1]);
    }
    __syncthreads();                                             // the tile may be refilled after this
    const uint32_t m = __float_as_uint(top) & 0x7FFFFFFFu;
    const uint32_t byte = mx_scale_byte_f32(m, RULE);
    uint32_t o[8];
    if (block_is_plain<RULE>(m)) {
        const float s = scale_operand(byte);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = encode4_plain(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3], s);
    } else {
        const float f = mx_inv_scale_f32(byte);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = encode4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3], f);
    }
    const int64_t grow = r0 + 32 * b;
    if (c0 + c < climit && grow < rows) {
        uint4* q = reinterpret_cast<uint4*>(q_col + (oc0 + c) * rows + grow);
        q[0] = make_uint4(o[0], o[1], o[2], o[3]);
        q[1] = make_uint4(o[4], o[5], o[6], o[7]);
        s_col[(oc0 + c) * (rows / 32) + grow / 32] = (uint8_t)byte;
    }
}

template <int RULE>
__device__ __forceinline__ void ck_row_out(const float (&x)[4][8], int64_t r0, int64_t c0, int64_t climit, int64_t oc0,
                                           int64_t rows, int64_t ocols, uint8_t* __restrict__ q_row,
                                           uint8_t* __restrict__ s_row) {
    const int tid = threadIdx.x, ch = tid & 15, rr = tid >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t gr = r0 + rr + 16 * j;
        uint32_t byte;
        const uint2 v = encode_row8<RULE>(x[j], byte);
        if (c0 + 8 * ch < climit && gr < rows) {
            stnt8(q_row + gr * ocols + oc0 + 8 * ch, v);
            if ((ch & 3) == 0) s_row[gr * (ocols / 32) + (oc0 + 8 * ch) / 32] = (uint8_t)byte;
        }
    }
}

struct CkBwdArgs {
    const uint8_t *ck_q, *ck_s;
    const uint16_t* dh;
    int64_t rows, F;
    uint8_t *q_row, *s_row, *q_col, *s_col, *h_q, *h_s;
};

template <int RULE>
__global__ __launch_bounds__(256) void swiglu_ck_bwd_kernel(CkBwdArgs a) {
    __shared__ __attribute__((aligned(16))) float tile[CT_ROWS * CT_COLS];
    const int tid = threadIdx.x, ch = tid & 15, rr = tid >> 4;
    const int64_t r0 = (int64_t)blockIdx.y * CT_ROWS, c0 = (int64_t)blockIdx.x * CT_COLS;
    const int64_t gc = c0 + 8 * ch, F = a.F;
    float xg[4][8], xu[4][8], xh[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t gr = r0 + rr + 16 * j;
#pragma unroll
        for (int e = 0; e < 8; ++e) { xg[j][e] = 0.0f; xu[j][e] = 0.0f; xh[j][e] = 0.0f; }
        if (gc < F && gr < a.rows) {
            float g[8], u[8], d[8];
            dequant8(ldnt8(a.ck_q + gr * 2 * F + gc), e8m0_value(a.ck_s[gr * (F / 16) + gc / 32]), g);
            dequant8(ldnt8(a.ck_q + gr * 2 * F + F + gc), e8m0_value(a.ck_s[gr * (F / 16) + F / 32 + gc / 32]), u);
            unpack8(ldnt16(a.dh + gr * F + gc), d);
            // sigma = 1 / (1 + e^-g), silu = g / (1 + e^-g), silu' = sigma (1 + g (1 - sigma))
            float silu[8], sig[8];
            silu8(g, silu, sig);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xg[j][e] = (d[e] * u[e]) * (sig[e] * (1.0f + g[e] * (1.0f - sig[e])));
                xu[j][e] = d[e] * silu[e];
                xh[j][e] = silu[e] * u[e];
            }
        }
    }
    if (a.q_row) {
        ck_row_out<RULE>(xg, r0, c0, F, c0, a.rows, 2 * F, a.q_row, a.s_row);
        ck_row_out<RULE>(xu, r0, c0, F, F + c0, a.rows, 2 * F, a.q_row, a.s_row);
    }
    if (a.q_col) {
        ck_col_out<RULE>(xg, tile, r0, c0, F, c0, a.rows, a.q_col, a.s_col);
        ck_col_out<RULE>(xu, tile, r0, c0, F, F + c0, a.rows, a.q_col, a.s_col);
    }
    if (a.h_q) ck_col_out<RULE>(xh, tile, r0, c0, F, c0, a.rows, a.h_q, a.h_s);
}

// ---------------------------------------------------------------------------------------- launchers
hipError_t launch_swiglu_checkpoint(const uint16_t* c, int64_t rows, int64_t F, uint8_t* q, uint8_t* s, uint8_t* ck_q,
                                    uint8_t* ck_s, int rule, hipStream_t stream) {
    const dim3 grid((unsigned)((rows * (F / 8) + 255) / 256));
    if (rule == RULE_FLOOR)
        hipLaunchKernelGGL(swiglu_ck_fwd_kernel<RULE_FLOOR>, grid, dim3(256), 0, stream, c, rows, F, q, s, ck_q, ck_s);
    else
        hipLaunchKernelGGL(swiglu_ck_fwd_kernel<RULE_RCEIL>, grid, dim3(256), 0, stream, c, rows, F, q, s, ck_q, ck_s);
    return hipGetLastError();
}

hipError_t launch_swiglu_bwd_checkpoint(const uint8_t* ck_q, const uint8_t* ck_s, const uint16_t* dh, int64_t rows,
                                        int64_t F, uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                                        uint8_t* h_q, uint8_t* h_s, int rule, hipStream_t stream) {
    const CkBwdArgs a{ck_q, ck_s, dh, rows, F, q_row, s_row, q_col, s_col, h_q, h_s};
    const dim3 grid((unsigned)((F + CT_COLS - 1) / CT_COLS), (unsigned)((rows + CT_ROWS - 1) / CT_ROWS));
    if (rule == RULE_FLOOR) hipLaunchKernelGGL(swiglu_ck_bwd_kernel<RULE_FLOOR>, grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(swiglu_ck_bwd_kernel<RULE_RCEIL>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxq
