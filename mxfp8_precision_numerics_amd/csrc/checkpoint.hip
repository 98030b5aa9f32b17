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
// A 512-thread workgroup walks 32 x 128 tiles, one 8-value chunk of g, u and dh per thread: row tid / 16, columns
// 8 (tid % 16) .. + 7. The row orientation leaves from registers. d_gate, d_up and h go to three fp32 LDS tiles
// (48 KiB), and after one barrier each of 3 x 128 threads encodes one column.
//
// silu and sigma by table: g^ is one of 256 codes times its block's scale, so for the CT_SCALES scales of ordinary
// activations (blocks whose largest value lies between 0.007 and 448) a workgroup evaluates both once per code, 4096
// pairs in 32 KiB of LDS, and reads them back in place of some 35 instructions a value. A wave that meets another scale
// evaluates its values directly; both ways give the same bits.
constexpr int CT_ROWS = 32, CT_COLS = 128, CT_THREADS = 512;
constexpr int CT_SCALES = 16, CT_SCALE0 = 112;
constexpr int64_t CT_GRID = 512;                               // two workgroups (2 x 80 KiB of LDS) per CU

struct CkBwdArgs {
    const uint8_t *ck_q, *ck_s;
    const uint16_t* dh;
    int64_t rows, F;
    uint8_t *q_row, *s_row, *q_col, *s_col, *h_q, *h_s;
    int col_tiles, subs;        // tiles across; row tiles a workgroup takes one after the other (4 or 1)
    int64_t ids;                // column tiles x groups of `subs` row tiles
};

__device__ __forceinline__ void put8(float* tile, int row, int ch, const float (&x)[8]) {
    float* d = &tile[row * CT_COLS + 8 * ch];
    *reinterpret_cast<float4*>(d) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(d + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

struct CkChunk {
    uint2 g, u;
    uint4 d;
    uint32_t gs, us;
};

__device__ __forceinline__ CkChunk ck_load(const CkBwdArgs& a, int64_t gr, int64_t gc) {
    CkChunk k{make_uint2(0u, 0u), make_uint2(0u, 0u), make_uint4(0u, 0u, 0u, 0u), 127u, 127u};
    if (gc < a.F && gr < a.rows) {                               // whole quads: F % 32 == 0
        const uint8_t* q = a.ck_q + gr * 2 * a.F + gc;
        const uint8_t* s = a.ck_s + gr * (a.F / 16) + gc / 32;
        k.g = ldnt8(q);
        k.u = ldnt8(q + a.F);
        k.d = ldnt16(a.dh + gr * a.F + gc);
        k.gs = s[0];
        k.us = s[a.F / 32];
    }
    return k;
}

template <int RULE>
__global__ __launch_bounds__(CT_THREADS, 4) void swiglu_ck_bwd_kernel(CkBwdArgs a) {
    __shared__ __attribute__((aligned(16))) float tile[3][CT_ROWS * CT_COLS];
    __shared__ __attribute__((aligned(16))) float2 table[CT_SCALES * 256];
    const int tid = threadIdx.x, ch = tid & 15, rr = tid >> 4;
    const int64_t F = a.F;
    int64_t id = blockIdx.x;
    int64_t c0 = id % a.col_tiles * CT_COLS, r0 = id / a.col_tiles * a.subs * CT_ROWS;
    int sub = 0;
    CkChunk next = ck_load(a, r0 + rr, c0 + 8 * ch);
    {
        float g[8], silu[8], sig[8];                             // codes 8 (tid % 32) .. + 7 of scale tid / 32
        const uint32_t q = 0x03020100u + 0x08080808u * (tid & 31);
        dequant8(make_uint2(q, q + 0x04040404u), e8m0_value(CT_SCALE0 + (tid >> 5)), g);
        silu8(g, silu, sig);
#pragma unroll
        for (int e = 0; e < 8; ++e) table[8 * tid + e] = make_float2(silu[e], sig[e]);
    }
    __syncthreads();
    uint4 held[3][2];                                            // this column's codes of the row tiles before, and
    uint32_t bytes = 0;                                          // their scale bytes
#pragma unroll
    for (int i = 0; i < 3; ++i) held[i][0] = held[i][1] = make_uint4(0u, 0u, 0u, 0u);
    while (id < a.ids) {
        const CkChunk k = next;
        const int64_t gr = r0 + rr, gc = c0 + 8 * ch, cr0 = r0, cc0 = c0;
        const int csub = sub;
        const bool ok = gc < F && gr < a.rows;
        r0 += CT_ROWS;
        if (++sub == a.subs || r0 >= a.rows) {                   // the next tile: below this one, or another group's
            sub = 0;
            id += gridDim.x;
            c0 = id % a.col_tiles * CT_COLS;
            r0 = id / a.col_tiles * a.subs * CT_ROWS;
        }
        if (id < a.ids) next = ck_load(a, r0 + rr, c0 + 8 * ch);
        {
            float g[8], u[8], d[8], silu[8], sig[8], xg[8], xu[8], xh[8];
            dequant8(k.g, e8m0_value(k.gs), g);
            dequant8(k.u, e8m0_value(k.us), u);
            unpack8(k.d, d);
            if (__any(k.gs - CT_SCALE0 >= (uint32_t)CT_SCALES)) {
                silu8(g, silu, sig);
            } else {
                const float2* t = table + 256 * (k.gs - CT_SCALE0);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 v = t[((e < 4 ? k.g.x : k.g.y) >> (8 * (e & 3))) & 255u];
                    silu[e] = v.x;
                    sig[e] = v.y;
                }
            }
            // silu = g / (1 + e^-g), sigma = 1 / (1 + e^-g), silu' = sigma (1 + g (1 - sigma))
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xg[e] = (d[e] * u[e]) * (sig[e] * (1.0f + g[e] * (1.0f - sig[e])));
                xu[e] = d[e] * silu[e];
                xh[e] = silu[e] * u[e];
            }
            if (a.q_row && ok) {
                uint32_t bg, bu;
                uint8_t* q = a.q_row + gr * 2 * F + gc;
                stnt8(q, encode_row8<RULE>(xg, bg));
                stnt8(q + F, encode_row8<RULE>(xu, bu));
                if ((ch & 3) == 0) {
                    uint8_t* s = a.s_row + gr * (F / 16) + gc / 32;
                    s[0] = (uint8_t)bg;
                    s[F / 32] = (uint8_t)bu;
                }
            }
            if (a.q_col || a.h_q) {
                put8(tile[0], rr, ch, xg);
                put8(tile[1], rr, ch, xu);
                put8(tile[2], rr, ch, xh);
            }
        }
        if (!a.q_col && !a.h_q) continue;
        __syncthreads();
        const int which = tid >> 7, c = tid & (CT_COLS - 1);     // 0: d_gate, 1: d_up, 2: h
        if (which < 3 && cc0 + c < F && (which < 2 ? a.q_col : a.h_q)) {
            float d[32], top = 0.0f;
#pragma unroll
            for (int r = 0; r < 32; r += 2) {
                d[r] = tile[which][r * CT_COLS + c];
                d[r + 1] = tile[which][(r + 1) * CT_COLS + c];
                top = amax3(top, d[r], d[r + 1]);
            }
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
            // Four row tiles make a 128-byte line of the column: it is written at once, from the registers, so that the
            // caches need not hold thousands of part-written lines.
            const uint4 o0 = make_uint4(o[0], o[1], o[2], o[3]), o1 = make_uint4(o[4], o[5], o[6], o[7]);
            bytes = (csub ? bytes : 0u) | byte << (8 * csub);
            if (csub == 0) { held[0][0] = o0; held[0][1] = o1; }
            if (csub == 1) { held[1][0] = o0; held[1][1] = o1; }
            if (csub == 2) { held[2][0] = o0; held[2][1] = o1; }
            if (sub == 0) {                                      // the group's last row tile
                const int64_t col = cc0 + c + (which == 1 ? F : 0), g0 = cr0 - csub * CT_ROWS;
                uint8_t* qd = a.q_col;
                uint8_t* sd = a.s_col;
                if (which == 2) { qd = a.h_q; sd = a.h_s; }
                uint4* q = reinterpret_cast<uint4*>(qd + col * a.rows + g0);          // rows % 32 == 0
                sd += col * (a.rows / 32) + g0 / CT_ROWS;
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (csub > i) {
                        q[2 * i] = held[i][0];
                        q[2 * i + 1] = held[i][1];
                    }
                q[2 * csub] = o0;
                q[2 * csub + 1] = o1;
                if (csub == 3 && a.rows % 128 == 0) {
                    *reinterpret_cast<uint32_t*>(sd) = bytes;
                } else {
                    for (int i = 0; i <= csub; ++i) sd[i] = (uint8_t)(bytes >> (8 * i));
                }
            }
        }
        __syncthreads();
    }
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
    const int64_t col_tiles = (F + CT_COLS - 1) / CT_COLS, row_tiles = (rows + CT_ROWS - 1) / CT_ROWS;
    // whole lines of the column orientation where that still fills the chip, else one row tile a workgroup
    const int64_t subs = col_tiles * ((row_tiles + 3) / 4) >= CT_GRID ? 4 : 1;
    const CkBwdArgs a{ck_q, ck_s, dh, rows, F, q_row, s_row, q_col, s_col, h_q, h_s, (int)col_tiles, (int)subs,
                      col_tiles * ((row_tiles + subs - 1) / subs)};
    const dim3 grid((unsigned)(a.ids < CT_GRID ? a.ids : CT_GRID));
    if (rule == RULE_FLOOR) hipLaunchKernelGGL(swiglu_ck_bwd_kernel<RULE_FLOOR>, grid, dim3(CT_THREADS), 0, stream, a);
    else hipLaunchKernelGGL(swiglu_ck_bwd_kernel<RULE_RCEIL>, grid, dim3(CT_THREADS), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxq
