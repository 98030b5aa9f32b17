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
// 132160 x 1024: 170 us, 5.6 TB/s of 7.09 bytes a value of h. 52 vector instructions a value at four cycles each take
// about that time as well (the exponential is 21 of them, one rounding each), so memory and the vector units are both
// near their limits. Stores through the caches: 182 us against 175 a call.
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
// 132160 x 1024: 320 us, 3.9 TB/s of 9.22 bytes a value of h, 56% of it writes; 16384 x 8192 314 us. Nothing is saturated:
// vector issue 0.42 of the cycles, LDS a third, waves waiting 0.41 of theirs. Without the row outputs 60 us less, without the
// column codes 75 less, both at fewer bytes a second, without the table's reads no less: two workgroups a CU (80 KiB of LDS
// each) take turns between the phases behind their barriers. 8 bytes a lane spill. All codes go past the caches: through
// the L2 the column codes cost 25 us, the row codes between -35 and +30 with where the buffers lie in memory. Values kept in
// registers, their column maxima by lane permutations and only codes through LDS: half the LDS traffic, but 64-byte row
// pieces and no room for loads ahead: 370 us.
//
// silu and its derivative by table: g^ is one of 256 codes times its block's scale, so for the CT_SCALES scales of
// ordinary activations (blocks whose largest value lies between 0.007 and 448) a workgroup evaluates both once per code,
// 4096 pairs in 32 KiB of LDS, and reads them back in place of some 40 instructions a value. A wave that meets another
// scale (a block of zeros has one) evaluates its values directly, 384 us if all do; both ways give the same bits.
constexpr int CT_ROWS = 32, CT_COLS = 128, CT_THREADS = 512;
constexpr int CT_SCALES = 16, CT_SCALE0 = 112;
constexpr int64_t CT_GRID = 512;                               // two workgroups (2 x 80 KiB of LDS) per CU

struct CkBwdArgs {
    const uint8_t *ck_q, *ck_s;
    const uint16_t* dh;
    int64_t rows, F;
    uint8_t *q_row, *s_row, *q_col, *s_col, *h_q, *h_s;
    uint32_t col_tiles, subs;   // tiles across; row tiles a workgroup takes one after the other (4 or 1)
    uint32_t ids, share;        // column tiles x groups of `subs` row tiles; an XCD's share of them
};

__device__ __forceinline__ void put8(float* tile, int row, int ch, const float (&x)[8]) {
    float* d = &tile[row * CT_COLS + 8 * ch];
    *reinterpret_cast<float4*>(d) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(d + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// silu = g / (1 + e^-g) and silu' = sigma (1 + g (1 - sigma)), sigma = 1 / (1 + e^-g); one rounding per operation.
__device__ __forceinline__ void silu_and_slope8(const float (&g)[8], float (&silu)[8], float (&slope)[8]) {
    silu8(g, silu, slope);
#pragma unroll
    for (int e = 0; e < 8; ++e) slope[e] = slope[e] * (1.0f + g[e] * (1.0f - slope[e]));
}

// A thread's chunk of a tile, and the tile a workgroup is at. Offsets inside a group of row tiles fit 32 bits.
struct CkChunk {
    uint2 g, u;
    uint4 d;
    uint32_t gs, us;
};
struct CkTile {
    uint32_t id, sub, rows;     // group, row tile within the group, rows of the group
    int64_t r0, c0;             // first row and column of the group
};

__device__ __forceinline__ void ck_group(const CkBwdArgs& a, CkTile& t) {
    t.r0 = (int64_t)(t.id / a.col_tiles) * (a.subs * CT_ROWS);
    t.c0 = (int64_t)(t.id % a.col_tiles) * CT_COLS;
    t.sub = 0;
    t.rows = (uint32_t)(a.rows - t.r0 < a.subs * CT_ROWS ? a.rows - t.r0 : a.subs * CT_ROWS);
}

__device__ __forceinline__ CkChunk ck_load(const CkBwdArgs& a, const CkTile& t, uint32_t rr, uint32_t cc) {
    CkChunk k{make_uint2(0u, 0u), make_uint2(0u, 0u), make_uint4(0u, 0u, 0u, 0u), CT_SCALE0, 127u};
    const uint32_t row = t.sub * CT_ROWS + rr, F = (uint32_t)a.F;
    if (t.c0 + cc < F && row < t.rows) {                         // whole quads: F % 32 == 0
        const uint8_t* q = a.ck_q + (t.r0 * 2 * F + t.c0);
        const uint8_t* s = a.ck_s + (t.r0 * (F / 16) + t.c0 / 32);
        const uint32_t qo = row * 2 * F + cc, so = row * (F / 16) + cc / 32;
        k.g = ldnt8(q + qo);
        k.u = ldnt8(q + F + qo);
        k.d = ldnt16(a.dh + (t.r0 * F + t.c0) + (row * F + cc));
        k.gs = s[so];
        k.us = s[F / 32 + so];
    }
    return k;
}

template <int RULE>
__global__ __launch_bounds__(CT_THREADS, 4) void swiglu_ck_bwd_kernel(CkBwdArgs a) {
    __shared__ __attribute__((aligned(16))) float tile[3][CT_ROWS * CT_COLS];
    __shared__ __attribute__((aligned(16))) float2 table[CT_SCALES * 256];
    const int tid = threadIdx.x;
    const uint32_t cc = 8 * (tid & 15), rr = tid >> 4, F = (uint32_t)a.F;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform: the values below stay out of the lanes
    const int which = wave >> 1, c = tid & (CT_COLS - 1);        // column phase: 0 d_gate, 1 d_up, 2 h
    uint8_t* const qd = which == 2 ? a.h_q : which < 2 ? a.q_col : nullptr;
    uint8_t* const sd = which == 2 ? a.h_s : a.s_col;
    // Workgroups go to the 8 XCDs in turn: each XCD takes an eighth of the groups in order, so that the scale bytes of
    // neighbouring tiles, a few to a 128-byte line, meet in one L2.
    const uint32_t end = min(a.ids, (blockIdx.x % 8 + 1) * a.share);
    CkTile t;
    t.id = blockIdx.x % 8 * a.share + blockIdx.x / 8;
    CkChunk next{};
    if (t.id < end) {
        ck_group(a, t);
        next = ck_load(a, t, rr, cc);
    }
    {
        float g[8], silu[8], slope[8];                           // codes 8 (tid % 32) .. + 7 of scale tid / 32
        const uint32_t q = 0x03020100u + 0x08080808u * (tid & 31);
        dequant8(make_uint2(q, q + 0x04040404u), e8m0_value(CT_SCALE0 + (tid >> 5)), g);
        silu_and_slope8(g, silu, slope);
#pragma unroll
        for (int e = 0; e < 8; ++e) table[8 * tid + e] = make_float2(silu[e], slope[e]);
    }
    __syncthreads();
    uint4 held[4][2];                                            // this column's codes of the group's row tiles, and
    uint32_t bytes = 0;                                          // their scale bytes
#pragma unroll
    for (int i = 0; i < 4; ++i) held[i][0] = held[i][1] = make_uint4(0u, 0u, 0u, 0u);
    while (t.id < end) {
        const CkChunk k = next;
        const CkTile now = t;
        const bool last = (now.sub + 1) * CT_ROWS >= now.rows;   // the group's last row tile
        if (last) {
            t.id += gridDim.x / 8;
            if (t.id < end) ck_group(a, t);
        } else {
            ++t.sub;
        }
        if (t.id < end) next = ck_load(a, t, rr, cc);
        const uint32_t row = now.sub * CT_ROWS + rr;
        float silu[8], slope[8], x[8], v[8];
        if (__any(k.gs - CT_SCALE0 >= (uint32_t)CT_SCALES)) {
            dequant8(k.g, e8m0_value(k.gs), v);
            silu_and_slope8(v, silu, slope);
        } else {
            const float2* e0 = table + 256 * (k.gs - CT_SCALE0);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 w = e0[((e < 4 ? k.g.x : k.g.y) >> (8 * (e & 3))) & 255u];
                silu[e] = w.x;
                slope[e] = w.y;
            }
        }
        const bool row_ok = a.q_row && now.c0 + cc < F && row < now.rows;
        uint8_t* qr = a.q_row + (now.r0 * 2 * F + now.c0);
        uint8_t* sr = a.s_row + (now.r0 * (F / 16) + now.c0 / 32);
        const uint32_t qo = row * 2 * F + cc, so = row * (F / 16) + cc / 32;
        uint32_t byte;
        float d[8];
        dequant8(k.u, e8m0_value(k.us), v);
        unpack8(k.d, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = silu[e] * v[e];       // h
        put8(tile[2], rr, cc / 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = d[e] * silu[e];       // d_up
        put8(tile[1], rr, cc / 8, x);
        if (row_ok) {
            stnt8(qr + F + qo, encode_row8<RULE>(x, byte));
            if ((tid & 3) == 0) sr[F / 32 + so] = (uint8_t)byte;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (d[e] * v[e]) * slope[e];   // d_gate
        put8(tile[0], rr, cc / 8, x);
        if (row_ok) {
            stnt8(qr + qo, encode_row8<RULE>(x, byte));
            if ((tid & 3) == 0) sr[so] = (uint8_t)byte;
        }
        if (!a.q_col && !a.h_q) continue;
        __syncthreads();
        if (qd && now.c0 + c < F) {
            float y[32], top = 0.0f;
#pragma unroll
            for (int r = 0; r < 32; r += 2) {
                y[r] = tile[which][r * CT_COLS + c];
                y[r + 1] = tile[which][(r + 1) * CT_COLS + c];
                top = amax3(top, y[r], y[r + 1]);
            }
            const uint32_t m = __float_as_uint(top) & 0x7FFFFFFFu;
            const uint32_t b = mx_scale_byte_f32(m, RULE);
            uint32_t o[8];
            if (block_is_plain<RULE>(m)) {
                const float s = scale_operand(b);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = encode4_plain(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3], s);
            } else {
                const float f = mx_inv_scale_f32(b);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = encode4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3], f);
            }
            const uint4 o0 = make_uint4(o[0], o[1], o[2], o[3]), o1 = make_uint4(o[4], o[5], o[6], o[7]);
            bytes = (now.sub ? bytes : 0u) | b << (8 * now.sub);
            if (now.sub == 0) { held[0][0] = o0; held[0][1] = o1; }
            if (now.sub == 1) { held[1][0] = o0; held[1][1] = o1; }
            if (now.sub == 2) { held[2][0] = o0; held[2][1] = o1; }
            if (now.sub == 3) { held[3][0] = o0; held[3][1] = o1; }
        }
        __syncthreads();
        if (!last) continue;
        // The group's codes: up to 128 bytes a column, one column per thread, through LDS (the tiles' memory) to 8 lanes
        // a column, so that memory gets whole 128-byte lines. Piece k of column c sits at k ^ (c % 8).
        uint4* stage = reinterpret_cast<uint4*>(&tile[0][0]);
        if (which < 3) {
#pragma unroll
            for (int i = 0; i < 8; ++i) stage[8 * tid + (i ^ (c & 7))] = held[i >> 1][i & 1];
        }
        if (qd && now.c0 + c < F) {
            uint8_t* s = sd + (now.c0 + c + (which == 1 ? F : 0)) * (a.rows / 32) + now.r0 / 32;
            if (now.rows == 128 && a.rows % 128 == 0) {
                *reinterpret_cast<uint32_t*>(s) = bytes;
            } else {
                for (uint32_t i = 0; i <= now.sub; ++i) s[i] = (uint8_t)(bytes >> (8 * i));
            }
        }
        __syncthreads();
        const uint32_t piece = tid & 7;
        if (16 * piece < now.rows) {                             // rows % 32 == 0
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                const uint32_t at = 64 * i + (tid >> 3);         // 0 .. 383: output at / 128, column at % 128
                const int out = (64 * i + 8 * wave) >> 7;
                uint8_t* q = out == 2 ? a.h_q : a.q_col;
                if (q && now.c0 + (at & 127) < F)
                    stnt16(q + (now.c0 + (at & 127) + (out == 1 ? F : 0)) * a.rows + now.r0 + 16 * piece,
                           stage[8 * at + (piece ^ (at & 7))]);
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
    const int64_t ids = col_tiles * ((row_tiles + subs - 1) / subs), share = (ids + 7) / 8;
    const CkBwdArgs a{ck_q, ck_s, dh, rows, F, q_row, s_row, q_col, s_col, h_q, h_s, (uint32_t)col_tiles,
                      (uint32_t)subs, (uint32_t)ids, (uint32_t)share};
    const dim3 grid((unsigned)(8 * (share < CT_GRID / 8 ? share : CT_GRID / 8)));
    if (rule == RULE_FLOOR) hipLaunchKernelGGL(swiglu_ck_bwd_kernel<RULE_FLOOR>, grid, dim3(CT_THREADS), 0, stream, a);
    else hipLaunchKernelGGL(swiglu_ck_bwd_kernel<RULE_RCEIL>, grid, dim3(CT_THREADS), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxq
