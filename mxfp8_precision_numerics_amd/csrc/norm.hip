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
    double inv_cols;            // 1 / cols
    uint16_t* sum;              // may be x or res: a lane writes the values it has read
    float* rstd;
    uint8_t *q_row, *s_row, *q_col, *s_col, *ck_q, *ck_s;
};

// gamma of chunk ch (zeros past the row).
__device__ __forceinline__ void load_gamma(const float* gamma, uint32_t ch, uint32_t chunks, float (&g)[8]) {
    float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v = u;
    if (ch < chunks) {
        u = *reinterpret_cast<const float4*>(gamma + 8 * ch);
        v = *reinterpret_cast<const float4*>(gamma + 8 * ch + 4);
    }
    g[0] = u.x; g[1] = u.y; g[2] = u.z; g[3] = u.w; g[4] = v.x; g[5] = v.y; g[6] = v.z; g[7] = v.w;
}

// A row's statistic. Squares of bf16 values are exact in fp32; 8 of them are added in pairs in fp32, which is what the
// kernels spend on it, and everything after that, a few operations a chunk and a row, runs in 64 bits: the chunks, lanes and
// waves, the mean, and 1 / sqrt from the hardware's approximation (24 bits) by one Newton step. So rstd is the exact value's
// rounding but for the 8-value sums (u = 2^-24 is half its last place): 0.49 u root mean square over 16384 x 2048 normal
// values, against 0.74 in fp32 throughout; codes near a rounding boundary follow the exact ones more often. With one
// fp32 accumulator a lane, the same number of additions as in pairs, rstd was 0.37 u too large on average and 13.7 u off on
// rows of many small values.
__device__ __forceinline__ float sum_squares8(const float (&v)[8]) {
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = v[e] * v[e];
    return tree_sum(s);
}

__device__ __forceinline__ float rstd_of(double ss, double inv_cols, float eps) {
    const double v = __builtin_fma(ss, inv_cols, (double)eps);   // eps > 0
    double y = __builtin_amdgcn_rsq(v);
    y = __builtin_fma(0.5 * y, __builtin_fma(-v * y, y, 1.0), y);
    return v == (double)__builtin_inff() ? 0.0f : (float)y;
}

// ---------------------------------------------------------------------------------------- forward, row form
// W waves per row, NCH chunks of 8 values per lane: chunk j of lane l of the row's waves is l + 64 W j, so a wave's
// loads are contiguous and a 32-value block is one quad of lanes. W < 4 packs 4 / W rows into a workgroup.
// Bound by memory: with the residual and the checkpoint 8.06 bytes a value, 16384 x 2048 in 48.5 us (5.6 TB/s), 4096 x 12288
// in 67.5 us (6.0 TB/s). The widths of a variant were chosen at its upper end.
template <int RULE, int W, int NCH>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void norm_row_kernel(NormArgs a) {
    constexpr int ROWS = W < 4 ? 4 / W : 1;              // rows per workgroup
    __shared__ double part[W > 1 ? ROWS * W : 1];
    const int t = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W);
    const int64_t row = (int64_t)blockIdx.x * ROWS + sub;
    const bool row_ok = row < a.rows;
    const int chunks = (int)(a.cols / 8);
    uint4 h[NCH];
    double sq[NCH];
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
        sq[j] = sum_squares8(v);
    }
    double ss = wave_sum(tree_sum(sq));
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
        __syncthreads();
        double p[W];
#pragma unroll
        for (int w = 0; w < W; ++w) p[w] = part[sub * W + w];
        ss = tree_sum(p);
    }
    const float rstd = rstd_of(ss, a.inv_cols, a.eps);
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

// A column pair of 32 rows of h (d[r], low half the first column), rstd rs[r], gammas g0 and g1 -> 32 codes and a scale
// byte each. y is formed twice (for the block maximum, then for the codes) rather than kept in 64 registers.
template <int RULE>
__device__ __forceinline__ void encode_pair(const uint32_t (&d)[32], const float* rs, float g0, float g1, uint4 (&c0)[2],
                                            uint4 (&c1)[2], uint32_t& b0, uint32_t& b1) {
    float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; r += 2) {
        const float2 k = *reinterpret_cast<const float2*>(rs + r);
        t0 = amax3(t0, (bf16_lo(d[r]) * k.x) * g0, (bf16_lo(d[r + 1]) * k.y) * g0);
        t1 = amax3(t1, (bf16_hi(d[r]) * k.x) * g1, (bf16_hi(d[r + 1]) * k.y) * g1);
    }
    const uint32_t m0 = __float_as_uint(t0) & 0x7FFFFFFFu, m1 = __float_as_uint(t1) & 0x7FFFFFFFu;
    b0 = mx_scale_byte_f32(m0, RULE);
    b1 = mx_scale_byte_f32(m1, RULE);
    const bool plain = block_is_plain<RULE>(m0) && block_is_plain<RULE>(m1);
    const float s0 = plain ? scale_operand(b0) : mx_inv_scale_f32(b0), s1 = plain ? scale_operand(b1) : mx_inv_scale_f32(b1);
    uint32_t o0[8], o1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 k = *reinterpret_cast<const float4*>(rs + 4 * i);
        const uint32_t* q = d + 4 * i;
        const float y0 = (bf16_lo(q[0]) * k.x) * g0, y1 = (bf16_lo(q[1]) * k.y) * g0, y2 = (bf16_lo(q[2]) * k.z) * g0,
                    y3 = (bf16_lo(q[3]) * k.w) * g0;
        const float z0 = (bf16_hi(q[0]) * k.x) * g1, z1 = (bf16_hi(q[1]) * k.y) * g1, z2 = (bf16_hi(q[2]) * k.z) * g1,
                    z3 = (bf16_hi(q[3]) * k.w) * g1;
        o0[i] = plain ? encode4_plain(y0, y1, y2, y3, s0) : encode4(y0, y1, y2, y3, s0);
        o1[i] = plain ? encode4_plain(z0, z1, z2, z3, s1) : encode4(z0, z1, z2, z3, s1);
    }
    c0[0] = make_uint4(o0[0], o0[1], o0[2], o0[3]);
    c0[1] = make_uint4(o0[4], o0[5], o0[6], o0[7]);
    c1[0] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
    c1[1] = make_uint4(o1[4], o1[5], o1[6], o1[7]);
}

// ---------------------------------------------------------------------------------------- forward, column form
// A 128 x 128 tile of h per 256-thread workgroup, through LDS: thread (p, b) reads the column pair 2p, 2p + 1 of rows
// 32 b .. 32 b + 31 and forms y twice (for the block maximum, then for the codes) rather than keep 64 fp32 values.
// The codes pass through LDS once more so that each column's 128 codes leave as 16-byte pieces of whole lines.
// The codes, whole lines, go past the caches (through them 22.8 and 32.0 us for the two sizes here).
// 3.03 bytes a value: 16384 x 2048 21.7 us (4.7 TB/s; part of h is still in the last-level cache), 4096 x 12288 30.5 us
// (5.0 TB/s). The row form's pass leaves h in bf16, so this reads 2 bytes a value where keeping y would cost 4.
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
        if (gc < cols && r0 + lr < rows) v = ldnt16(h + (r0 + lr) * cols + gc);
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
#pragma unroll
    for (int r = 0; r < 32; ++r) d[r] = lds[(32 * b + r) * (NT / 2) + p];
    uint4 c0v[2], c1v[2];
    uint32_t b0, b1;
    encode_pair<RULE>(d, rs + 32 * b, g0, g1, c0v, c1v, b0, b1);
    __syncthreads();                                             // every column pair has been read
    uint8_t* ob = reinterpret_cast<uint8_t*>(lds);               // 128 x 128 codes, then 128 x 4 scale bytes
    const int ce = 2 * p, co = 2 * p + 1, sw = p & 7;            // 16-byte piece k of column c sits at k ^ (c/2 % 8)
    uint4* e = reinterpret_cast<uint4*>(ob + ce * NT);
    uint4* o = reinterpret_cast<uint4*>(ob + co * NT);
    e[(2 * b) ^ sw] = c0v[0];
    e[(2 * b + 1) ^ sw] = c0v[1];
    o[(2 * b) ^ sw] = c1v[0];
    o[(2 * b + 1) ^ sw] = c1v[1];
    ob[NT * NT + 4 * ce + b] = (uint8_t)b0;
    ob[NT * NT + 4 * co + b] = (uint8_t)b1;
    __syncthreads();
    const int k = tid & 7;
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        const int c = 32 * pass + (tid >> 3);
        if (c0 + c < cols && r0 + 16 * k < rows)                 // rows % 32 == 0: a 16-row piece is whole
            stnt16(q_col + (c0 + c) * rows + r0 + 16 * k,
                   *reinterpret_cast<const uint4*>(ob + c * NT + 16 * (k ^ ((c >> 1) & 7))));
    }
    if (tid < NT && c0 + tid < cols) {
        uint8_t* dst = s_col + (c0 + tid) * (rows / 32) + r0 / 32;
        for (int q = 0; q < 4 && r0 + 32 * q < rows; ++q) dst[q] = ob[NT * NT + 4 * tid + q];
    }
}

// ---------------------------------------------------------------------------------------- forward, both forms
// Up to 1024 columns, 32 rows of h take at most 64 KiB of LDS, two workgroups fit on a CU, and one workgroup reads its 32
// rows once and writes everything: its waves take a row each in turn as norm_row_kernel does, and after one barrier each
// thread encodes a column pair of the 32 rows. The four workgroups whose 32 codes share a 128-byte line of q_col run on
// the same XCD (8 apart in launch order), whose L2 completes the line. 65536 x 512: 64 us against 67 in two passes,
// 16384 x 1024: 35 against 38. With 2048 columns (128 KiB, one workgroup a CU) it was no faster (75 against 73 us).
template <int RULE, int NCH, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_rows32_kernel(NormArgs a) {
    constexpr int COLS = 512 * NCH, WAVES = THREADS / 64, PER = 32 / WAVES;
    __shared__ __attribute__((aligned(16))) uint32_t lds[32 * COLS / 2];
    __shared__ __attribute__((aligned(16))) float rs[32];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const uint32_t id = blockIdx.x;
    const int64_t r0 = 32 * (4 * (int64_t)(8 * (id / 32) + id % 8) + (id / 8) % 4);
    if (r0 >= a.rows) return;                                    // the grid is rounded up to whole groups of 32
    const uint32_t cols = (uint32_t)a.cols, chunks = cols / 8;
    uint4 h[PER][NCH], res[PER][NCH];
#pragma unroll
    for (int q = 0; q < PER; ++q)
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const uint32_t ch = lane + 64 * j;
            const int64_t at = (r0 + w + WAVES * q) * cols + 8 * ch;
            h[q][j] = res[q][j] = make_uint4(0u, 0u, 0u, 0u);
            if (ch < chunks) {
                h[q][j] = ldnt16(a.x + at);
                if (a.res) res[q][j] = ldnt16(a.res + at);
            }
        }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int lr = w + WAVES * q;
        const int64_t row = r0 + lr;
        double sq[NCH];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const uint32_t ch = lane + 64 * j;
            float v[8];
            unpack8(h[q][j], v);
            if (a.res) {
                float r[8];
                unpack8(res[q][j], r);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] + r[e];
                h[q][j] = pack8(v);
                unpack8(h[q][j], v);
                if (ch < chunks) stnt16(a.sum + row * cols + 8 * ch, h[q][j]);
            }
            sq[j] = sum_squares8(v);
            if (ch < chunks) *reinterpret_cast<uint4*>(&lds[lr * (COLS / 2) + 4 * ch]) = h[q][j];
        }
        const float rstd = rstd_of(wave_sum(tree_sum(sq)), a.inv_cols, a.eps);
        if (lane == 0) {
            a.rstd[row] = rstd;
            rs[lr] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const uint32_t ch = lane + 64 * j;
            if (ch >= chunks) continue;                          // whole quads: cols is a multiple of 32
            const int64_t at = row * cols + 8 * ch, sat = row * (cols / 32) + ch / 4;
            uint32_t byte;
            if (a.ck_q) {
                stnt8(a.ck_q + at, encode_row8_bf16<RULE>(h[q][j], byte));
                if ((ch & 3) == 0) a.ck_s[sat] = (uint8_t)byte;
            }
            if (a.q_row) {
                float g[8], y[8];
                load_gamma(a.gamma, ch, chunks, g);
                unpack8(h[q][j], y);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = (y[e] * rstd) * g[e];
                stnt8(a.q_row + at, encode_row8<RULE>(y, byte));
                if ((ch & 3) == 0) a.s_row[sat] = (uint8_t)byte;
            }
        }
    }
    __syncthreads();
    for (uint32_t p = tid; p < cols / 2; p += THREADS) {
        const float2 g = *reinterpret_cast<const float2*>(a.gamma + 2 * p);
        uint32_t d[32];
        uint4 c0[2], c1[2];
        uint32_t b0, b1;
#pragma unroll
        for (int r = 0; r < 32; ++r) d[r] = lds[r * (COLS / 2) + p];
        encode_pair<RULE>(d, rs, g.x, g.y, c0, c1, b0, b1);
        uint4* q = reinterpret_cast<uint4*>(a.q_col + 2 * (int64_t)p * a.rows + r0);
        q[0] = c0[0];
        q[1] = c0[1];
        q = reinterpret_cast<uint4*>(a.q_col + (2 * (int64_t)p + 1) * a.rows + r0);
        q[0] = c1[0];
        q[1] = c1[1];
        uint8_t* sc = a.s_col + 2 * (int64_t)p * (a.rows / 32) + r0 / 32;
        sc[0] = (uint8_t)b0;
        sc[a.rows / 32] = (uint8_t)b1;
    }
}

// ---------------------------------------------------------------------------------------- backward
// W waves share a row as in the forward; W < 8 packs R = 8 / W rows into a workgroup. A workgroup walks its rows in steps
// of the whole grid. The next rows' loads are issued before these are reduced; xh is formed twice from the codes (for the
// sums, then for dx) rather than kept. Each lane keeps gamma and its columns' dgamma sums in registers over all its rows;
// the workgroup writes one partial row of dgamma at the end, and norm_dgamma_kernel adds the partial rows in a fixed
// order, so the result does not depend on timing. Rows too wide for that in the registers of 16 waves (two chunks a lane) read
// gamma again for each row and load nothing ahead; beyond 16384 columns (four chunks) the dgamma sums and the row exceed
// the registers all the same and 120 bytes a lane spill: 4096 x 32768 317 us (3.0 TB/s), 4096 x 16384 100 us (4.7).
// Bound by memory: 4096 x 12288 with the residual's gradient 67.0 us (5.3 TB/s of 7.03 bytes a value); with dgamma's
// second launch, 4.7 us, it is the two launches that a call of 333 x 1056 consists of (3.6 and 4.1 us).
template <int NCH>
struct BwdRow {
    uint4 dy[NCH], dr[NCH];
    uint2 q[NCH];
    uint32_t s[NCH];
    float rstd;
};

struct BwdArgs {
    const uint16_t *dy, *dres;
    const uint8_t *ck_q, *ck_s;
    const float *rstd, *gamma;
    int64_t rows;
    uint32_t cols;
    uint16_t* dx;
    float* partial;             // NULL: no dgamma
};

template <int W, int NCH, bool RES>
__device__ __forceinline__ void load_row(BwdRow<NCH>& x, const BwdArgs& a, int64_t row, uint32_t t) {
    const uint32_t cols = a.cols;
    const bool row_ok = row < a.rows;
    const uint16_t* p = a.dy + row * cols;
    const uint16_t* d = a.dres + row * cols;
    const uint8_t* q = a.ck_q + row * cols;
    const uint8_t* s = a.ck_s + row * (cols / 32);
    x.rstd = row_ok ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const uint32_t ch = t + 64 * W * j;
        x.dy[j] = x.dr[j] = make_uint4(0u, 0u, 0u, 0u);
        x.q[j] = make_uint2(0u, 0u);
        x.s[j] = 127u;
        if (row_ok && ch < cols / 8) {
            x.dy[j] = ldnt16(p + 8 * ch);
            x.q[j] = ldnt8(q + 8 * ch);
            x.s[j] = s[ch / 4];
            if constexpr (RES) x.dr[j] = ldnt16(d + 8 * ch);
        }
    }
}

template <int W, int NCH, bool RES>
__global__ __launch_bounds__(W < 8 ? 512 : 64 * W) void norm_bwd_kernel(BwdArgs a) {
    constexpr int R = W < 8 ? 8 / W : 1;
    constexpr bool AHEAD = W < 16 || NCH == 1;
    static_assert(R == 1 || NCH == 1, "rows that share a workgroup have one chunk a lane");
    __shared__ float part[2][R * W];
    __shared__ __attribute__((aligned(16))) float comb[R > 1 ? 512 * 8 : 4];
    const uint32_t t = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W), cols = a.cols, chunks = cols / 8;
    const int64_t step = (int64_t)gridDim.x * R;
    float g[NCH][8], acc[NCH][8];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        if constexpr (AHEAD) load_gamma(a.gamma, t + 64 * W * j, chunks, g[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[j][e] = 0.0f;
    }
    BwdRow<NCH> next;
    int64_t base = (int64_t)blockIdx.x * R;
    if constexpr (AHEAD) load_row<W, NCH, RES>(next, a, base + sub, t);
    int par = 0;
    for (; base < a.rows; base += step, par ^= 1) {
        const int64_t row = base + sub;
        BwdRow<NCH> x;
        if constexpr (AHEAD) {
            x = next;
            load_row<W, NCH, RES>(next, a, row + step, t);
        } else {
            load_row<W, NCH, RES>(x, a, row, t);
        }
        const float rs = x.rstd;
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            float v[8], xh[8];
            if constexpr (!AHEAD) load_gamma(a.gamma, t + 64 * W * j, chunks, g[j]);
            unpack8(x.dy[j], v);
            dequant8(x.q[j], e8m0_value(x.s[j]), xh);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[e] = xh[e] * rs;
                acc[j][e] += v[e] * xh[e];
                dot += (v[e] * g[j][e]) * xh[e];
            }
        }
        dot = wave_sum(dot);
        if constexpr (W > 1) {
            if ((threadIdx.x & 63) == 0) part[par][threadIdx.x >> 6] = dot;      // two buffers: one barrier a row
            __syncthreads();
            dot = part[par][sub * W];
#pragma unroll
            for (int w = 1; w < W; ++w) dot += part[par][sub * W + w];
        }
        const float m = dot / (float)cols;
        uint16_t* o = a.dx + row * cols;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const uint32_t ch = t + 64 * W * j;
            if (!(row < a.rows && ch < chunks)) continue;
            float v[8], xh[8];
            if constexpr (!AHEAD) load_gamma(a.gamma, ch, chunks, g[j]);
            unpack8(x.dy[j], v);
            dequant8(x.q[j], e8m0_value(x.s[j]), xh);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = rs * (v[e] * g[j][e] - (xh[e] * rs) * m);
            if constexpr (RES) {
                float r[8];
                unpack8(x.dr[j], r);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = r[e] + v[e];
            }
            stnt16(o + 8 * ch, pack8(v));
        }
    }
    if (!a.partial) return;
    if constexpr (R > 1) {                                       // the rows' sums, added in order
        float* c = comb + 8 * threadIdx.x;
        *reinterpret_cast<float4*>(c) = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
        *reinterpret_cast<float4*>(c + 4) = make_float4(acc[0][4], acc[0][5], acc[0][6], acc[0][7]);
        __syncthreads();
        if (sub != 0) return;
#pragma unroll
        for (int q = 1; q < R; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[0][e] += comb[8 * (t + 64 * W * q) + e];
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const uint32_t ch = t + 64 * W * j;
        if (ch >= chunks) continue;
        float* o = a.partial + (int64_t)blockIdx.x * cols + 8 * ch;
        *reinterpret_cast<float4*>(o) = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        *reinterpret_cast<float4*>(o + 4) = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
}

// dgamma[c] = (accumulate ? dgamma[c] : 0) + sum of the partial rows. A workgroup has 32 columns, 4 to a lane, and 32
// slices of the rows: slice k adds rows k, k + 32, ..., eight loads in flight, and the slices are added in order.
__global__ __launch_bounds__(256) void norm_dgamma_kernel(const float* partial, int parts, int64_t cols, float* dgamma,
                                                         int accumulate) {
    __shared__ __attribute__((aligned(16))) float s[32][32];
    const int c = 4 * (threadIdx.x & 7), k = threadIdx.x >> 3;
    const float* p = partial + (int64_t)blockIdx.x * 32 + c;     // cols % 32 == 0
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int r = k; r < parts; r += 32) {
        const float4 x = *reinterpret_cast<const float4*>(p + (int64_t)r * cols);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    *reinterpret_cast<float4*>(&s[k][c]) = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        float y = s[0][threadIdx.x];
#pragma unroll
        for (int q = 1; q < 32; ++q) y += s[q][threadIdx.x];
        float* d = dgamma + (int64_t)blockIdx.x * 32 + threadIdx.x;
        *d = accumulate ? *d + y : y;
    }
}

// ---------------------------------------------------------------------------------------- launchers
template <int RULE, int W, int NCH>
static void run_row(const NormArgs& a, hipStream_t stream) {
    constexpr int ROWS = W < 4 ? 4 / W : 1;
    hipLaunchKernelGGL((norm_row_kernel<RULE, W, NCH>), dim3((unsigned)((a.rows + ROWS - 1) / ROWS)),
                       dim3(W < 4 ? 256 : 64 * W), 0, stream, a);
}

template <int RULE, int NCH, int THREADS>
static void run_rows32(const NormArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((norm_rows32_kernel<RULE, NCH, THREADS>), dim3((unsigned)((a.rows / 32 + 31) / 32 * 32)), dim3(THREADS),
                       0, stream, a);
}

// The row form's threads a row, by run_norm's widths.
int64_t norm_max_rows(int64_t cols) {
    return kMaxThreads / (cols <= 2048 ? 64 : cols <= 8192 ? 256 : cols <= 12288 ? 512 : 1024);
}

template <int RULE>
static void run_norm(const NormArgs& a, hipStream_t stream) {
    if (a.q_col && a.cols <= 1024) {
        if (a.cols <= 512) run_rows32<RULE, 1, 512>(a, stream);
        else run_rows32<RULE, 2, 512>(a, stream);
        return;
    }
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
    const NormArgs a{x, res, gamma, rows, cols, eps, 1.0 / (double)cols, sum, rstd, q_row, s_row, q_col, s_col, ck_q, ck_s};
    if (rule == RULE_FLOOR) run_norm<RULE_FLOOR>(a, stream);
    else run_norm<RULE_RCEIL>(a, stream);
    return hipGetLastError();
}

// Workgroups: two to a CU while their registers allow it (W < 12), else one.
template <int W, int NCH>
static int run_bwd(const BwdArgs& a, hipStream_t stream) {
    constexpr int R = W < 8 ? 8 / W : 1;
    constexpr int64_t MOST = W < 12 ? kNormBwdParts : kNormBwdParts / 2;
    const int64_t groups = (a.rows + R - 1) / R;
    const int parts = (int)(groups < MOST ? groups : MOST);
    if (a.dres) hipLaunchKernelGGL((norm_bwd_kernel<W, NCH, true>), dim3(parts), dim3(64 * W * R), 0, stream, a);
    else hipLaunchKernelGGL((norm_bwd_kernel<W, NCH, false>), dim3(parts), dim3(64 * W * R), 0, stream, a);
    return parts;
}

hipError_t launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* dres, const uint8_t* ck_q, const uint8_t* ck_s,
                                   const float* rstd, const float* gamma, int64_t rows, int64_t cols, uint16_t* dx,
                                   float* dgamma, int accumulate, float* partial, hipStream_t stream) {
    const BwdArgs a{dy, dres, ck_q, ck_s, rstd, gamma, rows, (uint32_t)cols, dx, dgamma ? partial : nullptr};
    int parts = 0;
    if (rows > 0) {
        if (cols <= 512) parts = run_bwd<1, 1>(a, stream);
        else if (cols <= 1024) parts = run_bwd<2, 1>(a, stream);
        else if (cols <= 2048) parts = run_bwd<4, 1>(a, stream);
        else if (cols <= 4096) parts = run_bwd<8, 1>(a, stream);
        else if (cols <= 8192) parts = run_bwd<16, 1>(a, stream);
        else if (cols <= 12288) parts = run_bwd<12, 2>(a, stream);
        else if (cols <= 16384) parts = run_bwd<16, 2>(a, stream);
        else parts = run_bwd<16, 4>(a, stream);
    }
    if (dgamma)
        hipLaunchKernelGGL(norm_dgamma_kernel, dim3((unsigned)(cols / 32)), dim3(256), 0, stream, partial, parts, cols,
                           dgamma, accumulate);
    return hipGetLastError();
}

}  // namespace mxq
