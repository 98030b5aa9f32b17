// RMSNorm of every query and key head with the rotation by position in the same pass, and its backward, for gfx950.
//
// Forward:   rstd = 1 / sqrt(sum_d x^2 / D + eps), n = (x rstd) gamma            (n = x without gammas)
//            pair (i, j) of a head's first `rot` values: y_i = n_i cos a - n_j sin a, y_j = n_j cos a + n_i sin a,
//            a = position[axis of the pair] * inv_freq[pair];  the other values: y = n
// Backward:  d = dy turned back by a, xh = x rstd, t = d gamma:  dx = rstd (t - xh (sum_d t xh) / D)   (dx = d without)
//            dgamma[d] = sum over tokens and heads of d xh
//
// A head of D values is held by D / 16 lanes, 16 values each: two 16-byte chunks chosen so that both values of each of the
// lane's 8 pairs are its own (halves apart: chunk u of the first and of the second half; neighbours: 16 consecutive
// values). Values past `rot` are pairs with angle 0. P = D / 16 rounded up to a power of two lanes, so the sums over a head
// are log2 P lane exchanges, and a wave takes 64 / P heads of one token at once. An angle depends on the token and the pair
// alone: a wave computes a token's angles once, one pair a lane, and keeps them for all of the token's heads it takes.
#pragma clang fp contract(off)
#include "launch.h"
#include "mx_block.h"

namespace mxq {

// cos and sin of pos * w. The angle is formed in quarter turns in 64 bits with the products' own roundings kept, so what is
// left after the whole quarters is good to 2^-50 quarters for angles up to 2^50: positions may lie as far as they like.
// |r| <= 1/2 quarter; then the Taylor polynomials of degree 9 and 10, whose remainders are below 2^-28.
__device__ __forceinline__ float2 cos_sin(int64_t pos, float freq) {
    const double p = (double)pos, w = (double)freq;
    constexpr double kQuarters = 0.63661977236758134308;            // 2 / pi, and what its rounding left
    constexpr double kQuartersLow = -3.9357353350364971764e-17;
    const double a = p * w, a_low = __builtin_fma(p, w, -a);
    const double t = a * kQuarters;
    const double low = __builtin_fma(a, kQuarters, -t) + (a * kQuartersLow + a_low * kQuarters);
    double k = __builtin_rint(t);
    double r = (t - k) + low;
    const double k2 = __builtin_rint(r);                            // 0, or the low part's own whole quarters
    r = r - k2;
    k = k + k2;
    const int quarter = (int)(k - 4.0 * __builtin_floor(k * 0.25)) & 3;
    const float x = (float)(r * 1.57079632679489661923);
    const float z = x * x;
    float s = 1.0f / 362880.0f, c = -1.0f / 3628800.0f;
    s = __builtin_fmaf(s, z, -1.0f / 5040.0f);
    s = __builtin_fmaf(s, z, 1.0f / 120.0f);
    s = __builtin_fmaf(s, z, -1.0f / 6.0f);
    s = __builtin_fmaf(s * z, x, x);
    c = __builtin_fmaf(c, z, 1.0f / 40320.0f);
    c = __builtin_fmaf(c, z, -1.0f / 720.0f);
    c = __builtin_fmaf(c, z, 1.0f / 24.0f);
    c = __builtin_fmaf(c, z, -0.5f);
    c = __builtin_fmaf(c, z, 1.0f);
    const float cc = (quarter & 1) ? s : c, ss = (quarter & 1) ? c : s;
    return make_float2((quarter == 1 || quarter == 2) ? -cc : cc, quarter >= 2 ? -ss : ss);
}

// Where this lane's two chunks lie within a head, and its first pair.
struct Unit {
    bool on;                // the lane holds part of a head
    bool turns;             // its pairs turn
    int lo, hi;             // first value of either chunk
};

template <int P>
__device__ __forceinline__ Unit unit_of(const QkArgs& a, int u) {
    Unit r;
    r.on = u < a.dim / 16;
    r.turns = u < a.rot / 16;
    const bool halves = r.turns && !a.interleaved;
    r.lo = halves ? 8 * u : 16 * u;
    r.hi = halves ? a.rot / 2 + 8 * u : 16 * u + 8;
    return r;
}

// The token's cos and sin of this lane's 8 pairs (1 and 0 past rot), by way of the wave's own LDS words.
template <int P>
__device__ __forceinline__ void token_angles(const QkArgs& a, int64_t token, int lane, const Unit& un, float2* words,
                                             float (&c)[8], float (&s)[8]) {
    const int pairs = a.rot / 2;
    wave_lds_order();
#pragma unroll
    for (int base = 0; base < 8 * P; base += 64) {
        const int i = base + lane;
        if (i < pairs) {
            const int axis = (int)((a.axis[i >> 4] >> (2 * (i & 15))) & 3u);
            words[i] = cos_sin(a.positions[axis * a.tokens + token], a.inv_freq[i]);
        }
    }
    wave_lds_order();
    const int first = 8 * (lane % P);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 w = un.turns ? words[first + e] : make_float2(1.0f, 0.0f);
        c[e] = w.x;
        s[e] = w.y;
    }
}

// Turns the 8 pairs among a lane's 16 values, (e, 8 + e) where the halves are apart, neighbours otherwise; sign = 1
// forward, -1 back. Values past rot are left alone (an infinity among them is no business of its neighbour).
template <bool NEIGHBOURS>
__device__ __forceinline__ void turn_pairs(float (&v)[16], const float (&c)[8], const float (&s)[8], float sign) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = NEIGHBOURS ? 2 * e : e, j = NEIGHBOURS ? 2 * e + 1 : 8 + e;
        const float x = v[i], y = v[j], se = s[e] * sign;
        v[i] = __builtin_fmaf(x, c[e], -(y * se));
        v[j] = __builtin_fmaf(y, c[e], x * se);
    }
}

__device__ __forceinline__ void turn(float (&v)[16], const float (&c)[8], const float (&s)[8], const Unit& un,
                                     bool neighbours, float sign) {
    if (!un.turns) return;
    if (neighbours) turn_pairs<true>(v, c, s, sign);
    else turn_pairs<false>(v, c, s, sign);
}

// Sum over the P lanes of a head.
template <int P>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = 1; o < P; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

__device__ __forceinline__ float sum_squares16(const float (&v)[16]) {
    float q[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] = v[e] * v[e];
    return tree_sum(q);
}

__device__ __forceinline__ void load16(const uint16_t* lo, const uint16_t* hi, bool ok, float (&v)[16]) {
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const uint4 a = ok ? *reinterpret_cast<const uint4*>(lo) : z, b = ok ? *reinterpret_cast<const uint4*>(hi) : z;
    float x[8], y[8];
    unpack8(a, x);
    unpack8(b, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = x[e];
        v[8 + e] = y[e];
    }
}

__device__ __forceinline__ void store16(uint16_t* lo, uint16_t* hi, const float (&v)[16]) {
    float x[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = v[e];
        y[e] = v[8 + e];
    }
    *reinterpret_cast<uint4*>(lo) = pack8(x);
    *reinterpret_cast<uint4*>(hi) = pack8(y);
}

__device__ __forceinline__ void load_gamma16(const float* g, const Unit& un, float (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float4 w = un.on ? *reinterpret_cast<const float4*>(g + (h < 2 ? un.lo : un.hi) + 4 * (h & 1))
                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        v[4 * h] = w.x; v[4 * h + 1] = w.y; v[4 * h + 2] = w.z; v[4 * h + 3] = w.w;
    }
}

// A wave's work: blocks [first, last) of 64 / P heads of one token, the query blocks ahead of the key blocks.
struct Item {
    int64_t token;
    int first, last;
};

__device__ __forceinline__ Item item_of(const QkArgs& a, int64_t i) {
    Item r;
    r.token = i / a.splits;
    r.first = (int)(i - r.token * a.splits) * a.per_item;
    r.last = min(r.first + a.per_item, a.q_blocks + a.k_blocks);
    return r;
}

template <int P, bool NORM>
__global__ __launch_bounds__(256) void qk_forward_kernel(QkArgs a) {
    __shared__ __attribute__((aligned(16))) float2 angles[4][8 * P];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int HEADS = 64 / P;
    const Unit un = unit_of<P>(a, lane % P);
    const int64_t at = (int64_t)blockIdx.x * 4 + wave;
    if (at >= a.items) return;
    const Item it = item_of(a, at);
    float c[8], s[8];
    token_angles<P>(a, it.token, lane, un, angles[wave], c, s);
    float gamma[16];
    int loaded = -1;
    for (int b = it.first; b < it.last; ++b) {
        const bool is_k = b >= a.q_blocks;
        const int head = (is_k ? b - a.q_blocks : b) * HEADS + lane / P;
        const bool ok = un.on && head < (is_k ? a.hk : a.hq);
        if (NORM && loaded != (int)is_k) {
            load_gamma16(is_k ? a.gamma_k : a.gamma_q, un, gamma);
            loaded = is_k;
        }
        const uint16_t* x = a.x + it.token * a.ldx + (int64_t)((is_k ? a.hq : 0) + head) * a.dim;
        float v[16];
        load16(x + un.lo, x + un.hi, ok, v);
        if constexpr (NORM) {
            const float ss = head_sum<P>(sum_squares16(v));
            const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, a.inv_dim, a.eps));
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = (v[e] * rstd) * gamma[e];
        }
        turn(v, c, s, un, a.interleaved, 1.0f);
        if (ok) {
            uint16_t* y = is_k ? a.k + it.token * a.k_token + (int64_t)head * a.k_head
                               : a.q + it.token * a.q_token + (int64_t)head * a.q_head;
            store16(y + un.lo, y + un.hi, v);
        }
    }
}

// The gradients; with dgamma asked for (partial != NULL) every workgroup leaves one row of 2 D sums (queries, keys). A
// wave's items are every (4 gridDim)-th, so the sums are formed in a fixed order.
template <int P, bool NORM>
__global__ __launch_bounds__(256) void qk_backward_kernel(QkArgs a) {
    __shared__ __attribute__((aligned(16))) float2 angles[4][8 * P];
    __shared__ float sums[4][2][16 * P];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int HEADS = 64 / P;
    const Unit un = unit_of<P>(a, lane % P);
    float dg[2][16];
#pragma unroll
    for (int e = 0; e < 16; ++e) dg[0][e] = dg[1][e] = 0.0f;
    for (int64_t at = (int64_t)blockIdx.x * 4 + wave; at < a.items; at += 4 * (int64_t)gridDim.x) {
        const Item it = item_of(a, at);
        float c[8], s[8];
        token_angles<P>(a, it.token, lane, un, angles[wave], c, s);
        auto heads = [&](auto is_k_c, int first, int last) {
            constexpr bool is_k = decltype(is_k_c)::value;
            if (first >= last) return;
            float gamma[16];
            if constexpr (NORM) load_gamma16(is_k ? a.gamma_k : a.gamma_q, un, gamma);
            for (int b = first; b < last; ++b) {
                const int head = b * HEADS + lane / P;
                const bool ok = un.on && head < (is_k ? a.hk : a.hq);
                const uint16_t* dy = is_k ? a.k + it.token * a.k_token + (int64_t)head * a.k_head
                                          : a.q + it.token * a.q_token + (int64_t)head * a.q_head;
                const int64_t col = (int64_t)((is_k ? a.hq : 0) + head) * a.dim;
                float d[16];
                load16(dy + un.lo, dy + un.hi, ok, d);
                float x[16];
                if constexpr (NORM) load16(a.x + it.token * a.ldx + col + un.lo, a.x + it.token * a.ldx + col + un.hi, ok, x);
                turn(d, c, s, un, a.interleaved, -1.0f);
                if constexpr (NORM) {
                    const float ss = head_sum<P>(sum_squares16(x));
                    const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, a.inv_dim, a.eps));
                    float m[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        x[e] = x[e] * rstd;
                        dg[is_k][e] += d[e] * x[e];
                        d[e] = d[e] * gamma[e];
                        m[e] = d[e] * x[e];
                    }
                    const float mean = head_sum<P>(tree_sum(m)) * a.inv_dim;
#pragma unroll
                    for (int e = 0; e < 16; ++e) d[e] = rstd * (d[e] - x[e] * mean);
                }
                if (ok) {
                    uint16_t* dx = a.dx + it.token * a.lddx + col;
                    store16(dx + un.lo, dx + un.hi, d);
                }
            }
        };
        heads(std::false_type{}, it.first, min(it.last, a.q_blocks));
        heads(std::true_type{}, max(it.first, a.q_blocks) - a.q_blocks, it.last - a.q_blocks);
    }
    if constexpr (NORM) {
        if (a.partial == nullptr) return;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float v = dg[k][e];
#pragma unroll
                for (int o = P; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
                if (lane < P && un.on) sums[wave][k][(e < 8 ? un.lo : un.hi) + (e & 7)] = v;
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.dim; i += 256) {
            const int k = i >= a.dim, d = k ? i - a.dim : i;
            a.partial[(int64_t)blockIdx.x * 2 * a.dim + i] = (sums[0][k][d] + sums[1][k][d]) + (sums[2][k][d] + sums[3][k][d]);
        }
    }
}

// dgamma from the workgroups' rows: 16 threads a column take every sixteenth row in 64 bits, joined in a fixed order.
__global__ __launch_bounds__(256) void qk_dgamma_kernel(const float* __restrict__ partial, int parts, int dim,
                                                       float* __restrict__ dq, float* __restrict__ dk, int accumulate) {
    __shared__ double s[16][16];
    const int col = blockIdx.x * 16 + (threadIdx.x & 15), part = threadIdx.x >> 4;
    double v = 0.0;
    for (int p = part; p < parts; p += 16) v += (double)partial[(int64_t)p * 2 * dim + col];
    s[part][threadIdx.x & 15] = v;
    __syncthreads();
    if (part == 0) {
        double x[16];
#pragma unroll
        for (int p = 0; p < 16; ++p) x[p] = s[p][threadIdx.x];
        const double total = tree_sum(x);
        float* out = col < dim ? dq + col : dk + (col - dim);
        *out = (float)(accumulate ? (double)*out + total : total);
    }
}

namespace {

constexpr int64_t kWaves = 8192;          // a launch with fewer waves leaves the chip's memory queues empty

int lanes_per_head(int64_t dim) { return dim <= 64 ? (dim <= 16 ? 1 : dim <= 32 ? 2 : 4) : dim <= 128 ? 8 : 16; }

// Items: a token's head blocks in runs of per_item, as long as there are waves enough.
void split(QkArgs& a) {
    const int heads = 64 / lanes_per_head(a.dim);
    a.q_blocks = (a.hq + heads - 1) / heads;
    a.k_blocks = (a.hk + heads - 1) / heads;
    const int64_t blocks = a.q_blocks + a.k_blocks;
    a.inv_dim = 1.0f / (float)a.dim;
    if (a.tokens == 0 || blocks == 0) {
        a.splits = a.per_item = 1;
        a.items = 0;
        return;
    }
    int64_t per = a.tokens * blocks / kWaves;
    per = per < 1 ? 1 : per > blocks ? blocks : per;
    a.splits = (int)((blocks + per - 1) / per);
    a.per_item = (int)((blocks + a.splits - 1) / a.splits);
    a.items = a.tokens * a.splits;
}

template <bool NORM>
void forward(const QkArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.items + 3) / 4)), block(256);
    switch (lanes_per_head(a.dim)) {
        case 1: hipLaunchKernelGGL((qk_forward_kernel<1, NORM>), grid, block, 0, stream, a); break;
        case 2: hipLaunchKernelGGL((qk_forward_kernel<2, NORM>), grid, block, 0, stream, a); break;
        case 4: hipLaunchKernelGGL((qk_forward_kernel<4, NORM>), grid, block, 0, stream, a); break;
        case 8: hipLaunchKernelGGL((qk_forward_kernel<8, NORM>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((qk_forward_kernel<16, NORM>), grid, block, 0, stream, a); break;
    }
}

template <bool NORM>
void backward(const QkArgs& a, int64_t blocks, hipStream_t stream) {
    const dim3 grid((unsigned)blocks), block(256);
    switch (lanes_per_head(a.dim)) {
        case 1: hipLaunchKernelGGL((qk_backward_kernel<1, NORM>), grid, block, 0, stream, a); break;
        case 2: hipLaunchKernelGGL((qk_backward_kernel<2, NORM>), grid, block, 0, stream, a); break;
        case 4: hipLaunchKernelGGL((qk_backward_kernel<4, NORM>), grid, block, 0, stream, a); break;
        case 8: hipLaunchKernelGGL((qk_backward_kernel<8, NORM>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((qk_backward_kernel<16, NORM>), grid, block, 0, stream, a); break;
    }
}

}  // namespace

hipError_t launch_qk_forward(QkArgs a, hipStream_t stream) {
    split(a);
    if (a.gamma_q) forward<true>(a, stream);
    else forward<false>(a, stream);
    return hipGetLastError();
}

hipError_t launch_qk_backward(QkArgs a, float* dgamma_q, float* dgamma_k, int accumulate, hipStream_t stream) {
    split(a);
    int64_t blocks = (a.items + 3) / 4;
    if (blocks > kQkBwdParts) blocks = kQkBwdParts;
    if (blocks > 0) {
        if (a.gamma_q) backward<true>(a, blocks, stream);
        else backward<false>(a, blocks, stream);
    }
    if (dgamma_q)
        hipLaunchKernelGGL(qk_dgamma_kernel, dim3((unsigned)(2 * a.dim / 16)), dim3(256), 0, stream, a.partial, (int)blocks,
                           a.dim, dgamma_q, dgamma_k, accumulate);
    return hipGetLastError();
}

}  // namespace mxq
