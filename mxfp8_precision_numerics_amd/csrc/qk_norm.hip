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
#include <type_traits>

#include "launch.h"
#include "mx_block.h"

namespace mxq {

// cos and sin of pos * w. The angle is formed in quarter turns in 64 bits with the products' own roundings kept, so what is
// left after the whole quarters is good to 2^-50 quarters for angles up to 2^50, as long as pos itself is a 64-bit floating-point
// number (|pos| <= 2^53).
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

// Sum over the P lanes of a head, by lane permutations within 16 lanes; every lane gets the same result.
template <int P>
__device__ __forceinline__ float head_sum(float v) {
    auto add = [&](auto ctrl) {
        v += __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    if constexpr (P > 1) add(std::integral_constant<int, 0xB1>{});       // lane ^ 1
    if constexpr (P > 2) add(std::integral_constant<int, 0x4E>{});       // lane ^ 2
    if constexpr (P > 4) add(std::integral_constant<int, 0x141>{});      // the other four of eight
    if constexpr (P > 8) add(std::integral_constant<int, 0x140>{});      // the other eight of sixteen
    return v;
}

__device__ __forceinline__ float sum_squares16(const float (&v)[16]) {
    float q[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] = v[e] * v[e];
    return tree_sum(q);
}

// A lane's two chunks as they lie in memory. Each value is used once: the loads and stores pass the caches by.
struct Raw {
    uint4 lo, hi;
};
__device__ __forceinline__ Raw load_raw(const uint16_t* lo, const uint16_t* hi, bool ok) {
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    return Raw{ok ? ldnt16(lo) : z, ok ? ldnt16(hi) : z};
}

// Value e (0 .. 15) of them.
__device__ __forceinline__ float value_of(const Raw& r, int e) {
    const uint4& q = e < 8 ? r.lo : r.hi;
    const uint32_t w = (e & 7) < 2 ? q.x : (e & 7) < 4 ? q.y : (e & 7) < 6 ? q.z : q.w;
    return (e & 1) ? bf16_hi(w) : bf16_lo(w);
}

__device__ __forceinline__ void unpack16(const Raw& r, float (&v)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = value_of(r, e);
}

__device__ __forceinline__ void store16(uint16_t* lo, uint16_t* hi, const float (&v)[16]) {
    float x[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = v[e];
        y[e] = v[8 + e];
    }
    stnt16(lo, pack8(x));
    stnt16(hi, pack8(y));
}

__device__ __forceinline__ void load_gamma16(const float* g, const Unit& un, float (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float4 w = un.on ? *reinterpret_cast<const float4*>(g + (h < 2 ? un.lo : un.hi) + 4 * (h & 1))
                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        v[4 * h] = w.x; v[4 * h + 1] = w.y; v[4 * h + 2] = w.z; v[4 * h + 3] = w.w;
    }
}

// A workgroup takes queries or keys; its waves' items are runs of blocks of 64 / P heads of one token, each wave every
// (4 groups)-th item of the kind.
struct Item {
    int64_t token;
    int first, last;            // blocks
};

__device__ __forceinline__ Item item_of(const QkKind& k, uint32_t i) {
    Item r;
    const uint32_t t = i / (uint32_t)k.splits;
    r.token = t;
    r.first = (int)(i - t * k.splits) * k.per_item;
    r.last = min(r.first + k.per_item, k.blocks);
    return r;
}

// Bound by memory, 4 bytes a value: 4096 tokens of 96 + 96 heads of 128 in 69.3 us, 5.8 TB/s. The next block's values are on
// their way while a block is at work.
template <int P, bool NORM>
__global__ __launch_bounds__(256) void qk_forward_kernel(QkArgs a) {
    __shared__ __attribute__((aligned(16))) float2 angles[4][8 * P];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    constexpr int HEADS = 64 / P;
    const Unit un = unit_of<P>(a, lane % P);
    const int kind = (int)blockIdx.x >= a.kind[0].groups;
    const QkKind k = a.kind[kind];
    const int group = (int)blockIdx.x - (kind ? a.kind[0].groups : 0), slot = lane / P;
    float gamma[16];
    if constexpr (NORM) load_gamma16(k.gamma, un, gamma);
    for (uint32_t at = 4 * group + wave; at < k.items; at += 4 * k.groups) {
        const Item it = item_of(k, at);
        const uint16_t* x = a.x + it.token * a.ldx + k.column + (int64_t)slot * a.dim;
        uint16_t* y = k.y + it.token * k.token + (int64_t)slot * k.head;
        auto load = [&](int b) {
            const uint16_t* p = x + (int64_t)b * HEADS * a.dim;
            return load_raw(p + un.lo, p + un.hi, un.on && b * HEADS + slot < k.heads && b < it.last);
        };
        Raw next = load(it.first);
        float c[8], s[8];
        token_angles<P>(a, it.token, lane, un, angles[wave], c, s);
        for (int b = it.first; b < it.last; ++b) {
            float v[16];
            unpack16(next, v);
            next = load(b + 1);
            if constexpr (NORM) {
                const float ss = head_sum<P>(sum_squares16(v));
                const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, a.inv_dim, a.eps));
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = (v[e] * rstd) * gamma[e];
            }
            turn(v, c, s, un, a.interleaved, 1.0f);
            if (un.on && b * HEADS + slot < k.heads) {
                uint16_t* p = y + (int64_t)b * HEADS * k.head;
                store16(p + un.lo, p + un.hi, v);
            }
        }
    }
}

// The gradients; with dgamma asked for (partial != NULL) every workgroup leaves one row of D sums. A wave's items follow
// from its place alone, so the sums are formed in a fixed order. Bound by memory, 6 bytes a value: 4096 tokens of 96 + 96 heads of 128
// in 113 us with the launch that joins the rows, 5.3 TB/s.
template <int P, bool NORM>
__global__ __launch_bounds__(256) void qk_backward_kernel(QkArgs a) {
    __shared__ __attribute__((aligned(16))) float2 angles[4][8 * P];
    __shared__ float sums[4][16 * P];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    constexpr int HEADS = 64 / P;
    const Unit un = unit_of<P>(a, lane % P);
    const int kind = (int)blockIdx.x >= a.kind[0].groups;
    const QkKind k = a.kind[kind];
    const int group = (int)blockIdx.x - (kind ? a.kind[0].groups : 0), slot = lane / P;
    float gamma[16], dg[16];
    if constexpr (NORM) load_gamma16(k.gamma, un, gamma);
#pragma unroll
    for (int e = 0; e < 16; ++e) dg[e] = 0.0f;
    for (uint32_t at = 4 * group + wave; at < k.items; at += 4 * k.groups) {
        const Item it = item_of(k, at);
        const uint16_t* dy = k.y + it.token * k.token + (int64_t)slot * k.head;
        const uint16_t* xs = a.x + it.token * a.ldx + k.column + (int64_t)slot * a.dim;
        uint16_t* dx = a.dx + it.token * a.lddx + k.column + (int64_t)slot * a.dim;
        auto there = [&](int b) { return un.on && b * HEADS + slot < k.heads && b < it.last; };
        auto load_dy = [&](int b) {
            const uint16_t* p = dy + (int64_t)b * HEADS * k.head;
            return load_raw(p + un.lo, p + un.hi, there(b));
        };
        auto load_x = [&](int b) {
            const uint16_t* p = xs + (int64_t)b * HEADS * a.dim;
            return load_raw(p + un.lo, p + un.hi, there(b));
        };
        Raw next_dy = load_dy(it.first), next_x;
        if constexpr (NORM) next_x = load_x(it.first);
        float c[8], s[8];
        token_angles<P>(a, it.token, lane, un, angles[wave], c, s);
        for (int b = it.first; b < it.last; ++b) {
            float d[16];
            unpack16(next_dy, d);
            next_dy = load_dy(b + 1);
            turn(d, c, s, un, a.interleaved, -1.0f);
            if constexpr (NORM) {
                // both sums over the head are of the values as they came: sum t xh = rstd sum t x
                const Raw now = next_x;
                next_x = load_x(b + 1);
                float sq[4] = {0.0f, 0.0f, 0.0f, 0.0f}, tx[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x = value_of(now, e);
                    sq[e & 3] = __builtin_fmaf(x, x, sq[e & 3]);
                    tx[e & 3] = __builtin_fmaf(d[e] * gamma[e], x, tx[e & 3]);
                }
                const float ss = head_sum<P>(tree_sum(sq)), st = head_sum<P>(tree_sum(tx));
                const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, a.inv_dim, a.eps)), mean = (st * a.inv_dim) * rstd;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float xh = value_of(now, e) * rstd;
                    dg[e] = __builtin_fmaf(d[e], xh, dg[e]);
                    d[e] = rstd * __builtin_fmaf(-xh, mean, d[e] * gamma[e]);
                }
            }
            if (there(b)) {
                uint16_t* p = dx + (int64_t)b * HEADS * a.dim;
                store16(p + un.lo, p + un.hi, d);
            }
        }
    }
    if constexpr (NORM) {
        if (a.partial == nullptr) return;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float v = dg[e];
#pragma unroll
            for (int o = P; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
            if (lane < P && un.on) sums[wave][(e < 8 ? un.lo : un.hi) + (e & 7)] = v;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.dim; i += 256)
            a.partial[(int64_t)blockIdx.x * a.dim + i] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
    }
}

// dgamma of queries (blockIdx.y = 0) or keys from the workgroups' rows: 64 threads a column take every 64th row in 64 bits, eight
// loads in flight, joined in a fixed order.
__global__ __launch_bounds__(1024) void qk_dgamma_kernel(const float* __restrict__ partial, int parts_q, int parts_k, int dim,
                                                        float* __restrict__ dq, float* __restrict__ dk, int accumulate) {
    __shared__ double s[64][17];
    const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
    const int first = blockIdx.y ? parts_q : 0, rows = blockIdx.y ? parts_k : parts_q;
    const float* p = partial + (int64_t)first * dim + blockIdx.x * 16 + c;
    double v = 0.0;
    for (int r = part; r < rows; r += 8 * 64) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = r + 64 * i < rows ? p[(int64_t)(r + 64 * i) * dim] : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += (double)x[i];
    }
    s[part][c] = v;
    __syncthreads();
    if (threadIdx.x < 16) {
        double total = 0.0;
#pragma unroll
        for (int i = 0; i < 64; i += 16) {
            double x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = s[i + j][c];
            total += tree_sum(x);
        }
        float* out = (blockIdx.y ? dk : dq) + blockIdx.x * 16 + c;
        *out = (float)(accumulate ? (double)*out + total : total);
    }
}

namespace {

int lanes_per_head(int64_t dim) { return dim <= 64 ? (dim <= 16 ? 1 : dim <= 32 ? 2 : 4) : dim <= 128 ? 8 : 16; }

// Items: a token's head blocks of a kind in runs of up to 4, shorter ones while there are few tokens; workgroups: one for four
// items, up to `most` of both kinds together, divided by their blocks. Measured at 4096 tokens of 96 + 96 heads of 128: the
// forward takes 69.3 us with runs of 4 and up to 4096 workgroups, 71 to 74 with runs of 2 or 3, 76 to 83 with runs of 6 or 12 or
// no more workgroups than the chip holds at once (each workgroup's own stretch of memory is then short and is read in order).
// The backward keeps sums in registers and leaves a row for every workgroup: two of them a CU, all it holds, 113 us; 768 134,
// 1024 117.
constexpr int64_t kRun = 4, kForwardGroups = 4096;

void split(QkArgs& a, int64_t most) {
    const int heads = 64 / lanes_per_head(a.dim);
    a.inv_dim = 1.0f / (float)a.dim;
    int64_t blocks = 0;
    for (QkKind& k : a.kind) {
        k.blocks = (k.heads + heads - 1) / heads;
        blocks += k.blocks;
    }
    for (QkKind& k : a.kind) {
        k.splits = k.per_item = 1;
        k.items = 0;
        k.groups = 0;
        if (a.tokens == 0 || k.blocks == 0) continue;
        int64_t per = a.tokens * blocks / 8192;
        per = per < 1 ? 1 : per > kRun ? kRun : per;
        k.splits = (int)((k.blocks + per - 1) / per);
        k.per_item = (k.blocks + k.splits - 1) / k.splits;
        k.items = (uint32_t)(a.tokens * k.splits);
        const int64_t want = ((int64_t)k.items + 3) / 4, share = most * k.blocks / blocks;
        k.groups = (int)(want < share ? want : share < 1 ? 1 : share);
    }
}

template <bool NORM>
void forward(const QkArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.kind[0].groups + a.kind[1].groups)), block(256);
    switch (lanes_per_head(a.dim)) {
        case 1: hipLaunchKernelGGL((qk_forward_kernel<1, NORM>), grid, block, 0, stream, a); break;
        case 2: hipLaunchKernelGGL((qk_forward_kernel<2, NORM>), grid, block, 0, stream, a); break;
        case 4: hipLaunchKernelGGL((qk_forward_kernel<4, NORM>), grid, block, 0, stream, a); break;
        case 8: hipLaunchKernelGGL((qk_forward_kernel<8, NORM>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((qk_forward_kernel<16, NORM>), grid, block, 0, stream, a); break;
    }
}

template <bool NORM>
void backward(const QkArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.kind[0].groups + a.kind[1].groups)), block(256);
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
    split(a, kForwardGroups);
    if (a.kind[0].gamma) forward<true>(a, stream);
    else forward<false>(a, stream);
    return hipGetLastError();
}

hipError_t launch_qk_backward(QkArgs a, float* dgamma_q, float* dgamma_k, int accumulate, hipStream_t stream) {
    split(a, kQkBwdParts);
    if (a.kind[0].groups + a.kind[1].groups > 0) {
        if (a.kind[0].gamma) backward<true>(a, stream);
        else backward<false>(a, stream);
    }
    if (dgamma_q)
        hipLaunchKernelGGL(qk_dgamma_kernel, dim3((unsigned)(a.dim / 16), 2), dim3(1024), 0, stream, a.partial,
                           a.kind[0].groups, a.kind[1].groups, a.dim, dgamma_q, dgamma_k, accumulate);
    return hipGetLastError();
}

}  // namespace mxq
