// Device helpers shared by the block kernels (norm.hip, checkpoint.hip, moe_few.hip): 8 values of one row as packed
// bf16, fp32 or MXFP8, and the sums across a wave. Internal; not part of the C ABI.
#pragma once
#include <type_traits>

#include "mxq_device.h"

namespace mxq {

// fp32 value of an E8M0 byte: 2^(byte - 127); 0xFF (a block that held a NaN) gives NaN, so every value of that block
// reads back as NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    const uint32_t bits = byte == 0u ? 0x00400000u : byte << 23;
    return __uint_as_float(byte == 255u ? 0x7FC00000u : bits);
}

// 8 bf16 (one 16-byte chunk) -> fp32.
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
}

// 8 fp32 -> bf16, to nearest even (the hardware's packed conversion; a NaN stays a NaN).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, v2bf));
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// 8 E4M3 codes times their block's scale -> fp32 (exact: 4 significant bits times a power of two).
__device__ __forceinline__ void dequant8(uint2 q, float s, float (&x)[8]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true);
    const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
    x[0] = a.x * s; x[1] = a.y * s; x[2] = b.x * s; x[3] = b.y * s;
    x[4] = c.x * s; x[5] = c.y * s; x[6] = d.x * s; x[7] = d.y * s;
}

// 4 fp32 -> 4 E4M3 codes, f = 1 / scale (a power of two), saturating, NaN kept.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float f) {
    return cvt_f32_pair<FMT_E4M3, true>(
        cvt_f32_pair<FMT_E4M3, false>(0u, clamp_keep_nan(a * f, 448.0f), clamp_keep_nan(b * f, 448.0f)),
        clamp_keep_nan(c * f, 448.0f), clamp_keep_nan(d * f, 448.0f));
}

// The same by the scaled conversion (v_cvt_scalef32_pk_fp8_f32 divides by 2^E, E the exponent field of s): half an
// instruction a value where the clamped form takes five and a half. It does not saturate, so it serves blocks whose
// values are finite and at most 448 scales: see block_is_plain.
__device__ __forceinline__ uint32_t encode4_plain(float a, float b, float c, float d, float s) {
    v2s o = __builtin_bit_cast(v2s, __builtin_nondeterministic_value(0u));
    o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, a, b, s, false);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, c, d, s, true);
    return __builtin_bit_cast(uint32_t, o);
}

// The rceil rule's scale keeps every finite value of a block within 448 scales. Blocks at the ends of the exponent range
// (all zero, below 2^-119, holding an infinity or a NaN) take the clamped form.
template <int RULE>
__device__ __forceinline__ bool block_is_plain(uint32_t amax_bits) {
    return RULE == RULE_RCEIL && amax_bits - 0x04000000u < 0x7F800000u - 0x04000000u;
}

// Largest magnitude of two values and m; a NaN stays (v_maximum3_f32).
__device__ __forceinline__ float amax3(float m, float a, float b) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(a)), __builtin_fabsf(b));
}

__device__ __forceinline__ uint32_t amax8_f32(const float (&x)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) m = amax3(m, x[e], x[e + 1]);
    return __float_as_uint(m) & 0x7FFFFFFFu;
}

// The MXFP8 row form of this lane's 8 consecutive values, its 32-value block being the 4 lanes of its quad.
template <int RULE>
__device__ __forceinline__ uint2 encode_row8(const float (&x)[8], uint32_t& byte) {
    const uint32_t m = quad_max(amax8_f32(x));
    byte = mx_scale_byte_f32(m, RULE);
    if (block_is_plain<RULE>(m)) {
        const float s = scale_operand(byte);
        return make_uint2(encode4_plain(x[0], x[1], x[2], x[3], s), encode4_plain(x[4], x[5], x[6], x[7], s));
    }
    const float f = mx_inv_scale_f32(byte);
    return make_uint2(encode4(x[0], x[1], x[2], x[3], f), encode4(x[4], x[5], x[6], x[7], f));
}

// The same for 8 bf16 values.
template <int RULE>
__device__ __forceinline__ uint2 encode_row8_bf16(uint4 v, uint32_t& byte) {
    const uint32_t m = quad_max(amax_bits8(v));
    byte = mx_scale_byte(m, RULE);
    const float s = scale_operand(byte);
    uint32_t lo = cvt_mx_quad(v.x, v.y, s), hi = cvt_mx_quad(v.z, v.w, s);
    if (RULE == RULE_FLOOR || m >= 0x7F80u) {
        const uint32_t thr = mx_sat_threshold(byte);
        lo = mx_patch4(lo, v.x, v.y, thr);
        hi = mx_patch4(hi, v.z, v.w, thr);
    }
    return make_uint2(lo, hi);
}

// Orders what the lanes of a wave wrote to LDS before it and read after it, or the reverse. The hardware runs one wave's LDS
// accesses in order, so this costs no instruction; it keeps the compiler from moving an access across, which it may where
// it finds that no lane reads an address of its own.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// The sum of N values, added in pairs, the pairs in pairs: each term passes log2 N roundings instead of up to N.
template <class T, int N>
__device__ __forceinline__ T tree_sum(const T (&x)[N]) {
    if constexpr (N == 1) {
        return x[0];
    } else {
        T y[(N + 1) / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) y[i] = x[2 * i] + x[2 * i + 1];
        if constexpr (N % 2 == 1) y[N / 2] = x[N - 1];
        return tree_sum(y);
    }
}

// Joins a value over the 64 lanes of a wave by lane permutations within 16-lane rows and swaps of rows and halves (no
// LDS); every lane gets the same result, as each step joins the same two values on both sides.
template <class Op>
__device__ __forceinline__ float wave_join(float v, Op op) {
    auto dpp = [](float x, auto ctrl) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    v = op(v, dpp(v, std::integral_constant<int, 0xB1>{}));      // lanes i ^ 1
    v = op(v, dpp(v, std::integral_constant<int, 0x4E>{}));      // lanes i ^ 2
    v = op(v, dpp(v, std::integral_constant<int, 0x141>{}));     // the other quad of 8 (row_half_mirror)
    v = op(v, dpp(v, std::integral_constant<int, 0x140>{}));     // the other 8 of 16 (row_mirror)
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float((uint32_t)r[0]), __uint_as_float((uint32_t)r[1]));
    const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float((uint32_t)h[0]), __uint_as_float((uint32_t)h[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
    return wave_join(v, [](float a, float b) { return a + b; });
}
// The same sum in 64 bits, the two words of a value moved alike.
__device__ __forceinline__ double wave_sum(double v) {
    auto join = [](uint2 a, uint2 b) {
        return __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b);
    };
    auto dpp = [&](double x, auto ctrl) {
        const uint2 w = __builtin_bit_cast(uint2, x);
        return join(w, make_uint2((uint32_t)__builtin_amdgcn_mov_dpp((int)w.x, decltype(ctrl)::value, 0xF, 0xF, false),
                                  (uint32_t)__builtin_amdgcn_mov_dpp((int)w.y, decltype(ctrl)::value, 0xF, 0xF, false)));
    };
    v = dpp(v, std::integral_constant<int, 0xB1>{});
    v = dpp(v, std::integral_constant<int, 0x4E>{});
    v = dpp(v, std::integral_constant<int, 0x141>{});
    v = dpp(v, std::integral_constant<int, 0x140>{});
    uint2 w = __builtin_bit_cast(uint2, v);
    const auto rl = __builtin_amdgcn_permlane16_swap(w.x, w.x, false, false);
    const auto rh = __builtin_amdgcn_permlane16_swap(w.y, w.y, false, false);
    v = join(make_uint2((uint32_t)rl[0], (uint32_t)rh[0]), make_uint2((uint32_t)rl[1], (uint32_t)rh[1]));
    w = __builtin_bit_cast(uint2, v);
    const auto hl = __builtin_amdgcn_permlane32_swap(w.x, w.x, false, false);
    const auto hh = __builtin_amdgcn_permlane32_swap(w.y, w.y, false, false);
    return join(make_uint2((uint32_t)hl[0], (uint32_t)hh[0]), make_uint2((uint32_t)hl[1], (uint32_t)hh[1]));
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_join(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}

// ------------------------------------------------------------------ SwiGLU, bit for bit swiglu_f32's values
// exp_fixed without its three special cases: x is first brought into [-105, 89], outside of which the fixed sequence
// gives 0 and infinity by itself. (A NaN becomes a number here; the quotient g / (1 + e) is a NaN all the same.)
__device__ __forceinline__ float exp_fixed_clamped(float x) {
    return exp_fixed_sequence(__builtin_amdgcn_fmed3f(x, -105.0f, 89.0f));
}

// silu[e] = g / d and sig[e] = 1 / d, d = 1 + e^-g, both correctly rounded. Markstein's division: y, one Newton step
// from the hardware's reciprocal, is the correctly rounded 1 / d (checked for every mantissa of d); q = g y is within an
// ulp of the quotient, its remainder g - q d is exact, and q + remainder y rounds to the quotient. That holds while
// nothing under- or overflows, which 2^-100 <= |g| <= 80 ensures; a wave that holds any other value (zeros, tiny or
// huge ones, NaN) divides by the ordinary sequence: 6 operations instead of 20 for the pair.
__device__ __forceinline__ void silu8(const float (&g)[8], float (&silu)[8], float (&sig)[8]) {
    float hi = 0.0f, lo = 80.0f, d[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        d[e] = 1.0f + exp_fixed_clamped(-g[e]);
        const float y0 = __builtin_amdgcn_rcpf(d[e]);
        sig[e] = __builtin_fmaf(__builtin_fmaf(-d[e], y0, 1.0f), y0, y0);
        const float q = g[e] * sig[e];
        silu[e] = __builtin_fmaf(__builtin_fmaf(-q, d[e], g[e]), sig[e], q);
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        hi = amax3(hi, g[e], g[e + 1]);
        lo = __builtin_elementwise_minimum(__builtin_elementwise_minimum(lo, __builtin_fabsf(g[e])), __builtin_fabsf(g[e + 1]));
    }
    if (__any(!(hi <= 80.0f && lo >= 0x1p-100f))) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            silu[e] = g[e] / d[e];
            sig[e] = 1.0f / d[e];
        }
    }
}

}  // namespace mxq
