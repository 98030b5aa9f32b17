// Device helpers shared by the block kernels (norm.hip, checkpoint.hip, moe_few.hip): 8 values of one row as packed
// bf16, fp32 or MXFP8, and the sums across a wave. Internal; not part of the C ABI.
#pragma once
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

__device__ __forceinline__ uint32_t amax8_f32(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
    return m;
}

// The MXFP8 row form of this lane's 8 consecutive values, its 32-value block being the 4 lanes of its quad.
template <int RULE>
__device__ __forceinline__ uint2 encode_row8(const float (&x)[8], uint32_t& byte) {
    byte = mx_scale_byte_f32(quad_max(amax8_f32(x)), RULE);
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

// Sum over the 64 lanes of a wave; every lane gets the same value (each step adds the same two numbers on both sides).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

}  // namespace mxq
