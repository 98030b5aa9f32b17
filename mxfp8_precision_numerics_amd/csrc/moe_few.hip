// The routed experts of a few tokens (T <= 64) in two launches, for gfx950. Per token t, with the k largest logits
// (ties to the lower expert) and p their softmax weights:
//     c = bf16(x^ Wup_e^T),  h = MX(silu(c_gate) c_up),  y = bf16(sum_e p_e (h^ Wdown_e^T))
// where ^ is the value an MXFP8 tensor stands for: the arithmetic of the grouped products and the fused SwiGLU
// quantize that training uses, so a decoded token sees the numbers of the training forward.
//
// The work is reading the chosen experts' weights once. Both kernels convert codes times block scale to bf16 (exact)
// in registers and multiply with v_mfma_f32_16x16x32_bf16: weight rows are the instruction's rows, tokens its columns,
// so up to 16 tokens of an expert cost one pass of matrix instructions over weights that are already on the chip.
// Operand layout used (lane l): A row l % 16, B column l % 16, k = 8 (l / 16) .. + 7; D column l % 16, rows
// 4 (l / 16) .. + 3. The order of k inside a product is free, so lane group l / 16 takes the 16 bytes 16 (l / 16) of a
// 64-byte piece of its row with one load and feeds its two halves to two instructions.
//
// Slots. A workgroup finds for itself which tokens its expert has, from the logits. With T k < experts a slot is a
// (token, rank) pair and a pair whose expert an earlier token also chose stands down; otherwise a slot is an expert.
#pragma clang fp contract(off)
#include "launch.h"
#include "mx_block.h"

namespace mxq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes -> bf16, times 2^E with E the exponent field of `scale` (exact where the product is representable).
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t lo, uint32_t hi, float scale) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, scale, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, scale, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, scale, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

constexpr int MF_THREADS = 512, MF_WAVES = 8, MF_TOK = 64;

struct MoeArgs {
    const uint8_t *x_q, *x_s;
    const float* logits;
    const uint8_t *up_q, *up_s, *down_q, *down_s;
    int T, E, k, D, F, pairs, slots, normalize;     // pairs: a slot is a (token, rank) pair
    // workspace
    int* slot_e;            // [slots] the slot's expert
    int* slot_n;            // [slots] its tokens, 0 for a slot that stands down
    uint16_t* slot_tok;     // [slots][64] token | rank << 8
    float* sel;             // [E or k][64]: the logit of a chosen expert, -inf where none is, NaN for a refused token
    uint8_t *h_q, *h_s;     // [T k][F], [T k][F / 32]
    uint16_t* y;
};

// Which tokens choose expert e: wave 0's lane t returns its rank of e (0 .. k-1), or -1. `bad` (LDS) marks tokens whose
// logits hold a NaN or +inf: they choose nothing. Every thread of the workgroup calls this.
__device__ __forceinline__ int ranks_of(const MoeArgs& a, int e, float (*tile)[65], int* cnt, int* bad, float& mine) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    if (tid < MF_TOK) { cnt[tid] = 0; bad[tid] = 0; }
    mine = lane < a.T ? a.logits[(int64_t)lane * a.E + e] : 0.0f;
    for (int j0 = 0; j0 < a.E; j0 += 64) {
        __syncthreads();
        for (int i = tid; i < a.T * 64; i += MF_THREADS) {
            const int t = i >> 6, j = i & 63;
            tile[t][j] = j0 + j < a.E ? a.logits[(int64_t)t * a.E + j0 + j] : -__builtin_inff();
        }
        __syncthreads();
        int n = 0, b = 0;
        if (lane < a.T) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int j = 8 * w + q;
                const float v = tile[lane][j];
                n += (v > mine || (v == mine && j0 + j < e)) ? 1 : 0;
                b |= !(v < __builtin_inff()) ? 1 : 0;
            }
            if (n) atomicAdd(&cnt[lane], n);
            if (b) atomicOr(&bad[lane], 1);
        }
    }
    __syncthreads();
    return lane < a.T && !bad[lane] && cnt[lane] < a.k && mine > -__builtin_inff() ? cnt[lane] : -1;
}

// ---------------------------------------------------------------------------------------- up/gate and SwiGLU
// Workgroup (f0, slot): 32 gate and 32 up rows of one expert; its 8 waves split the contraction in 64-byte pieces and
// join their partial sums through LDS in a fixed order.
__global__ __launch_bounds__(MF_THREADS) void moe_up_kernel(MoeArgs a) {
    __shared__ __attribute__((aligned(16))) float red[MF_WAVES][16][68];
    __shared__ int cnt[MF_TOK], bad[MF_TOK];
    __shared__ uint16_t list[MF_TOK];
    __shared__ int chosen, total;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int slot = blockIdx.y;
    float (*tile)[65] = reinterpret_cast<float (*)[65]>(&red[0][0][0]);       // 64 x 65 floats of the 8 x 16 x 68
    int e = slot, t0 = 0, r0 = 0;
    if (a.pairs) {
        t0 = slot / a.k;
        r0 = slot - t0 * a.k;
        if (tid == 0) chosen = -1;
        __syncthreads();
        const float* l = a.logits + (int64_t)t0 * a.E;
        for (int j = tid; j < a.E; j += MF_THREADS) {
            const float v = l[j];
            int n = 0, nan = 0;
            for (int i = 0; i < a.E; ++i) {
                const float o = l[i];
                n += (o > v || (o == v && i < j)) ? 1 : 0;
                nan |= o != o ? 1 : 0;
            }
            if (!nan && n == r0) chosen = j;                                 // ranks are distinct: one thread writes
        }
        __syncthreads();
        e = chosen;
        if (e < 0) {                                                         // the token's logits hold a NaN
            if (blockIdx.x == 0 && tid == 0) {
                a.slot_n[slot] = 0;
                a.sel[r0 * MF_TOK + t0] = __builtin_nanf("");
            }
            return;
        }
    }
    float mine;
    const int rank = ranks_of(a, e, tile, cnt, bad, mine);
    if (w == 0) {
        const uint64_t m = __ballot(rank >= 0);
        const int n = __builtin_popcountll(m);
        const int at = __builtin_popcountll(m & ((1ull << lane) - 1));
        if (rank >= 0) list[at] = (uint16_t)(lane | rank << 8);
        const bool dup = a.pairs && ((m & ((1ull << t0) - 1)) != 0 || ((m >> t0) & 1) == 0);
        if (lane == 0) total = dup ? 0 : n;
        if (blockIdx.x == 0) {
            if (a.pairs) {
                if (lane == t0) a.sel[r0 * MF_TOK + t0] = bad[lane] ? __builtin_nanf("") : mine;
            } else if (lane < a.T) {
                a.sel[e * MF_TOK + lane] = bad[lane] ? __builtin_nanf("") : rank >= 0 ? mine : -__builtin_inff();
            }
            if (rank >= 0) a.slot_tok[slot * MF_TOK + at] = (uint16_t)(lane | rank << 8);
            if (lane == 0) {
                a.slot_e[slot] = e;
                a.slot_n[slot] = dup ? 0 : n;
            }
        }
    }
    __syncthreads();
    const int n = total;
    const int64_t f0 = (int64_t)blockIdx.x * 32;
    const int64_t D = a.D, F = a.F;
    const int r = lane & 15, g = lane >> 4;
    const uint8_t* wq[4];
    const uint8_t* ws[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {                                            // gate rows 0-15, 16-31, up rows 0-15, 16-31
        const int64_t row = (int64_t)e * 2 * F + (i >> 1) * F + f0 + 16 * (i & 1) + r;
        wq[i] = a.up_q + row * D;
        ws[i] = a.up_s + row * (D / 32);
    }
    for (int tb = 0; tb < n; tb += 16) {
        v4f acc[4] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
        const int tok = tb + r < n ? list[tb + r] & 255 : -1;
        for (int kc = 64 * w; kc < D; kc += 64 * MF_WAVES) {
            const int k = kc + 16 * g;
            const bool in = k < D;                                           // D % 32 == 0: 16 bytes are whole
            uint4 xv = make_uint4(0u, 0u, 0u, 0u);
            uint32_t xs = 0;
            if (in && tok >= 0) {
                xv = *reinterpret_cast<const uint4*>(a.x_q + tok * D + k);
                xs = a.x_s[tok * (D / 32) + k / 32];
            }
            const float xf = scale_operand(xs);
            const bf16x8 x0 = codes_bf16(xv.x, xv.y, xf), x1 = codes_bf16(xv.z, xv.w, xf);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                uint32_t s = 0;
                if (in) {
                    v = *reinterpret_cast<const uint4*>(wq[i] + k);
                    s = ws[i][k / 32];
                }
                const float f = scale_operand(s);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(v.x, v.y, f), x0, acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(v.z, v.w, f), x1, acc[i], 0, 0, 0);
            }
        }
        __syncthreads();                                                     // red: read by the tile before
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(&red[w][r][16 * i + 4 * g]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        __syncthreads();
        const int f = tid & 31, col = tid >> 5;
        float cg = 0.0f, cu = 0.0f;
#pragma unroll
        for (int q = 0; q < MF_WAVES; ++q) {
            cg += red[q][col][f];
            cu += red[q][col][32 + f];
        }
        cg = (float)(__bf16)cg;                                              // the product's output type
        cu = (float)(__bf16)cu;
        const float h = swiglu_f32(cg, cu);
        uint32_t m = __float_as_uint(h) & 0x7FFFFFFFu;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
        const uint32_t byte = mx_scale_byte_f32(m, RULE_RCEIL);
        const uint32_t code = encode4(h, h, h, h, mx_inv_scale_f32(byte)) & 0xFFu;
        if (tb + col < n) {
            const int tr = list[tb + col];
            const int64_t pair = (int64_t)(tr & 255) * a.k + (tr >> 8);
            a.h_q[pair * F + f0 + f] = (uint8_t)code;
            if (f == 0) a.h_s[pair * (F / 32) + blockIdx.x] = (uint8_t)byte;
        }
    }
}

// ---------------------------------------------------------------------------------------- down and the weighted sum
// Workgroup: 16 output columns of every token. Wave w takes the w-th, (w + 8)-th, ... slot that has tokens, and adds
// p times its product into its own LDS rows; the 8 waves' rows are added in order at the end.
__global__ __launch_bounds__(MF_THREADS) void moe_down_kernel(MoeArgs a) {
    __shared__ __attribute__((aligned(16))) float yl[MF_WAVES][MF_TOK][20];   // 16 columns, padded against bank conflicts
    __shared__ float red[MF_WAVES][MF_TOK], top[MF_TOK], inv[MF_TOK];
    __shared__ int bad[MF_TOK];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int64_t d0 = (int64_t)blockIdx.x * 16, D = a.D, F = a.F;
    const int r = lane & 15, g = lane >> 4;
    const float ninf = -__builtin_inff();
    // softmax statistics of token = lane over its chosen logits (or over all of them)
    const int n_sel = a.pairs ? a.k : a.E;
    float m = ninf;
    int nan = 0;
    if (lane < a.T)
        for (int j = w; j < n_sel; j += MF_WAVES) {
            const float v = a.sel[j * MF_TOK + lane];
            nan |= v != v ? 1 : 0;
            m = __builtin_fmaxf(m, v);
        }
    if (tid < MF_TOK) bad[tid] = 0;
    red[w][lane] = m;
    for (int i = lane; i < MF_TOK * 20; i += 64) (&yl[w][0][0])[i] = 0.0f;
    __syncthreads();
    if (nan) atomicOr(&bad[lane], 1);
#pragma unroll
    for (int q = 0; q < MF_WAVES; ++q) m = __builtin_fmaxf(m, red[q][lane]);
    __syncthreads();
    float s = 0.0f;
    if (lane < a.T && m > ninf) {
        if (a.normalize) {
            for (int j = w; j < n_sel; j += MF_WAVES) s += exp_fixed(a.sel[j * MF_TOK + lane] - m);
        } else {
            for (int j = w; j < a.E; j += MF_WAVES) s += exp_fixed(a.logits[(int64_t)lane * a.E + j] - m);
        }
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0) {
        s = 0.0f;
#pragma unroll
        for (int q = 0; q < MF_WAVES; ++q) s += red[q][lane];
        top[lane] = m;
        inv[lane] = 1.0f / s;
    }
    __syncthreads();
    int seen = 0;                                                            // slots with tokens so far
    for (int sb = 0; sb < a.slots; sb += 64) {
        const int cntv = sb + lane < a.slots ? a.slot_n[sb + lane] : 0;
        uint64_t live = __ballot(cntv > 0);
        while (live) {
            const int at = __builtin_ctzll(live);
            live &= live - 1;
            if ((seen++ & (MF_WAVES - 1)) != w) continue;
            const int slot = sb + at;
            const int n = __builtin_amdgcn_readfirstlane(__shfl(cntv, at, 64));
            const int e = a.slot_e[slot];
            const int64_t row = (int64_t)e * D + d0 + r;
            const uint8_t* wq = a.down_q + row * F;
            const uint8_t* ws = a.down_s + row * (F / 32);
            for (int tb = 0; tb < n; tb += 16) {
                const int tr = tb + r < n ? a.slot_tok[slot * MF_TOK + tb + r] : -1;
                const int64_t pair = tr < 0 ? 0 : (int64_t)(tr & 255) * a.k + (tr >> 8);
                v4f acc = v4f{0, 0, 0, 0};
#pragma unroll 4
                for (int kc = 0; kc < F; kc += 64) {
                    const int k = kc + 16 * g;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u), hv = v;
                    uint32_t vs = 0, hs = 0;
                    if (k < F) {
                        v = *reinterpret_cast<const uint4*>(wq + k);
                        vs = ws[k / 32];
                    }
                    if (k < F && tr >= 0) {
                        hv = *reinterpret_cast<const uint4*>(a.h_q + pair * F + k);
                        hs = a.h_s[pair * (F / 32) + k / 32];
                    }
                    const float vf = scale_operand(vs), hf = scale_operand(hs);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(v.x, v.y, vf), codes_bf16(hv.x, hv.y, hf), acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(v.z, v.w, vf), codes_bf16(hv.z, hv.w, hf), acc, 0, 0, 0);
                }
                if (tr >= 0) {
                    const int t = tr & 255;
                    const float p = exp_fixed(a.logits[(int64_t)t * a.E + e] - top[t]) * inv[t];
                    float4* o = reinterpret_cast<float4*>(&yl[w][t][4 * g]);
                    float4 y = *o;
                    y.x += p * acc[0]; y.y += p * acc[1]; y.z += p * acc[2]; y.w += p * acc[3];
                    *o = y;
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * 16; i += MF_THREADS) {
        const int t = i >> 4, c = i & 15;
        float y = 0.0f;
#pragma unroll
        for (int q = 0; q < MF_WAVES; ++q) y += yl[q][t][c];
        if (bad[t]) y = __builtin_nanf("");
        a.y[t * D + d0 + c] = __builtin_bit_cast(uint16_t, (__bf16)y);
    }
}

// ---------------------------------------------------------------------------------------- launcher
static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Slots: (token, rank) pairs while they are fewer than the experts, else one per expert.
static int moe_few_slots(int64_t T, int64_t E, int64_t k) { return (int)(T * k < E ? T * k : E); }

size_t moe_few_workspace(int64_t T, int64_t E, int64_t k, int64_t F) {
    const size_t slots = (size_t)moe_few_slots(T, E, k);
    return 2 * up256(4 * slots) + up256(2 * slots * MF_TOK) + up256(4 * (size_t)E * MF_TOK) + up256((size_t)(T * k * F)) +
           up256((size_t)(T * k * (F / 32)));
}

hipError_t launch_moe_few(const uint8_t* x_q, const uint8_t* x_s, const float* logits, const uint8_t* up_q,
                          const uint8_t* up_s, const uint8_t* down_q, const uint8_t* down_s, int64_t T, int64_t E,
                          int64_t k, int64_t D, int64_t F, int normalize, uint16_t* y, void* workspace,
                          hipStream_t stream) {
    const int slots = moe_few_slots(T, E, k);
    MoeArgs a{x_q, x_s, logits, up_q, up_s, down_q, down_s, (int)T, (int)E, (int)k, (int)D, (int)F,
              T * k < E ? 1 : 0, slots, normalize};
    uint8_t* p = static_cast<uint8_t*>(workspace);
    a.slot_e = reinterpret_cast<int*>(p); p += up256(4 * (size_t)slots);
    a.slot_n = reinterpret_cast<int*>(p); p += up256(4 * (size_t)slots);
    a.slot_tok = reinterpret_cast<uint16_t*>(p); p += up256(2 * (size_t)slots * MF_TOK);
    a.sel = reinterpret_cast<float*>(p); p += up256(4 * (size_t)E * MF_TOK);
    a.h_q = p; p += up256((size_t)(T * k * F));
    a.h_s = p;
    a.y = y;
    hipLaunchKernelGGL(moe_up_kernel, dim3((unsigned)(F / 32), (unsigned)slots), dim3(MF_THREADS), 0, stream, a);
    hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(D / 16)), dim3(MF_THREADS), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxq
