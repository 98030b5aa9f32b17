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

constexpr int MF_UP_THREADS = 512, MF_UP_WAVES = 8, MF_DOWN_THREADS = 1024, MF_DOWN_WAVES = 16, MF_TOK = 64;

struct MoeArgs {
    const uint8_t *x_q, *x_s;
    const float* logits;
    const uint8_t *up_q, *up_s, *down_q, *down_s;
    int T, E, k, D, F, pairs, slots, normalize;     // pairs: a slot is a (token, rank) pair
    // workspace
    int* slot_e;            // [slots] the slot's expert
    int* slot_n;            // [slots] its tokens, 0 for a slot that stands down
    uint16_t* slot_tok;     // [slots][64] token | rank << 8
    float* sel;             // [k][64]: a token's logit of each rank, -inf for a masked one; NaN for a refused token
    uint8_t *h_q, *h_s;     // [T k][F], [T k][F / 32]
    uint16_t* y;
};

// The wave holds one token's logits, expert 64 q + lane in v[q], -inf past the last.
template <int NQ>
struct LogitRow {
    float v[NQ];
    __device__ __forceinline__ LogitRow(const float* row, int E) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int q = 0; q < NQ; ++q) v[q] = 64 * q + lane < E ? row[64 * q + lane] : -__builtin_inff();
    }
    __device__ __forceinline__ bool refused() const {            // a NaN or +inf among them
        bool b = false;
#pragma unroll
        for (int q = 0; q < NQ; ++q) b = b || !(v[q] < __builtin_inff());
        return __any(b);
    }
    // The expert of rank r (equal logits by the lower index), its logit in `value`; -1 if that logit is -inf.
    __device__ __forceinline__ int expert_of(int r, float& value) {
        const int lane = threadIdx.x & 63;
        int e = -1;
        for (int i = 0; i <= r; ++i) {
            float m = v[0];
#pragma unroll
            for (int q = 1; q < NQ; ++q) m = __builtin_fmaxf(m, v[q]);
            value = m = wave_max(m);
            if (m == -__builtin_inff()) return -1;
            e = -1;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const uint64_t b = __ballot(v[q] == m);
                if (e < 0 && b) {
                    e = 64 * q + __builtin_ctzll(b);
                    if (lane == (e & 63)) v[q] = -__builtin_inff();
                }
            }
        }
        return e;
    }
    // The rank of expert e, its logit in `value`.
    __device__ __forceinline__ int rank_of(int e, float& value) const {
        const int lane = threadIdx.x & 63;
        value = 0.0f;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            if (q == e >> 6) value = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v[q]), e & 63));
        int n = 0;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            n += __builtin_popcountll(__ballot(v[q] > value || (v[q] == value && 64 * q + lane < e)));
        return n;
    }
};

// ---------------------------------------------------------------------------------------- up/gate and SwiGLU
// Workgroup (f0, slot): 32 gate and 32 up rows of one expert. Its 8 waves take 256 of every 2048 values of the
// contraction each, with all 16 weight loads of a lane (16 KiB a wave) in flight together, and join their partial sums
// through LDS in a fixed order. An expert's tokens go 16 at a time; further ones find the weights in the caches.
// WIDE: D % 256 == 0, so a row's 8 scale bytes of a wave's slice are one aligned load.
template <int NQ, bool WIDE>
__global__ __launch_bounds__(MF_UP_THREADS, 4) void moe_up_kernel(MoeArgs a) {
    __shared__ __attribute__((aligned(16))) float red[MF_UP_WAVES][16][68];
    __shared__ int rk[MF_TOK];
    __shared__ int list[MF_TOK];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.y;
    const bool lead = blockIdx.x == 0;
    const float nan = __builtin_nanf("");
    int e = slot, t0 = 0;
    if (a.pairs) {
        t0 = slot / a.k;
        const int r0 = slot - t0 * a.k;
        LogitRow<NQ> row(a.logits + (int64_t)t0 * a.E, a.E);
        const bool refused = row.refused();
        float value = 0.0f;
        e = refused ? -1 : __builtin_amdgcn_readfirstlane(row.expert_of(r0, value));
        if (lead && tid == 0) a.sel[r0 * MF_TOK + t0] = refused ? nan : value;
        if (e < 0) {
            if (lead && tid == 0) a.slot_n[slot] = 0;
            return;
        }
    }
    if (tid < MF_TOK) rk[tid] = -1;
    __syncthreads();
    for (int t = w; t < a.T; t += MF_UP_WAVES) {
        const LogitRow<NQ> row(a.logits + (int64_t)t * a.E, a.E);
        const bool refused = row.refused();
        float value;
        const int r = row.rank_of(e, value);
        if (lane == 0) {
            if (!refused && r < a.k && value > -__builtin_inff()) rk[t] = r;
            if (lead && !a.pairs) {
                if (refused && e < a.k) a.sel[e * MF_TOK + t] = nan;
                if (!refused && r < a.k) a.sel[r * MF_TOK + t] = value;
            }
        }
    }
    __syncthreads();
    const int rank = rk[lane];
    const uint64_t who = __ballot(rank >= 0);
    const bool dup = a.pairs && (who & ((1ull << t0) - 1)) != 0;              // an earlier token has this expert too
    const int n = dup ? 0 : __builtin_popcountll(who);
    const int at = __builtin_popcountll(who & ((1ull << lane) - 1));
    if (w == 0) {
        if (rank >= 0) list[at] = lane | rank << 8;
        if (lead) {
            if (rank >= 0) a.slot_tok[slot * MF_TOK + at] = (uint16_t)(lane | rank << 8);
            if (lane == 0) {
                a.slot_e[slot] = e;
                a.slot_n[slot] = n;
            }
        }
    }
    if (n == 0) return;
    __syncthreads();
    const uint32_t D = a.D, F = a.F, f0 = blockIdx.x * 32;
    const int r = lane & 15, g = lane >> 4;
    const uint8_t* wq = a.up_q + ((int64_t)e * 2 * F + f0) * D;              // uniform; 32-bit lane offsets below
    const uint8_t* ws = a.up_s + ((int64_t)e * 2 * F + f0) * (D / 32);
    for (int tb = 0; tb < n; tb += 16) {
        v4f acc[4] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
        const int tok = tb + r < n ? list[tb + r] & 255 : -1;
        for (uint32_t k0 = 256 * w; k0 < D; k0 += 256 * MF_UP_WAVES) {
            uint4 v[4][4];                                                   // [piece][gate 0-15, 16-31, up 0-15, 16-31]
            uint2 s8[4];
            uint32_t s1[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t row = (i >> 1) * F + 16 * (i & 1) + r;
                const uint8_t* p = wq + (uint64_t)row * D + k0;
                const uint8_t* q = ws + (uint64_t)row * (D / 32) + k0 / 32;
                if constexpr (WIDE) s8[i] = *reinterpret_cast<const uint2*>(q);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    v[c][i] = make_uint4(0u, 0u, 0u, 0u);
                    s1[c][i] = 0u;
                    if (WIDE || k0 + 64 * c + 16 * g < D) {                  // D % 32 == 0: 16 bytes are whole
                        v[c][i] = ldnt16(p + 64 * c + 16 * g);
                        if constexpr (!WIDE) s1[c][i] = q[2 * c + (g >> 1)];
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint4 xv = make_uint4(0u, 0u, 0u, 0u);
                uint32_t xs = 0;
                const uint32_t k = k0 + 64 * c + 16 * g;
                if (tok >= 0 && (WIDE || k < D)) {
                    xv = *reinterpret_cast<const uint4*>(a.x_q + (tok * D + k));
                    xs = a.x_s[tok * (D / 32) + k / 32];
                }
                const float xf = scale_operand(xs);
                const bf16x8 x0 = codes_bf16(xv.x, xv.y, xf), x1 = codes_bf16(xv.z, xv.w, xf);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t s = s1[c][i];
                    if constexpr (WIDE) s = ((c < 2 ? s8[i].x : s8[i].y) >> (16 * (c & 1) + 8 * (g >> 1))) & 255u;
                    const float f = scale_operand(s);
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(v[c][i].x, v[c][i].y, f), x0, acc[i], 0, 0, 0);
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(v[c][i].z, v[c][i].w, f), x1, acc[i], 0, 0, 0);
                }
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
        for (int q = 0; q < MF_UP_WAVES; ++q) {
            cg += red[q][col][f];
            cu += red[q][col][32 + f];
        }
        cg = (float)(__bf16)cg;                                              // the product's output type
        cu = (float)(__bf16)cu;
        const float h = swiglu_f32(cg, cu);
        uint32_t m = __float_as_uint(h) & 0x7FFFFFFFu;                       // the 32 lanes of a token: one block
        m = quad_max(m);
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, false));
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, false));
        const auto sw = __builtin_amdgcn_permlane16_swap(m, m, false, false);
        m = max((uint32_t)sw[0], (uint32_t)sw[1]);
        const uint32_t byte = mx_scale_byte_f32(m, RULE_RCEIL);
        const uint32_t code = encode4(h, h, h, h, mx_inv_scale_f32(byte)) & 0xFFu;
        if (tb + col < n) {
            const int tr = list[tb + col];
            const uint32_t pair = (tr & 255) * a.k + (tr >> 8);
            a.h_q[(uint64_t)pair * F + f0 + f] = (uint8_t)code;
            if (f == 0) a.h_s[pair * (F / 32) + blockIdx.x] = (uint8_t)byte;
        }
    }
}

// ---------------------------------------------------------------------------------------- down and the weighted sum
// Workgroup: 8 output columns of every token, so that 2048 columns are 256 workgroups. The instruction's 16 rows are
// these 8 weight rows twice, rows 8-15 with the other half of the contraction, and its 16 columns 8 tokens twice; the
// two diagonal 8 x 8 quarters of the result add up to the product. Wave w takes the w-th, (w + 16)-th, ... slot that has
// tokens (two waves a slot, half of the contraction each, while there are at most 8), and adds p times its product into
// its own LDS rows; the 16 waves' rows are added in order at the end, so the result does not depend on timing.
constexpr int MF_PIECES = 8;                                                 // weight loads of a lane in flight

template <int NQ>
__global__ __launch_bounds__(MF_DOWN_THREADS, 4) void moe_down_kernel(MoeArgs a) {
    __shared__ __attribute__((aligned(16))) float yl[MF_DOWN_WAVES][MF_TOK][8];
    __shared__ float top[MF_TOK], inv[MF_TOK];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t D = a.D, F = a.F, d0 = blockIdx.x * 8;
    const int r = lane & 15, g = lane >> 4, r8 = r & 7;
    for (int i = lane; i < a.T * 8; i += 64) (&yl[w][0][0])[i] = 0.0f;
    // softmax statistics: a token per wave, its chosen logits (or all of them) over the lanes
    for (int t = w; t < a.T; t += MF_DOWN_WAVES) {
        const float m = a.sel[t];                                            // rank 0: the largest
        float s = 0.0f;
        if (a.normalize) {
            if (lane < a.k) s = exp_fixed(a.sel[lane * MF_TOK + t] - m);
        } else {
            const LogitRow<NQ> row(a.logits + (int64_t)t * a.E, a.E);
#pragma unroll
            for (int q = 0; q < NQ; ++q) s += exp_fixed(row.v[q] - m);
        }
        s = wave_sum(s);
        if (lane == 0) {
            top[t] = m;
            inv[t] = m == -__builtin_inff() ? 0.0f : 1.0f / s;               // no expert at all: zeros
        }
    }
    int live = 0;
    for (int b = 0; b < a.slots; b += 64) live += __builtin_popcountll(__ballot(b + lane < a.slots && a.slot_n[b + lane] > 0));
    __syncthreads();
    const uint32_t pieces = (F + 63) / 64, split = live <= MF_DOWN_WAVES / 2 ? 2 : 1;
    const uint32_t half = (pieces + 1) / 2;                                  // 64-byte pieces of the lower rows' half
    const uint32_t span = (half + split - 1) / split;                        // ... of which a wave takes this many
    const uint32_t first = (w & (split - 1)) * span, last = min(half, first + span);
    const int mine = w / split, step = MF_DOWN_WAVES / split;
    int seen = 0;                                                            // slots with tokens so far
    for (int b = 0; b < a.slots; b += 64) {
        const int cnt = b + lane < a.slots ? a.slot_n[b + lane] : 0;
        uint64_t rest = __ballot(cnt > 0);
        for (; rest; rest &= rest - 1, ++seen) {
            if (seen % step != mine) continue;
            const int at = __builtin_ctzll(rest), slot = b + at;
            const int n = __builtin_amdgcn_readlane(cnt, at);
            const int e = __builtin_amdgcn_readfirstlane(a.slot_e[slot]);
            const uint8_t* wq = a.down_q + ((int64_t)e * D + d0) * F;        // uniform; 32-bit lane offsets below
            const uint8_t* ws = a.down_s + ((int64_t)e * D + d0) * (F / 32);
            for (uint32_t c0 = first; c0 < last; c0 += MF_PIECES) {
                uint4 v[MF_PIECES];
                uint32_t s[MF_PIECES];
#pragma unroll
                for (int c = 0; c < MF_PIECES; ++c) {
                    const uint32_t k = 64 * (c0 + c + (r >> 3) * half) + 16 * g;
                    v[c] = make_uint4(0u, 0u, 0u, 0u);
                    s[c] = 0u;
                    if (c0 + c < last && k < F) {                            // F % 32 == 0: 16 bytes are whole
                        v[c] = ldnt16(wq + ((uint64_t)r8 * F + k));
                        s[c] = ws[r8 * (F / 32) + k / 32];
                    }
                }
                for (int tb = 0; tb < n; tb += 8) {
                    const int tr = tb + r8 < n ? a.slot_tok[slot * MF_TOK + tb + r8] : -1;
                    const uint32_t pair = tr < 0 ? 0 : (tr & 255) * a.k + (tr >> 8);
                    const uint8_t* hq = a.h_q + (uint64_t)pair * F;
                    const uint8_t* hs = a.h_s + (uint64_t)pair * (F / 32);
                    v4f acc = v4f{0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < MF_PIECES; ++c) {
                        if (c0 + c >= last) break;
                        if (c % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                        const uint32_t k = 64 * (c0 + c + (r >> 3) * half) + 16 * g;
                        uint4 hv = make_uint4(0u, 0u, 0u, 0u);
                        uint32_t hb = 0;
                        if (tr >= 0 && k < F) {
                            hv = *reinterpret_cast<const uint4*>(hq + k);
                            hb = hs[k / 32];
                        }
                        const float vf = scale_operand(s[c]), hf = scale_operand(hb);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(v[c].x, v[c].y, vf), codes_bf16(hv.x, hv.y, hf), acc, 0, 0, 0);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(v[c].z, v[c].w, vf), codes_bf16(hv.z, hv.w, hf), acc, 0, 0, 0);
                    }
                    float o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {                            // + the quarter of rows and columns 8-15
                        const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i]), __float_as_uint(acc[i]), false, false);
                        o[i] = acc[i] + __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)sw[1], 0x128, 0xF, 0xF, false));
                    }
                    if (tr >= 0 && r < 8 && g < 2) {
                        const int t = tr & 255;
                        const float p = exp_fixed(a.logits[(int64_t)t * a.E + e] - top[t]) * inv[t];
                        float4* d = reinterpret_cast<float4*>(&yl[w][t][4 * g]);
                        float4 y = *d;
                        y.x += p * o[0]; y.y += p * o[1]; y.z += p * o[2]; y.w += p * o[3];
                        *d = y;
                    }
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * 8; i += MF_DOWN_THREADS) {
        const int t = i >> 3, c = i & 7;
        float y = 0.0f;
#pragma unroll
        for (int q = 0; q < MF_DOWN_WAVES; ++q) y += yl[q][t][c];
        if (top[t] != top[t]) y = __builtin_nanf("");                        // a NaN or +inf among the token's logits
        a.y[(int64_t)t * D + d0 + c] = __builtin_bit_cast(uint16_t, (__bf16)y);
    }
}

// ---------------------------------------------------------------------------------------- launcher
static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Slots: (token, rank) pairs while they are fewer than the experts, else one per expert.
static int moe_few_slots(int64_t T, int64_t E, int64_t k) { return (int)(T * k < E ? T * k : E); }

size_t moe_few_workspace(int64_t T, int64_t E, int64_t k, int64_t F) {
    const size_t slots = (size_t)moe_few_slots(T, E, k);
    return 2 * up256(4 * slots) + up256(2 * slots * MF_TOK) + up256(4 * (size_t)k * MF_TOK) + up256((size_t)(T * k * F)) +
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
    a.sel = reinterpret_cast<float*>(p); p += up256(4 * (size_t)k * MF_TOK);
    a.h_q = p; p += up256((size_t)(T * k * F));
    a.h_s = p;
    a.y = y;
    const dim3 up((unsigned)(F / 32), (unsigned)slots), down((unsigned)(D / 8));
#define MXQ_MOE_FEW(NQ)                                                                                            \
    do {                                                                                                           \
        if (D % 256 == 0) hipLaunchKernelGGL((moe_up_kernel<NQ, true>), up, dim3(MF_UP_THREADS), 0, stream, a);    \
        else hipLaunchKernelGGL((moe_up_kernel<NQ, false>), up, dim3(MF_UP_THREADS), 0, stream, a);                \
        hipLaunchKernelGGL(moe_down_kernel<NQ>, down, dim3(MF_DOWN_THREADS), 0, stream, a);                        \
    } while (0)
    if (E <= 64) MXQ_MOE_FEW(1);
    else if (E <= 256) MXQ_MOE_FEW(4);
    else MXQ_MOE_FEW(16);
#undef MXQ_MOE_FEW
    return hipGetLastError();
}

}  // namespace mxq
