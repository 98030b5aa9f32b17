// The routed experts of a few tokens (T <= 64) in two or three launches, for gfx950. Per token t, with the k largest logits
// (ties to the lower expert) and p their softmax weights:
//     c = bf16(x^ Wup_e^T),  h = MX(silu(c_gate) c_up),  y = bf16(sum_e p_e (h^ Wdown_e^T))
// where ^ is the value an MXFP8 tensor stands for: the arithmetic of the grouped products and the fused SwiGLU quantize that
// training uses, but for the order of the sums and the experts' outputs, which stay in fp32 until they are added up.
//
// The work is reading the chosen experts' weights, once while a slot has at most 16 tokens (32 in the streaming form's second
// shape, and any number in the split form's while D <= 2048). Both kernels convert codes times block scale to bf16 (exact)
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
    float* o;               // [T k][D]: the experts' outputs (many slots)
    uint16_t* y;
};

// The wave holds one token's logits, expert 64 q + lane in v[q], -inf past the last.
template <int NQ>
struct LogitRow {
    float v[NQ];
    __device__ __forceinline__ LogitRow() {}
    __device__ __forceinline__ LogitRow(const float* row, int E) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int q = 0; q < NQ; ++q) v[q] = 64 * q + lane < E ? row[64 * q + lane] : -__builtin_inff();
    }
    __device__ __forceinline__ void load(const float* logits, int E, int t, int T) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int q = 0; q < NQ; ++q) v[q] = t < T && 64 * q + lane < E ? logits[(int64_t)t * E + 64 * q + lane] : -__builtin_inff();
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

// ---------------------------------------------------------------------------------------- up/gate, few slots
// Workgroup (f0, slot): 32 gate and 32 up rows of one expert. Its 8 waves take 256 of every 2048 values of the
// contraction each, with all 16 weight loads of a lane (16 KiB a wave) in flight together, and join their partial sums
// through LDS in a fixed order. An expert's tokens go 16 at a time.
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
    constexpr int BATCH = NQ == 1 ? 8 : NQ == 4 ? 2 : 1;                     // tokens whose logits are loaded together
    const uint32_t D = a.D, F = a.F, f0 = blockIdx.x * 32;
    const int r = lane & 15, g = lane >> 4;
    int e = slot, t0 = 0, r0 = 0;
    if (a.pairs) {
        t0 = slot / a.k;
        r0 = slot - t0 * a.k;
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
    uint4 v[4][4];                                                           // [piece][gate 0-15, 16-31, up 0-15, 16-31]
    uint2 s8[4];
    uint32_t s1[4][4];
    auto load = [&](uint32_t k0) {
        const uint8_t* wq = a.up_q + ((int64_t)e * 2 * F + f0) * D;          // uniform; 32-bit lane offsets
        const uint8_t* ws = a.up_s + ((int64_t)e * 2 * F + f0) * (D / 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t* p = wq + ((uint64_t)(i >> 1) * F + 16 * (i & 1)) * D;
            const uint8_t* q = ws + ((uint64_t)(i >> 1) * F + 16 * (i & 1)) * (D / 32);
            if constexpr (WIDE) s8[i] = *reinterpret_cast<const uint2*>(q + (r * (D / 32) + k0 / 32));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t k = k0 + 64 * c + 16 * g;
                v[c][i] = make_uint4(0u, 0u, 0u, 0u);
                s1[c][i] = 0u;
                if (WIDE || k < D) {                                         // D % 32 == 0: 16 bytes are whole
                    v[c][i] = ldnt16(p + (r * D + k));
                    if constexpr (!WIDE) s1[c][i] = q[r * (D / 32) + k / 32];
                }
            }
        }
    };
    // the ranks of e: token t = w + 8 i is ranked by wave w
    LogitRow<NQ> row[BATCH];
    if (a.T > 1 || !a.pairs) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) row[i].load(a.logits, a.E, w + MF_UP_WAVES * i, a.T);
    }
    if (tid < MF_TOK) rk[tid] = a.T == 1 && a.pairs && tid == 0 ? r0 : -1;
    __syncthreads();
    if (a.T > 1 || !a.pairs) {
        for (int tt = w; tt < a.T; tt += MF_UP_WAVES * BATCH) {
            if (tt != w) {
#pragma unroll
                for (int i = 0; i < BATCH; ++i) row[i].load(a.logits, a.E, tt + MF_UP_WAVES * i, a.T);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int t = tt + MF_UP_WAVES * i;
                if (t >= a.T) break;
                const bool refused = row[i].refused();
                float value;
                const int rank = row[i].rank_of(e, value);
                if (lane == 0) {
                    if (!refused && rank < a.k && value > -__builtin_inff()) rk[t] = rank;
                    if (lead && !a.pairs) {
                        if (refused && e < a.k) a.sel[e * MF_TOK + t] = nan;
                        if (!refused && rank < a.k) a.sel[rank * MF_TOK + t] = value;
                    }
                }
            }
        }
        __syncthreads();
    }
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
    if (256 * w < D) load(256 * w);
    __syncthreads();
    for (int tb = 0; tb < n; tb += 16) {
        v4f acc[4] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
        const int tok = tb + r < n ? list[tb + r] & 255 : -1;
        for (uint32_t k0 = 256 * w; k0 < D; k0 += 256 * MF_UP_WAVES) {
            // the first slice is there; one slice (D <= 2048) stays in the registers for all tokens
            if ((tb != 0 && D > 256 * MF_UP_WAVES) || k0 >= 256 * MF_UP_WAVES) load(k0);
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
        if (tb + (w << 1) >= n) continue;                                    // this wave's two tokens are past the list
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

// ---------------------------------------------------------------------------------------- down and the sum, few slots
// Workgroup: 8 output columns of every token, so that 2048 columns are 256 workgroups. The instruction's 16 rows are
// these 8 weight rows twice, rows 8-15 with the other half of the contraction, and its 16 columns 8 tokens twice; the
// two diagonal 8 x 8 quarters of the result add up to the product. Wave w takes the w-th, (w + 16)-th, ... slot that has
// tokens (two waves a slot, half of the contraction each, while there are at most 8), and adds p times its product into
// its own LDS rows; the 16 waves' rows are added in order at the end, so the result does not depend on timing. Slots are
// taken in the order of their experts, which is the same for every order of the batch's tokens (a single token's, in the
// order of its ranks).
constexpr int MF_PIECES = 4;                                                 // weight loads of a lane in flight

// One slot's share of a wave: 8 rows of its weights (up to MF_PIECES 64-byte pieces of each half of the contraction), and
// the slot's token list, entry l in lane l.
struct DownItem {
    uint4 v[MF_PIECES];
    uint32_t s[MF_PIECES];
    int tok;
};

template <int NQ>
__global__ __launch_bounds__(MF_DOWN_THREADS, 4) void moe_down_kernel(MoeArgs a) {
    __shared__ __attribute__((aligned(16))) float yl[MF_DOWN_WAVES][MF_TOK][8];
    __shared__ float top[MF_TOK], inv[MF_TOK];
    __shared__ int live_slot[NQ * 64], live_e[NQ * 64], live_n[NQ * 64], live_count;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t D = a.D, F = a.F, d0 = blockIdx.x * 8;
    const int r = lane & 15, g = lane >> 4, r8 = r & 7;
    if (w == MF_DOWN_WAVES - 1) {                                            // the slots that have tokens
        int cnt[NQ], ex[NQ], before = 0;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const bool in = 64 * q + lane < a.slots;
            cnt[q] = in ? a.slot_n[64 * q + lane] : 0;
            ex[q] = in ? a.slot_e[64 * q + lane] : 0;
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const uint64_t b = __ballot(cnt[q] > 0);
            int at = before + __builtin_popcountll(b & ((1ull << lane) - 1));
            if (q == 0 && a.pairs && a.T > 1) {                              // at most 16 slots: all in lanes 0 to 15
                at = 0;
#pragma unroll
                for (int i = 0; i < MF_DOWN_WAVES; ++i)
                    at += (b >> i & 1) && __builtin_amdgcn_readlane(ex[0], i) < ex[0] ? 1 : 0;
            }
            if (cnt[q] > 0) {
                live_slot[at] = 64 * q + lane;
                live_e[at] = ex[q];
                live_n[at] = cnt[q];
            }
            before += __builtin_popcountll(b);
        }
        if (lane == 0) live_count = before;
    }
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
    for (int i = lane; i < a.T * 8; i += 64) (&yl[w][0][0])[i] = 0.0f;
    __syncthreads();
    const int live = __builtin_amdgcn_readfirstlane(live_count);
    const uint32_t pieces = (F + 63) / 64, split = live <= MF_DOWN_WAVES / 2 ? 2 : 1;
    const uint32_t half = (pieces + 1) / 2;                                  // 64-byte pieces of the lower rows' half
    const uint32_t span = (half + split - 1) / split;                        // ... of which a wave takes this many
    const uint32_t first = (w & (split - 1)) * span, last = min(half, first + span);
    const int step = MF_DOWN_WAVES / split;
    const uint32_t kl = 64 * (r >> 3) * half + 16 * g;                       // this lane's place in a piece pair

    auto load = [&](DownItem& it, int at, uint32_t c0) {
        const int e = __builtin_amdgcn_readfirstlane(live_e[at]);
        const uint8_t* wq = a.down_q + ((int64_t)e * D + d0) * F;            // uniform; 32-bit lane offsets
        const uint8_t* ws = a.down_s + ((int64_t)e * D + d0) * (F / 32);
        it.tok = lane < __builtin_amdgcn_readfirstlane(live_n[at]) ? a.slot_tok[live_slot[at] * MF_TOK + lane] : -1;
#pragma unroll
        for (int c = 0; c < MF_PIECES; ++c) {
            const uint32_t k = 64 * (c0 + c) + kl;
            it.v[c] = make_uint4(0u, 0u, 0u, 0u);
            it.s[c] = 0u;
            if (c0 + c < last && k < F) {                                    // F % 32 == 0: 16 bytes are whole
                it.v[c] = ldnt16(wq + (r8 * F + k));
                it.s[c] = ws[r8 * (F / 32) + k / 32];
            }
        }
    };
    int at = w / split;
    uint32_t c0 = first;
    DownItem next;
    if (at < live) load(next, at, c0);
    while (at < live) {
        const DownItem it = next;
        const int e = __builtin_amdgcn_readfirstlane(live_e[at]), n = __builtin_amdgcn_readfirstlane(live_n[at]);
        const uint32_t base = c0;
        c0 += MF_PIECES;
        if (c0 >= last) {
            c0 = first;
            at += step;
        }
        if (at < live) load(next, at, c0);
        // the tokens' weights, entry l in lane l
        float p = 0.0f;
        if (lane < n) {
            const int t = it.tok & 255;
            p = exp_fixed(a.logits[(int64_t)t * a.E + e] - top[t]) * inv[t];
        }
        for (int tb = 0; tb < n; tb += 8) {
            const int tr = __shfl(it.tok, tb + r8, 64);                      // -1 past the list
            const float pt = __shfl(p, tb + r8, 64);
            const uint32_t pair = tr < 0 ? 0 : (tr & 255) * a.k + (tr >> 8);
            const uint8_t* hq = a.h_q + (uint64_t)pair * F;
            const uint8_t* hs = a.h_s + (uint64_t)pair * (F / 32);
            v4f acc = v4f{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < MF_PIECES; ++c) {
                if (base + c >= last) break;
                const uint32_t k = 64 * (base + c) + kl;
                uint4 hv = make_uint4(0u, 0u, 0u, 0u);
                uint32_t hb = 0;
                if (tr >= 0 && k < F) {
                    hv = *reinterpret_cast<const uint4*>(hq + k);
                    hb = hs[k / 32];
                }
                const float vf = scale_operand(it.s[c]), hf = scale_operand(hb);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(it.v[c].x, it.v[c].y, vf), codes_bf16(hv.x, hv.y, hf), acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(it.v[c].z, it.v[c].w, vf), codes_bf16(hv.z, hv.w, hf), acc, 0, 0, 0);
            }
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {                                    // + the quarter of rows and columns 8-15
                const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i]), __float_as_uint(acc[i]), false, false);
                o[i] = acc[i] + __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)sw[1], 0x128, 0xF, 0xF, false));
            }
            if (tr >= 0 && r < 8 && g < 2) {
                float4* d = reinterpret_cast<float4*>(&yl[w][tr & 255][4 * g]);
                float4 y = *d;
                y.x += pt * o[0]; y.y += pt * o[1]; y.z += pt * o[2]; y.w += pt * o[3];
                *d = y;
            }
            wave_lds_order();                                                // the next tile may hold this token in another lane
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

// ---------------------------------------------------------------------------------------- many slots
// With many slots a wave streams 64 weight rows over the whole contraction for 16 NT tokens of the slot, 256 / NT values at
// a time, the next ones being on their way while it converts and multiplies. A workgroup is one wave, blockIdx.z its
// share of the slot's tokens; those with none come last in launch order and leave at once. NT = 2 where a slot may have
// more than 16 tokens, so that its weights are still read once for up to 32 (twice for more).
// 16 tokens of 64 experts, 2048 and 1024 columns, top 8: up 55 us, down 27 us, 4.2 and 4.3 TB/s of the chosen experts'
// weights; 16% more is fetched than these hold. 61 tokens: 64 and 34 us. (In the split form a workgroup's 128 KiB are in flight at
// once, but only two workgroups fit on a CU, and their ranking, joining and SwiGLU leave the memory idle: 85 us against
// 45 us for a plain read of the same weights. Streaming without the second buffer, ranking, token loads, conversions and
// matrix instructions added up to 79 us; 32 rows a wave read each token twice as often, 10 us of it.)
constexpr int MF_STREAM_THREADS = 64;

// The scale bytes of a wave's 64 rows and 16 tokens wait in LDS, 2048 values' worth at a time: a load touches 16 rows
// whatever its width, so fetching them with each 128 values made half as many requests again as the weights do.
constexpr int MF_SPAN = 2048, MF_SCALE_WORDS = MF_SPAN / 128 + 1;            // a row's words, padded against bank conflicts

// 64-byte pieces of a step: two steps are in flight, 16 KiB of weights each for one tile of tokens, 8 KiB for two, which is
// what the registers of two waves a SIMD hold. With one tile, three waves and 8 KiB a step: 90.6 us against 88.4 at 16
// tokens of 64 experts, 2048 and 1024 columns, top 8, and 145 against 130 at 2080 and 992 columns.
template <int NT>
constexpr int MF_STEP = NT == 1 ? 4 : 2;

template <int NT>
struct StreamBuf {
    uint4 v[MF_STEP<NT>][4], x[MF_STEP<NT>][NT];
};

template <int NT>
struct StreamRows {
    const uint8_t *wq[4], *ws[4];   // lane l's rows 16 i + (l % 16): codes, scales
    const uint8_t *tq[NT], *ts[NT]; // lane l's tokens; past the slot's tokens, its first (the results are not used)
    uint32_t K;
    bool second;                    // there is a second tile of tokens
};

// The scale bytes of values k0 .. k0 + 2047 into the wave's LDS rows: 64 weight rows, then the tokens.
template <int NT>
__device__ __forceinline__ void stream_scales(const StreamRows<NT>& p, uint32_t k0, uint32_t (*lds)[MF_SCALE_WORDS]) {
    const int r = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const uint32_t first = k0 / 32 + 16 * g, bytes = p.K / 32;               // this lane's 16 of the row's bytes
    if (p.K % 512 == 0) {
        uint4 v[4 + NT];
#pragma unroll
        for (int i = 0; i < 4 + NT; ++i) {
            const uint8_t* q = i < 4 ? p.ws[i] : p.ts[i - 4];
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (first < bytes) v[i] = *reinterpret_cast<const uint4*>(q + first);
        }
#pragma unroll
        for (int i = 0; i < 4 + NT; ++i) {
            uint32_t* d = &lds[16 * i + r][4 * g];
            d[0] = v[i].x; d[1] = v[i].y; d[2] = v[i].z; d[3] = v[i].w;
        }
        return;
    }
    // rows that do not start on 16 bytes: byte by byte, 16 in flight, repeating the row's last where it has ended
#pragma unroll
    for (int i = 0; i < 4 + NT; ++i) {
        const uint8_t* q = i < 4 ? p.ws[i] : p.ts[i - 4];
        uint32_t x[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = q[min(first + c, bytes - 1)];
        uint32_t* d = &lds[16 * i + r][4 * g];
#pragma unroll
        for (int c = 0; c < 4; ++c) d[c] = x[4 * c] | x[4 * c + 1] << 8 | x[4 * c + 2] << 16 | x[4 * c + 3] << 24;
    }
}

// One step from k0. WIDE: K is a whole number of steps; otherwise K % 32 == 0 and 16 bytes are whole.
template <bool WIDE, int NT>
__device__ __forceinline__ void stream_load(StreamBuf<NT>& b, const StreamRows<NT>& p, uint32_t k0) {
    const uint32_t k = k0 + 16 * ((threadIdx.x & 63) >> 4);
#pragma unroll
    for (int c = 0; c < MF_STEP<NT>; ++c) {
        const bool in = WIDE || k + 64 * c < p.K;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            b.x[c][t] = make_uint4(0u, 0u, 0u, 0u);
            if (in) b.x[c][t] = *reinterpret_cast<const uint4*>(p.tq[t] + k + 64 * c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b.v[c][i] = make_uint4(0u, 0u, 0u, 0u);
            if (in) b.v[c][i] = ldnt16(p.wq[i] + k + 64 * c);
        }
    }
}

template <int NT>
__device__ __forceinline__ void stream_multiply(const StreamBuf<NT>& b, bool second, const uint32_t (*lds)[MF_SCALE_WORDS],
                                                uint32_t step, v4f (&acc)[NT][4]) {
    const int r = threadIdx.x & 15, sh = 8 * ((threadIdx.x & 63) >> 5);      // lane group g: byte g / 2 of a 64-value piece
#pragma unroll
    for (int c = 0; c < MF_STEP<NT>; ++c) {
        const uint32_t w = (MF_STEP<NT> / 2) * step + c / 2;                 // a word holds the scales of two pieces
        uint32_t vs[4], xs[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xs[t] = lds[64 + 16 * t + r][w] >> (16 * (c & 1) + sh);
#pragma unroll
        for (int i = 0; i < 4; ++i) vs[i] = lds[16 * i + r][w] >> (16 * (c & 1) + sh);
        bf16x8 x0[NT], x1[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float f = scale_operand(xs[t] & 255u);
            x0[t] = codes_bf16(b.x[c][t].x, b.x[c][t].y, f);
            x1[t] = codes_bf16(b.x[c][t].z, b.x[c][t].w, f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = scale_operand(vs[i] & 255u);
            const bf16x8 w0 = codes_bf16(b.v[c][i].x, b.v[c][i].y, f), w1 = codes_bf16(b.v[c][i].z, b.v[c][i].w, f);
            acc[0][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, x0[0], acc[0][i], 0, 0, 0);
            acc[0][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, x1[0], acc[0][i], 0, 0, 0);
            if constexpr (NT == 2) {
                if (second) {
                    acc[1][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, x0[1], acc[1][i], 0, 0, 0);
                    acc[1][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, x1[1], acc[1][i], 0, 0, 0);
                }
            }
        }
    }
}

// acc[t][i] = rows 16 i + (l % 16) times the wave's tokens over K values. The wave begins `turn` steps into the contraction
// and wraps: thousands of waves that all begin at their rows' first bytes, 2 KiB apart, would ask the same few memory
// channels at a time. The place depends on the expert and the rows alone, so a token meets the same order of sums wherever it
// stands in the batch.
template <bool WIDE, int NT>
__device__ __forceinline__ void stream_rows(const StreamRows<NT>& p, uint32_t turn, uint32_t (*lds)[MF_SCALE_WORDS],
                                            v4f (&acc)[NT][4]) {
    StreamBuf<NT> a, b;
    constexpr uint32_t LEN = 64 * MF_STEP<NT>;
    const uint32_t K = p.K;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = v4f{0, 0, 0, 0};
    for (uint32_t base = 0; base < K; base += MF_SPAN) {
        const uint32_t steps = (min(K - base, (uint32_t)MF_SPAN) + LEN - 1) / LEN;
        uint32_t at = turn % steps;
        auto next = [&](uint32_t x) { return x + 1 == steps ? 0u : x + 1; };
        stream_load<WIDE>(a, p, base + LEN * at);
        wave_lds_order();                                                    // the span before has been read
        stream_scales(p, base, lds);
        wave_lds_order();                                                    // each lane reads words that others wrote
        // No load stands behind a condition: where one may be skipped, a wait for the other buffer waits for all.
        uint32_t left = steps;
        for (; left > 2; left -= 2) {
            const uint32_t at1 = next(at), at2 = next(at1);
            stream_load<WIDE>(b, p, base + LEN * at1);
            stream_multiply(a, p.second, lds, at, acc);
            stream_load<WIDE>(a, p, base + LEN * at2);
            stream_multiply(b, p.second, lds, at1, acc);
            at = at2;
        }
        if (left == 2) {
            stream_load<WIDE>(b, p, base + LEN * next(at));
            stream_multiply(a, p.second, lds, at, acc);
            stream_multiply(b, p.second, lds, next(at), acc);
        } else {
            stream_multiply(a, p.second, lds, at, acc);
        }
    }
}

// Up/gate and SwiGLU. Workgroup (f0, slot, tokens): 32 gate and the same 32 up rows, so h and its 32-value blocks form in
// the wave's registers. Ranking: lane t counts how many of token t's logits precede expert e's.
template <int NQ, bool WIDE, int NT>
__global__ __launch_bounds__(MF_STREAM_THREADS, 2) void moe_up_slots_kernel(MoeArgs a) {
    __shared__ int list[MF_TOK];
    __shared__ __attribute__((aligned(16))) uint32_t scales[64 + 16 * NT][MF_SCALE_WORDS];
    const int lane = threadIdx.x;
    const int slot = blockIdx.y, first = 16 * NT * blockIdx.z;
    const bool lead = blockIdx.x == 0 && blockIdx.z == 0;
    const float nan = __builtin_nanf(""), inf = __builtin_inff();
    int e = slot, t0 = 0, r0 = 0;
    if (a.pairs) {
        t0 = slot / a.k;
        r0 = slot - t0 * a.k;
        LogitRow<NQ> row(a.logits + (int64_t)t0 * a.E, a.E);
        const bool refused = row.refused();
        float value = 0.0f;
        e = refused ? -1 : __builtin_amdgcn_readfirstlane(row.expert_of(r0, value));
        if (lead && lane == 0) a.sel[r0 * MF_TOK + t0] = refused ? nan : value;
        if (e < 0) {
            if (lead && lane == 0) a.slot_n[slot] = 0;
            return;
        }
    }
    float mine = 0.0f;
    int rank = 0, worse = 0;
    auto count = [&](float v, int j) {
        rank += (v > mine || (v == mine && j < e)) ? 1 : 0;
        worse |= !(v < inf) ? 1 : 0;
    };
    if (lane < a.T) {
        const float* row = a.logits + lane * a.E;
        mine = row[e];
        if (a.E % 4 == 0) {                                                  // the rows start on 16 bytes
#pragma unroll 8
            for (int j = 0; j < a.E; j += 4) {
                const float4 v = *reinterpret_cast<const float4*>(row + j);
                count(v.x, j); count(v.y, j + 1); count(v.z, j + 2); count(v.w, j + 3);
            }
        } else {
#pragma unroll 8
            for (int j = 0; j < a.E; ++j) count(row[j], j);
        }
    }
    const bool refused = worse != 0;
    const bool has = lane < a.T && !refused && rank < a.k && mine > -inf;
    const uint64_t who = __ballot(has);
    const bool dup = a.pairs && (who & ((1ull << t0) - 1)) != 0;              // an earlier token has this expert too
    const int n = dup ? 0 : __builtin_popcountll(who);
    const int at = __builtin_popcountll(who & ((1ull << lane) - 1));
    if (has) list[at] = lane | rank << 8;
    if (lead) {
        if (has) a.slot_tok[slot * MF_TOK + at] = (uint16_t)(lane | rank << 8);
        if (!a.pairs && lane < a.T) {
            if (refused && e < a.k) a.sel[e * MF_TOK + lane] = nan;
            if (!refused && rank < a.k) a.sel[rank * MF_TOK + lane] = mine;
        }
        if (lane == 0) {
            a.slot_e[slot] = e;
            a.slot_n[slot] = n;
        }
    }
    if (first >= n) return;
    __syncthreads();                                                         // one wave: orders the list's writes and reads
    const uint32_t D = a.D, F = a.F, f0 = blockIdx.x * 32;
    const int r = lane & 15, g = lane >> 4;
    StreamRows<NT> rows;
#pragma unroll
    for (int i = 0; i < 4; ++i) {                                            // gate rows 0-15, 16-31, up rows 0-15, 16-31
        const uint64_t row = (uint64_t)e * 2 * F + (i >> 1) * F + f0 + 16 * (i & 1) + r;
        rows.wq[i] = a.up_q + row * D;
        rows.ws[i] = a.up_s + row * (D / 32);
    }
    int tr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int at = first + 16 * t + r;
        tr[t] = at < n ? list[at] : -1;
        const uint32_t token = (tr[t] < 0 ? list[first] : tr[t]) & 255;
        rows.tq[t] = a.x_q + token * D;
        rows.ts[t] = a.x_s + token * (D / 32);
    }
    rows.K = D;
    rows.second = first + 16 < n;
    v4f acc[NT][4];
    stream_rows<WIDE, NT>(rows, 5 * blockIdx.x + 3 * e, scales, acc);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (first + 16 * t >= n) break;
        float h[2][4];
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) {                                    // the products' output type is bf16
                h[p][i] = swiglu_f32((float)(__bf16)acc[t][p][i], (float)(__bf16)acc[t][2 + p][i]);
                m = max(m, __float_as_uint(h[p][i]) & 0x7FFFFFFFu);
            }
        const auto x = __builtin_amdgcn_permlane16_swap(m, m, false, false); // a token's 32 values: 4 lanes of 8
        m = max((uint32_t)x[0], (uint32_t)x[1]);
        const auto y = __builtin_amdgcn_permlane32_swap(m, m, false, false);
        m = max((uint32_t)y[0], (uint32_t)y[1]);
        const uint32_t byte = mx_scale_byte_f32(m, RULE_RCEIL);
        if (tr[t] >= 0) {
            const uint32_t pair = (tr[t] & 255) * a.k + (tr[t] >> 8);
            uint8_t* q = a.h_q + ((uint64_t)pair * F + f0 + 4 * g);
#pragma unroll
            for (int p = 0; p < 2; ++p)
                *reinterpret_cast<uint32_t*>(q + 16 * p) = encode4(h[p][0], h[p][1], h[p][2], h[p][3], mx_inv_scale_f32(byte));
            if (g == 0) a.h_s[pair * (F / 32) + blockIdx.x] = (uint8_t)byte;
        }
    }
}

// Down. Workgroup (64 output columns, slot): a wave writes its tokens' products (fp32) to their pair's row;
// moe_sum_kernel adds a token's rows in rank order. D % 64 == 32 leaves the last workgroup's upper 32 rows out: they read
// row d0 and store nothing.
template <bool WIDE, int NT>
__global__ __launch_bounds__(MF_STREAM_THREADS, 2) void moe_down_slots_kernel(MoeArgs a) {
    __shared__ __attribute__((aligned(16))) uint32_t scales[64 + 16 * NT][MF_SCALE_WORDS];
    const int lane = threadIdx.x;
    const int slot = blockIdx.y, base = 16 * NT * blockIdx.z;
    const uint32_t D = a.D, F = a.F, d0 = blockIdx.x * 64;
    const int r = lane & 15, g = lane >> 4;
    int tok[NT];                                                             // past the slot's count: not used
#pragma unroll
    for (int t = 0; t < NT; ++t) tok[t] = a.slot_tok[slot * MF_TOK + min(base + 16 * t + r, MF_TOK - 1)];
    const int n = __builtin_amdgcn_readfirstlane(a.slot_n[slot]);
    const int e = a.pairs ? __builtin_amdgcn_readfirstlane(a.slot_e[slot]) : slot;
    if (base >= n) return;
    StreamRows<NT> rows;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t row = (uint64_t)e * D + d0 + (d0 + 16 * i < D ? 16 * i : 0) + r;
        rows.wq[i] = a.down_q + row * F;
        rows.ws[i] = a.down_s + row * (F / 32);
    }
    const int first = __builtin_amdgcn_readfirstlane(tok[0]);                // lane 0's token is there: base < n
    uint32_t pair[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int mine = base + 16 * t + r < n ? tok[t] : first;
        pair[t] = (mine & 255) * a.k + (mine >> 8);
        rows.tq[t] = a.h_q + (uint64_t)pair[t] * F;
        rows.ts[t] = a.h_s + (uint64_t)pair[t] * (F / 32);
    }
    rows.K = F;
    rows.second = base + 16 < n;
    v4f acc[NT][4];
    stream_rows<WIDE, NT>(rows, 5 * blockIdx.x + 3 * e, scales, acc);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (base + 16 * t + r >= n) continue;
        float* o = a.o + ((uint64_t)pair[t] * D + d0 + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (d0 + 16 * i < D)
                *reinterpret_cast<float4*>(o + 16 * i) = make_float4(acc[t][i][0], acc[t][i][1], acc[t][i][2], acc[t][i][3]);
    }
}

// y[t] = sum over ranks of p o[t k + rank], in rank order: 4 columns a thread, 1024 columns of a token a workgroup. Every
// wave forms the softmax of its token's chosen logits for itself.
template <int NQ>
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeArgs a) {
    const int lane = threadIdx.x & 63, t = blockIdx.y;
    const uint32_t d = blockIdx.x * 1024 + 4 * threadIdx.x, D = a.D;
    const float l = lane < a.k ? a.sel[lane * MF_TOK + t] : -__builtin_inff();
    const float m = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(l)));      // rank 0: the largest
    float p = lane < a.k ? exp_fixed(l - m) : 0.0f, sum;
    if (a.normalize) {
        sum = wave_sum(p);
    } else {
        const LogitRow<NQ> row(a.logits + (int64_t)t * a.E, a.E);
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < NQ; ++i) q += exp_fixed(row.v[i] - m);
        sum = wave_sum(q);
    }
    p = p / sum;
    // Lane i's p and logit are read from lane i, so every lane stays; those past the row sum column 0 and store nothing.
    const bool in = d < D;                                                   // D % 32 == 0
    const uint32_t at = in ? d : 0;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < a.k; ++i) {
        if (!(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(l), i)) > -__builtin_inff())) continue;   // masked
        const float pi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p), i));
        const float4 o = *reinterpret_cast<const float4*>(a.o + ((uint64_t)(t * a.k + i) * D + at));
        y[0] += pi * o.x; y[1] += pi * o.y; y[2] += pi * o.z; y[3] += pi * o.w;
    }
    if (m != m) y[0] = y[1] = y[2] = y[3] = m;                               // a NaN or +inf among the token's logits
    if (in) *reinterpret_cast<uint2*>(a.y + ((uint64_t)t * D + d)) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

// ---------------------------------------------------------------------------------------- launcher
static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Slots: (token, rank) pairs while they are fewer than the experts, else one per expert.
static int moe_few_slots(int64_t T, int64_t E, int64_t k) { return (int)(T * k < E ? T * k : E); }

// Up to this many slots the contractions are split over waves; then the streaming form.
static bool moe_few_split(int slots) { return slots <= MF_DOWN_WAVES; }

size_t moe_few_workspace(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F) {
    const size_t slots = (size_t)moe_few_slots(T, E, k);
    return 2 * up256(4 * slots) + up256(2 * slots * MF_TOK) + up256(4 * (size_t)k * MF_TOK) + up256((size_t)(T * k * F)) +
           up256((size_t)(T * k * (F / 32))) + (moe_few_split((int)slots) ? 0 : up256(4 * (size_t)(T * k * D)));
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
    a.h_s = p; p += up256((size_t)(T * k * (F / 32)));
    a.o = reinterpret_cast<float*>(p);
    a.y = y;
    const dim3 up((unsigned)(F / 32), (unsigned)slots), down((unsigned)(D / 8));
    const unsigned shares = T <= 16 ? 1 : (unsigned)((T + 31) / 32);         // of the tokens a slot may have
    const dim3 up_slots(up.x, up.y, shares), down_slots((unsigned)((D + 63) / 64), (unsigned)slots, shares);
    const dim3 sum((unsigned)((D + 1023) / 1024), (unsigned)T), one(MF_STREAM_THREADS);
#define MXQ_MOE_SLOTS(NQ, NT)                                                                                        \
    do {                                                                                                             \
        if (D % (256 / NT) == 0) hipLaunchKernelGGL((moe_up_slots_kernel<NQ, true, NT>), up_slots, one, 0, stream, a); \
        else hipLaunchKernelGGL((moe_up_slots_kernel<NQ, false, NT>), up_slots, one, 0, stream, a);                  \
        if (F % (256 / NT) == 0) hipLaunchKernelGGL((moe_down_slots_kernel<true, NT>), down_slots, one, 0, stream, a); \
        else hipLaunchKernelGGL((moe_down_slots_kernel<false, NT>), down_slots, one, 0, stream, a);                  \
    } while (0)
#define MXQ_MOE_FEW(NQ)                                                                                              \
    do {                                                                                                             \
        if (moe_few_split(slots)) {                                                                                  \
            if (D % 256 == 0) hipLaunchKernelGGL((moe_up_kernel<NQ, true>), up, dim3(MF_UP_THREADS), 0, stream, a);  \
            else hipLaunchKernelGGL((moe_up_kernel<NQ, false>), up, dim3(MF_UP_THREADS), 0, stream, a);              \
            hipLaunchKernelGGL(moe_down_kernel<NQ>, down, dim3(MF_DOWN_THREADS), 0, stream, a);                      \
        } else {                                                                                                     \
            if (T <= 16) MXQ_MOE_SLOTS(NQ, 1);                                                                       \
            else MXQ_MOE_SLOTS(NQ, 2);                                                                               \
            hipLaunchKernelGGL(moe_sum_kernel<NQ>, sum, dim3(256), 0, stream, a);                                    \
        }                                                                                                            \
    } while (0)
    if (E <= 64) MXQ_MOE_FEW(1);
    else if (E <= 256) MXQ_MOE_FEW(4);
    else MXQ_MOE_FEW(16);
#undef MXQ_MOE_FEW
#undef MXQ_MOE_SLOTS
    return hipGetLastError();
}

}  // namespace mxq
