"""One routed (mixture-of-experts) block in MXFP8: trained for a few steps with 8-bit activation checkpoints, then used
to decode single tokens from the same weight caches.

    python examples/moe_block.py

Block: h = x + residual;  y = RMSNorm(h);  out = h + sum over the top-k experts of p_e SwiGLU-MLP_e(y).
Between forward and backward a step keeps, of its activations, only 8-bit tensors: the norm's checkpoint of h, the
dispatched y in the column orientation (the up projection's Wgrad operand) and the checkpoint of the up/gate output, from
which the backward recomputes the hidden layer. The router is fixed here; torch does the routing, the dispatch and the
loss, the package everything else:

    forward   rmsnorm_mx_quantize -> grouped_scaled_gemm -> swiglu_mx_quantize_checkpoint -> grouped_scaled_gemm
    backward  route_weighted_mx_quantize -> grouped_scaled_gemm_strided (dgrad over the column weight cache)
              -> swiglu_backward_mx_checkpoint -> grouped_wgrad_mx, grouped_scaled_gemm_strided, grouped_wgrad_mx
              -> rmsnorm_backward_mx_checkpoint
    update    fp8_adam_step_mx_cache (rebuilds both orientations of each weight's cache)
    decode    rmsnorm_mx_quantize -> moe_mx_few_tokens
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_precision_numerics_amd as mxq  # noqa: E402

EPS = 1e-6


def dequantize(q, s):
    """bf16 values of an MXFP8 row orientation (exact)."""
    v = q.view(torch.float8_e4m3fn).float().reshape(*q.shape[:-1], -1, 32)
    return (v * torch.exp2(s.float() - 127.0)[..., None]).reshape(q.shape).to(torch.bfloat16)


class AdamWeight:
    """An expert weight [E][rows][cols]: fp32 master, FP8 Adam state, MXFP8 caches in both orientations."""

    def __init__(self, w):
        self.shape = w.shape
        self.master = w.reshape(-1).contiguous()
        n, dev = w.numel(), w.device
        self.m = torch.zeros(n, dtype=torch.uint8, device=dev)
        self.m_scale = torch.ones(1, device=dev)
        self.v = torch.zeros(n, dtype=torch.float16, device=dev)
        self.cache = mxq.mx_quantize(w.reshape(-1, w.shape[-1]).to(torch.bfloat16))
        self.step = 0

    def update(self, grad, lr):
        self.step += 1
        hp = mxq.AdamHParams(lr, 0.9, 0.95, 1e-8, 0.0, self.step)
        E, r, c = self.shape
        self.cache = mxq.fp8_adam_step_mx_cache(self.master, grad.reshape(-1), self.m, self.m_scale, self.v, None, hp, E * r, c)

    def rows(self):
        """The forward operand: codes [E][rows][cols] and scales."""
        E, r, c = self.shape
        return self.cache.q_row.view(E, r, c), self.cache.s_row.view(E, r, c // 32)


class Block:
    def __init__(self, D=256, F=128, E=8, topk=2, device="cuda:0", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.D, self.F, self.E, self.topk = D, F, E, topk
        self.gamma = 1.0 + 0.1 * n(D)
        self.router = n(D, E) / D ** 0.5
        self.up = AdamWeight(n(E, 2 * F, D) / D ** 0.5)
        self.down = AdamWeight(n(E, D, F) / F ** 0.5)

    def logits(self, norm, h):
        """Router logits of the normalized values (fp32, from the residual stream)."""
        return (h.float() * norm.rstd[:, None] * self.gamma) @ self.router

    def dispatch(self, logits):
        """Rows in expert order, each expert's padded to 32: token of each row (0 for padding), route weight (0), offsets."""
        top, who = torch.sort(logits, dim=-1, descending=True, stable=True)
        top, who = top[:, :self.topk], who[:, :self.topk]
        p = torch.softmax(top, -1)
        token, weight, offsets = [], [], [0]
        for e in range(self.E):
            t, k = torch.nonzero(who == e, as_tuple=True)
            pad = -len(t) % 32
            token.append(torch.cat([t, t.new_zeros(pad)]))
            weight.append(torch.cat([p[t, k], p.new_zeros(pad)]))
            offsets.append(offsets[-1] + len(t) + pad)
        return torch.cat(token), torch.cat(weight), torch.tensor(offsets, dtype=torch.int64, device=logits.device)

    def forward(self, x, residual):
        norm = mxq.rmsnorm_mx_quantize(x, self.gamma, EPS, residual=residual, colwise=False)
        token, weight, offs = self.dispatch(self.logits(norm, norm.sum))
        yq, ys = norm.mx.q_row[token], norm.mx.s_row[token]
        c = mxq.grouped_scaled_gemm(yq, ys, offs, *self.up.rows())
        hid, c_ck = mxq.swiglu_mx_quantize_checkpoint(c)
        o = mxq.grouped_scaled_gemm(hid.q_row, hid.s_row, offs, *self.down.rows())
        out = norm.sum.float().index_add(0, token, o.float() * weight[:, None])
        y_col = mxq.mx_quantize(dequantize(yq, ys), rowwise=False)
        return out, (norm.checkpoint, norm.rstd, y_col, c_ck, token, weight, offs)

    def backward(self, dout, saved):
        """dout: bf16 [tokens][D] -> gradients of x (and of the residual), gamma, up and down."""
        h_ck, rstd, y_col, c_ck, token, weight, offs = saved
        D, F, E = self.D, self.F, self.E
        do = mxq.route_weighted_mx_quantize(dout[token], weight)
        down, up = self.down.cache, self.up.cache
        dh = mxq.grouped_scaled_gemm_strided(do.q_row, do.s_row, offs, down.q_col, down.s_col, E, F, D, ldb=E * D,
                                             b_group_stride=D, ldbs=E * D // 32, bs_group_stride=D // 32)
        dc, hid = mxq.swiglu_backward_mx_checkpoint(c_ck, dh)
        d_down = mxq.grouped_wgrad_mx(do.q_col, do.s_col, hid.q_col, hid.s_col, offs)
        dy = mxq.grouped_scaled_gemm_strided(dc.q_row, dc.s_row, offs, up.q_col, up.s_col, E, D, 2 * F, ldb=E * 2 * F,
                                             b_group_stride=2 * F, ldbs=E * 2 * F // 32, bs_group_stride=2 * F // 32)
        d_up = mxq.grouped_wgrad_mx(dc.q_col, dc.s_col, y_col.q_col, y_col.s_col, offs)
        dy = torch.zeros(dout.shape, device=dout.device).index_add_(0, token, dy.float() * (weight > 0)[:, None])
        dx, dgamma = mxq.rmsnorm_backward_mx_checkpoint(dy.to(torch.bfloat16), h_ck, rstd, self.gamma, residual_grad=dout)
        return dx, dgamma, d_up, d_down

    def decode(self, x, residual):
        """The block on up to 64 tokens: the norm's launch and the experts' two or three."""
        norm = mxq.rmsnorm_mx_quantize(x, self.gamma, EPS, residual=residual, colwise=False, checkpoint=False)
        y = mxq.moe_mx_few_tokens(norm.mx.q_row, norm.mx.s_row, self.logits(norm, norm.sum), self.topk, *self.up.rows(),
                                  *self.down.rows())
        return norm.sum.float() + y.float()


def train(block, steps=8, tokens=256, lr=2e-3, seed=1, device="cuda:0"):
    """Fits the block to a random target; returns the losses."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    x = torch.randn((tokens, block.D), generator=g, device=device).to(torch.bfloat16)
    r = torch.randn((tokens, block.D), generator=g, device=device).to(torch.bfloat16)
    target = torch.randn((tokens, block.D), generator=g, device=device)
    losses = []
    for _ in range(steps):
        out, saved = block.forward(x, r)
        diff = out - target
        losses.append(float((diff ** 2).mean()))
        # Adam does not mind the loss's scale, but its fp16 second moment holds nothing below 6e-8: the gradient of a tenth
        # of half the squared error, not of its mean over all values
        _, dgamma, d_up, d_down = block.backward((0.1 * diff).to(torch.bfloat16), saved)
        block.gamma -= lr * dgamma.sign()
        block.up.update(d_up, lr)
        block.down.update(d_down, lr)
    return losses, (x, r)


def main():
    block = Block()
    losses, (x, r) = train(block)
    print("loss by step:", " ".join(f"{v:.4f}" for v in losses))
    out, _ = block.forward(x, r)
    for n in (1, 7):
        y = block.decode(x[:n].contiguous(), r[:n].contiguous())
        d = (y - out[:n]).norm() / out[:n].norm()
        print(f"decode of {n} token(s): {float(d):.2e} from the training forward")


if __name__ == "__main__":
    main()
