"""Cases of the 8-bit integer products and of the head norms with rotary positions: quantization of each token to int8,
the product of int8 operands with a scale for each token and each output channel, the same over ragged expert groups,
and RMSNorm of every query and key head with the rotation by position in the same pass, forward and backward.

Each operator has a plain form (elementary torch operations in 32 bits) and the call a user makes of this package
(`own`).
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6


def listed():
    return [
        # one new token in front of a projection of the served model of width 2048: launch latency
        dict(name="quant_1x2048", op="quant", rows=1, cols=2048),
        # the activations of one training or prompt step, 16384 tokens
        dict(name="quant_16384x8192", op="quant", rows=16384, cols=8192),
        # QKV projection of one token of the width-2048 model
        dict(name="gemm_1x6144x2048", op="gemm", M=1, N=6144, K=2048, swiglu=False),
        # QKV projection of the dense 12288-wide model for an odd batch of decoding sequences
        dict(name="gemm_61x36864x12288", op="gemm", M=61, N=36864, K=12288, swiglu=False),
        # the same projection over a prompt of 4096 tokens
        dict(name="gemm_4096x36864x12288", op="gemm", M=4096, N=36864, K=12288, swiglu=False),
        # experts' gate/up projection with its SwiGLU for a decoding batch of 16 tokens, 8 of 64 experts each
        dict(name="grouped_up_16_tokens", op="grouped", tokens=16, experts=64, topk=8, N=2048, K=2048, swiglu=True),
        # gate/up and down projections of the 16384-token, 64-expert, top-8 workload
        dict(name="grouped_up_16384_tokens", op="grouped", tokens=16384, experts=64, topk=8, N=2048, K=2048, swiglu=True),
        dict(name="grouped_down_16384_tokens", op="grouped", tokens=16384, experts=64, topk=8, N=2048, K=1024, swiglu=False),
        # queries and keys of one new token of the width-2048 model (16 heads of 128)
        dict(name="qk_fwd_1x16", op="qk_fwd", tokens=1, hq=16, hk=16, dim=128, rot=128, axes=1, interleaved=False,
             norm=True),
        # queries and keys of the dense model (96 heads of 128), 4096 tokens
        dict(name="qk_fwd_4096x96", op="qk_fwd", tokens=4096, hq=96, hk=96, dim=128, rot=128, axes=1, interleaved=False,
             norm=True),
        # backward of a short odd batch of video tokens (time, height, width), shared key heads
        dict(name="qk_bwd_333x16", op="qk_bwd", tokens=333, hq=16, hk=4, dim=128, rot=128, axes=3, interleaved=False,
             norm=True),
        # backward of the dense model's queries and keys
        dict(name="qk_bwd_4096x96", op="qk_bwd", tokens=4096, hq=96, hk=96, dim=128, rot=128, axes=1, interleaved=False,
             norm=True),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    hi = max(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "grouped", "grouped", "qk_fwd", "qk_bwd"])
    if op == "quant":
        cols = 32 * _spread(rng, 8, 384)
        return dict(op=op, rows=_spread(rng, 1, min(16384, 134_000_000 // cols)), cols=cols)
    if op == "gemm":
        K = 32 * _spread(rng, 8, 384)
        swiglu = rng.random() < 0.3
        N = 2 * _spread(rng, 32, 18432) if swiglu else _spread(rng, 64, 36864)
        return dict(op=op, M=_spread(rng, 1, min(16384, 1_800_000_000_000 // (N * K))), N=N, K=K, swiglu=swiglu)
    if op == "grouped":
        E = rng.choice([8, 16, 40, 64])
        swiglu = rng.random() < 0.5
        N, K = 2 * _spread(rng, 128, 1024), 32 * _spread(rng, 8, 64)
        return dict(op=op, tokens=_spread(rng, 1, 16384), experts=E, topk=rng.choice([1, 2, 5, 8]), N=N, K=K,
                    swiglu=swiglu)
    dim = rng.choice([64, 96, 128, 192, 256])
    hk = _spread(rng, 1, 32)
    hq = hk * rng.choice([1, 1, 2, 4, 7])
    return dict(op=op, tokens=_spread(rng, 1, min(16384, 100_000_000 // ((hq + hk) * dim))), hq=hq, hk=hk, dim=dim,
                rot=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 1, 3]), interleaved=rng.random() < 0.3,
                norm=rng.random() < 0.8)


# ------------------------------------------------------------------------------------------ inputs
def _int8_rows(w):
    """float32 [..., n] -> int8 codes and one float32 scale for each row."""
    s = w.abs().amax(-1) / 127.0
    return torch.round(w / s[..., None]).clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def activations(rows, cols):
        # a few channels far larger than the rest
        channel = 1.0 + 9.0 * (torch.rand(cols, generator=g, device=DEV) < 0.002)
        return normal(rows, cols) * channel

    op = case["op"]
    st = dict(case)
    if op == "quant":
        st.update(x=activations(case["rows"], case["cols"]).to(torch.bfloat16))
    elif op == "gemm":
        a_q, a_s = _int8_rows(activations(case["M"], case["K"]))
        b_q, b_s = _int8_rows(0.02 * normal(case["N"], case["K"]))
        st.update(a_q=a_q, a_s=a_s, b_q=b_q, b_s=b_s)
    elif op == "grouped":
        T, E, N, K = (case[k] for k in ("tokens", "experts", "N", "K"))
        # some experts are asked for more than others; a token's chosen experts are distinct
        logits = normal(T, E) - 0.2 * torch.log(1.0 + torch.arange(E, device=DEV, dtype=torch.float32))
        chosen = torch.topk(logits, case["topk"], dim=-1).indices
        counts = torch.bincount(chosen.reshape(-1), minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
        offsets[1:] = torch.cumsum(counts, 0)
        a_q, a_s = _int8_rows(activations(T * case["topk"], K))
        b_q, b_s = _int8_rows(0.02 * normal(E, N, K))
        st.update(a_q=a_q, a_s=a_s, b_q=b_q, b_s=b_s, offsets=offsets, most=int(counts.max()))
    else:
        T, hq, hk, dim, rot = (case[k] for k in ("tokens", "hq", "hk", "dim", "rot"))
        pairs = rot // 2
        qkv = (normal(T, (hq + 2 * hk) * dim) * 1.5).to(torch.bfloat16)
        inv = 1.0 / (1e6 ** (torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs))
        start = int(torch.randint(0, 1_000_000, (1,), generator=g, device=DEV))
        i = torch.arange(T, device=DEV, dtype=torch.int64)
        if case["axes"] == 1:
            positions, axis = (start + i)[None], [0] * pairs
        else:                                    # frames of 12 x 20 patches; a quarter of the pairs turn with the time
            positions = torch.stack([start + i // 240, start + i // 20 % 12, start + i % 20])
            t = pairs // 4
            h = (pairs - t) // 2
            axis = [0] * t + [1] * h + [2] * (pairs - t - h)
        st.update(qkv=qkv, positions=positions.contiguous(), inv_freq=inv.to(torch.float32), pair_axis=tuple(axis),
                  axis=torch.tensor(axis, device=DEV),
                  gamma_q=1.0 + 0.2 * normal(dim) if case["norm"] else None,
                  gamma_k=1.0 + 0.2 * normal(dim) if case["norm"] else None)
        if op == "qk_bwd":
            st.update(dq=(1e-3 * normal(T, hq, dim)).to(torch.bfloat16), dk=(1e-3 * normal(T, hk, dim)).to(torch.bfloat16))
    return st


# ------------------------------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_quant(st):
    x = st["x"].to(torch.float32)
    amax = x.abs().amax(-1, keepdim=True)
    # 127 x is exact in 32 bits; the quotient of whole bf16 significands is never so near a half that its rounding counts
    q = torch.round(x * 127.0 / amax.clamp(min=1e-30))
    return dict(q=q.to(torch.int8), scale=(amax / 127.0)[:, 0])


def _own_quant(st):
    import mxfp8_precision_numerics_amd as mxq
    r = mxq.int8_quantize_tokens(st["x"])
    return dict(q=r.q, scale=r.scale)


def _silu_mul(c):
    gate, up = c.chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_gemm(st):
    c = torch.matmul(st["a_q"].to(torch.float32), st["b_q"].to(torch.float32).t())
    c = c * st["a_s"][:, None] * st["b_s"]
    return (_silu_mul(c) if st["swiglu"] else c).to(torch.bfloat16)


def _own_gemm(st):
    import mxfp8_precision_numerics_amd as mxq
    return mxq.int8_scaled_gemm(st["a_q"], st["a_s"], st["b_q"], st["b_s"], swiglu=st["swiglu"])


def _plain_grouped(st):
    # every expert's rows padded to the longest expert's, one batched product, the rows gathered back
    off, total = st["offsets"], st["a_q"].shape[0]
    at = off[:-1, None] + torch.arange(st["most"], device=off.device)
    at = at.clamp(max=total - 1)
    c = torch.bmm(st["a_q"][at].to(torch.float32), st["b_q"].to(torch.float32).transpose(1, 2))
    row = torch.arange(total, device=off.device)
    e = torch.searchsorted(off[1:].contiguous(), row, right=True)
    c = c[e, row - off[e]] * st["a_s"][:, None] * st["b_s"][e]
    return (_silu_mul(c) if st["swiglu"] else c).to(torch.bfloat16)


def _own_grouped(st):
    import mxfp8_precision_numerics_amd as mxq
    return mxq.int8_grouped_gemm(st["a_q"], st["a_s"], st["offsets"], st["b_q"], st["b_s"], swiglu=st["swiglu"])


def _angles(st):
    """cos and sin [tokens][1][pairs]; the angles in 64 bits, as positions go far."""
    a = st["positions"][st["axis"]].t().to(torch.float64) * st["inv_freq"].to(torch.float64)
    return torch.cos(a).to(torch.float32)[:, None], torch.sin(a).to(torch.float32)[:, None]


def _turn(y, cos, sin, rot, interleaved):
    """y [tokens][heads][dim] with its first `rot` values turned pair by pair."""
    if interleaved:
        a, b = y[..., :rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1) if rot < y.shape[-1] else turned


def _heads(st):
    T, hq, hk, dim = st["tokens"], st["hq"], st["hk"], st["dim"]
    x = st["qkv"]
    return (x[:, :hq * dim].reshape(T, hq, dim).to(torch.float32),
            x[:, hq * dim:(hq + hk) * dim].reshape(T, hk, dim).to(torch.float32))


def _plain_qk_fwd(st):
    cos, sin = _angles(st)

    def one(x, gamma):
        if gamma is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma
        return _turn(x, cos, sin, st["rot"], st["interleaved"]).to(torch.bfloat16)

    q, k = _heads(st)
    return dict(q=one(q, st["gamma_q"]), k=one(k, st["gamma_k"]))


def _own_qk_fwd(st):
    import mxfp8_precision_numerics_amd as mxq
    q, k = mxq.qk_norm_rope(st["qkv"], st["hq"], st["hk"], st["dim"], st["positions"], st["inv_freq"], st["gamma_q"],
                            st["gamma_k"], EPS, pair_axis=st["pair_axis"], interleaved=st["interleaved"])
    return dict(q=q, k=k)


def _plain_qk_bwd(st):
    cos, sin = _angles(st)

    def one(x, dy, gamma):
        d = _turn(dy.to(torch.float32), cos, -sin, st["rot"], st["interleaved"])
        if gamma is None:
            return d.flatten(1).to(torch.bfloat16), None
        rstd = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
        xh = x * rstd
        t = d * gamma
        dx = rstd * (t - xh * (t * xh).mean(-1, keepdim=True))
        return dx.flatten(1).to(torch.bfloat16), (d * xh).sum((0, 1))

    q, k = _heads(st)
    dq, gq = one(q, st["dq"], st["gamma_q"])
    dk, gk = one(k, st["dk"], st["gamma_k"])
    return dict(dqk=torch.cat([dq, dk], -1), dgamma_q=gq, dgamma_k=gk)


def _own_qk_bwd(st):
    import mxfp8_precision_numerics_amd as mxq
    r = mxq.qk_norm_rope_backward(st["dq"], st["dk"], st["qkv"], st["positions"], st["inv_freq"], st["gamma_q"],
                                  st["gamma_k"], EPS, pair_axis=st["pair_axis"], interleaved=st["interleaved"])
    return dict(dqk=r.dqk, dgamma_q=r.dgamma_q, dgamma_k=r.dgamma_k)


_plain = dict(quant=_plain_quant, gemm=_plain_gemm, grouped=_plain_grouped, qk_fwd=_plain_qk_fwd, qk_bwd=_plain_qk_bwd)
_own = dict(quant=_own_quant, gemm=_own_gemm, grouped=_own_grouped, qk_fwd=_own_qk_fwd, qk_bwd=_own_qk_bwd)


# ------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["cols"]
        return dict(bytes=3.0 * n + 4 * case["rows"], flops=3.0 * n)                  # x; codes and scales
    if op in ("gemm", "grouped"):
        N, K = case["N"], case["K"]
        rows = case["M"] if op == "gemm" else case["tokens"] * case["topk"]
        # experts that some token picks, were all equally likely
        used = 1 if op == "gemm" else case["experts"] * (1.0 - (1.0 - case["topk"] / case["experts"]) ** case["tokens"])
        out = N // 2 if case["swiglu"] else N
        return dict(bytes=rows * (K + 4 + 2.0 * out) + used * N * (K + 4.0), flops=2.0 * rows * N * K)
    n = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
    small = 8.0 * case["tokens"] * case["axes"] + 2 * case["rot"]
    if op == "qk_fwd":
        return dict(bytes=4.0 * n + small, flops=8.0 * n)                             # x; y
    return dict(bytes=6.0 * n + small, flops=16.0 * n)                                # x, dy; dx


# ------------------------------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op == "quant":
        x = st["x"].to(d)
        most = x.abs().max(dim=1).values
        code = 127.0 * x / torch.where(most == 0.0, torch.ones_like(most), most).unsqueeze(1)
        return dict(q=torch.round(code).to(torch.int8), scale=most / 127.0)
    if op == "gemm":
        c = (st["a_q"].to(d) @ st["b_q"].to(d).t()) * torch.outer(st["a_s"].to(d), st["b_s"].to(d))
        if not case["swiglu"]:
            return c
        F = case["N"] // 2
        return c[:, :F] * torch.sigmoid(c[:, :F]) * c[:, F:]
    if op == "grouped":
        off = st["offsets"].tolist()
        parts = []
        for e in range(case["experts"]):
            lo, hi = off[e], off[e + 1]
            if lo < hi:
                c = (st["a_q"][lo:hi].to(d) @ st["b_q"][e].to(d).t()) * torch.outer(st["a_s"][lo:hi].to(d), st["b_s"][e].to(d))
                F = case["N"] // 2
                parts.append(c[:, :F] * torch.sigmoid(c[:, :F]) * c[:, F:] if case["swiglu"] else c)
        return torch.cat(parts)
    T, hq, hk, dim, rot = (case[k] for k in ("tokens", "hq", "hk", "dim", "rot"))
    pairs = rot // 2
    # the pair's rotation as a complex factor
    first = torch.arange(pairs, device=DEV) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else pairs)
    where = st["positions"].to(d)
    angle = torch.stack([where[a] * float(f) for a, f in zip(st["pair_axis"], st["inv_freq"].tolist())], 1)
    factor = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    x = st["qkv"].to(d)

    def turned(y, f):
        z = torch.complex(y[..., first], y[..., second]) * f
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {}
    for name, lo, heads, gamma in (("q", 0, hq, st["gamma_q"]), ("k", hq, hk, st["gamma_k"])):
        h = x[:, lo * dim:(lo + heads) * dim].reshape(T, heads, dim)
        r = torch.ones((T, heads, 1), dtype=d, device=DEV) if gamma is None else \
            (h.pow(2).sum(-1, keepdim=True) / dim + EPS).pow(-0.5)
        w = torch.ones(dim, dtype=d, device=DEV) if gamma is None else gamma.to(d)
        if op == "qk_fwd":
            out[name] = turned(h * r * w, factor)
            continue
        back = turned(st["d" + name].to(d), factor.conj())
        gx = back * w * r
        if gamma is not None:
            gx = gx - h * r.pow(3) * ((back * w * h).sum(-1, keepdim=True) / dim)
        out["dx" + name] = gx.reshape(T, heads * dim)
        out["dgamma_" + name] = None if gamma is None else torch.einsum("thd,thd,tho->d", back, h, r)
    if op == "qk_fwd":
        return out
    return dict(dqk=torch.cat([out["dxq"], out["dxk"]], 1), dgamma_q=out["dgamma_q"], dgamma_k=out["dgamma_k"])
