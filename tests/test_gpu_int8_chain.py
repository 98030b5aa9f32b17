"""The int8 operators and the head norms together, as a decoder layer and a routed block use them: eager, captured into a
graph and replayed, on a stream of its own, and next to the MXFP8 path that trains on the same gradients."""
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
from gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu
D, HQ, HK, DIM, F, E, TOPK = 256, 4, 2, 64, 128, 6, 2


def _weights(g):
    n = lambda *s: (torch.randn(*s, generator=g, device=DEV) * 0.06).bfloat16()  # noqa: E731
    q = lambda w: mxq.int8_quantize_tokens(w)  # noqa: E731
    w = dict(qkv=q(n((HQ + 2 * HK) * DIM, D)), o=q(n(D, HQ * DIM)))
    up, down = q(n(E * 2 * F, D)), q(n(E * D, F))
    w["up"] = (up.q.view(E, 2 * F, D), up.scale.view(E, 2 * F))
    w["down"] = (down.q.view(E, D, F), down.scale.view(E, D))
    w["gq"], w["gk"] = 1 + 0.1 * torch.randn(DIM, generator=g, device=DEV), 1 + 0.1 * torch.randn(DIM, generator=g, device=DEV)
    w["inv"] = (1e4 ** (-torch.arange(DIM // 2, device=DEV) / (DIM // 2))).float()
    return w


def _layer(w, x, pos, rows, offsets):
    """QKV projection, head norms and rotation, then the experts on the routed rows (a gather of the quantized tokens)."""
    a = mxq.int8_quantize_tokens(x)
    qkv = mxq.int8_scaled_gemm(a.q, a.scale, w["qkv"].q, w["qkv"].scale)
    q, k = mxq.qk_norm_rope(qkv, HQ, HK, DIM, pos, w["inv"], w["gq"], w["gk"])
    h = mxq.int8_grouped_gemm(a.q[rows], a.scale[rows], offsets, *w["up"], swiglu=True)
    hq = mxq.int8_quantize_tokens(h)
    y = mxq.int8_grouped_gemm(hq.q, hq.scale, offsets, *w["down"])
    return q, k, y


def _inputs(g, T):
    x = torch.randn(T, D, generator=g, device=DEV).bfloat16()
    pos = torch.arange(T, device=DEV) + 1000
    pick = torch.topk(torch.randn(T, E, generator=g, device=DEV), TOPK).indices.reshape(-1)
    order = torch.argsort(pick, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(torch.bincount(pick, minlength=E), 0)
    return x, pos, order // TOPK, offsets


def _expected(w, x, pos, rows, off):
    """The layer in 64 bits from the same codes: quantization is recomputed from the definition."""
    def quant(v):
        m = v.double().abs().amax(1, keepdim=True)
        return torch.round(127.0 * v.double() / m) * (m / 127.0)
    deq = lambda t: t[0].double() * t[1].double()[..., None]  # noqa: E731
    a = quant(x)
    qkv = a @ deq((w["qkv"].q, w["qkv"].scale)).t()
    import qk_reference as ref
    q, k = ref.forward(qkv, HQ, HK, DIM, pos, w["inv"], w["gq"], w["gk"], 1e-6)
    up, down, r = deq(w["up"]), deq(w["down"]), a[rows]
    y = torch.zeros(len(rows), D, dtype=torch.float64, device=DEV)
    o = off.tolist()
    for e in range(E):
        c = r[o[e]:o[e + 1]] @ up[e].t()
        h = c[:, :F] / (1 + torch.exp(-c[:, :F])) * c[:, F:]
        if len(h):
            y[o[e]:o[e + 1]] = quant(h) @ down[e].t()
    return q, k, y


@pytest.mark.parametrize("T", [1, 5, 40, 700])
def test_layer(T):
    need_gpu()
    g = torch.Generator(device=DEV).manual_seed(T)
    w = _weights(g)
    args = _inputs(g, T)
    say("layer", T)
    q, k, y = _layer(w, *args)
    eq, ek, ey = _expected(w, *args)
    # q, k: two roundings to bf16, 2^-8 each, of values of unit scale; y: h's rounding to bf16 (2^-8) may also move a code
    # by one, 1/127 of the row's largest: independent over the F terms, so in the 2-norm below 2^-8 + 2^-8 + 1/127
    for got, want, bound in ((q, eq, 2.0 ** -7), (k, ek, 2.0 ** -7), (y, ey, 2.0 ** -7 + 1 / 127)):
        assert float((got.double() - want).norm() / want.norm()) <= bound


@pytest.mark.parametrize("T", [1, 40, 700])
def test_captured_and_replayed(T):
    """Two graphs on the same inputs, replayed in turn with eager work between, against the eager result every time; then
    new inputs in the same buffers."""
    need_gpu()
    g = torch.Generator(device=DEV).manual_seed(T + 100)
    w = _weights(g)
    args = _inputs(g, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _layer(w, *args)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = _layer(w, *args)
        graphs.append((gr, out))
    for turn in range(3):
        want = [t.clone() for t in _layer(w, *args)]
        for gr, out in graphs:
            for t in out:
                t.zero_()
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        for t, n in zip(args, _inputs(g, T)):
            t.copy_(n)


def test_backward_captured_and_replayed():
    need_gpu()
    g = torch.Generator(device=DEV).manual_seed(9)
    T = 300
    qkv = torch.randn(T, (HQ + HK) * DIM, generator=g, device=DEV).bfloat16()
    dq, dk = torch.randn(T, HQ, DIM, generator=g, device=DEV).bfloat16(), torch.randn(T, HK, DIM, generator=g, device=DEV).bfloat16()
    w = _weights(g)
    pos = torch.arange(T, device=DEV)
    run = lambda: mxq.qk_norm_rope_backward(dq, dk, qkv, pos, w["inv"], w["gq"], w["gk"])  # noqa: E731
    run()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = run()
    for _ in range(3):
        want = run()
        for t in out:
            t.fill_(5.0)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        dq.copy_(torch.randn(dq.shape, generator=g, device=DEV))


def test_on_another_stream_and_into_the_training_path():
    """The calls go to the current stream; the gradient rows they write are what the MXFP8 projection's backward takes."""
    need_gpu()
    g = torch.Generator(device=DEV).manual_seed(4)
    T = 64
    w = _weights(g)
    args = _inputs(g, T)
    want = _layer(w, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _layer(w, *args)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    qkv = torch.randn(T, (HQ + 2 * HK) * DIM, generator=g, device=DEV).bfloat16()
    dqkv = torch.randn(T, (HQ + 2 * HK) * DIM, generator=g, device=DEV).bfloat16()      # values' gradient in its place
    dv = dqkv[:, (HQ + HK) * DIM:].clone()
    dq, dk = torch.randn(T, HQ, DIM, generator=g, device=DEV).bfloat16(), torch.randn(T, HK, DIM, generator=g, device=DEV).bfloat16()
    r = mxq.qk_norm_rope_backward(dq, dk, qkv, args[1], w["inv"], w["gq"], w["gk"], out=dqkv)
    assert torch.equal(dqkv[:, (HQ + HK) * DIM:], dv)
    mx = mxq.mx_quantize(r.dqk)                                            # the projection's dgrad and Wgrad operand
    back = mx.q_row.view(torch.float8_e4m3fn).float().view(T, -1, 32) * torch.exp2(mx.s_row.float() - 127)[..., None]
    assert float((back.view(T, -1) - dqkv.float()).norm() / dqkv.float().norm()) < 2.0 ** -4


@pytest.mark.parametrize("swiglu", [False, True])
def test_large_products_side_by_side_and_replayed(swiglu):
    """Products whose workgroups hold whole CUs, on two streams at once and from two graphs of the same buffers: the same
    bytes as alone (the sums are exact)."""
    need_gpu()
    g = torch.Generator(device=DEV).manual_seed(5)
    M, N, K, G = 2300, 8200, 416, 9
    c = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)  # noqa: E731
    sc = lambda *s: torch.rand(s, generator=g, device=DEV) * 1e-4 + 1e-6  # noqa: E731
    a, sa, b, sb = c(M, K), sc(M), c(G, N, K), sc(G, N)
    off = torch.tensor([0, 0, 300, 301, 900, 1400, 1656, 2000, 2000, M], device=DEV)
    dense = lambda: mxq.int8_scaled_gemm(a, sa, b[1], sb[1], swiglu=swiglu)  # noqa: E731
    routed = lambda: mxq.int8_grouped_gemm(a, sa, off, b, sb, swiglu=swiglu)  # noqa: E731
    say("large products side by side", swiglu)
    want_d, want_r = dense(), routed()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        with torch.cuda.stream(s1):
            got.append((dense(), want_d))
        with torch.cuda.stream(s2):
            got.append((routed(), want_r))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)
    graphs = []
    for f in (dense, routed):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f()
        graphs.append((graph, out, f))
    for _ in range(3):
        a.copy_(c(M, K))
        for graph, out, f in graphs:
            graph.replay()
            assert torch.equal(out, f())
