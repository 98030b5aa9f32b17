"""The routed experts of a few tokens against a plain 64-bit implementation and against the grouped path.

Two kinds of comparison. With small whole numbers as operands the first product is exact in any order, so its bf16
rounding and the MXFP8 of h are the oracle's byte for byte, and with one expert a token the output keeps the GEMM bound
2^-7 |y| + 2^-20 sum |h w|. With normal operands a different order of the fp32 sums may move a value of c to its
neighbouring bf16 (2^-8 of it) and, rarely, a code of h to its neighbour (2^-3 of one of F terms, which may be twice as
large as the typical one); so y is compared as a whole: each token's error is at most 2^-8 + 2^-2 / sqrt(F) of the token's
2-norm (bf16's own rounding is 2^-9 at most), and no value is off by more than 2^-7 |y| + 1 / sqrt(F) of the row's root
mean square (the same with a weight four deviations out)."""
import numpy as np
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
import oracle
from gpu_util import DEV, need_gpu, say, u16, u8
from mxfp8_precision_numerics_amd import workloads

pytestmark = pytest.mark.gpu


def _values(q, s):
    v = oracle.fp8_value(u8(q), oracle.E4M3).astype(np.float64)
    b = np.minimum(u8(s).astype(np.int64), 254)
    return v * np.repeat(np.ldexp(1.0, b - 127), 32, axis=-1)


def _mx(t):
    q = mxq.mx_quantize(t.reshape(-1, t.shape[-1]).contiguous(), colwise=False)
    return q.q_row.reshape(t.shape), q.s_row.reshape(*t.shape[:-1], t.shape[-1] // 32)


def _operands(T, E, D, F, k=0):
    x = _mx(workloads.normal_bf16((T, D), 1.0, 52, 10 * k, DEV))
    up = _mx(workloads.normal_bf16((E, 2 * F, D), 0.02 * (2048 / D) ** 0.5, 52, 10 * k + 1, DEV))
    down = _mx(workloads.normal_bf16((E, D, F), 0.02, 52, 10 * k + 2, DEV))
    logits = workloads.normal_f32((T, E), 1.5, 52, 10 * k + 3, DEV)
    return x, up, down, logits


def _choice(logits, k):
    """Each token's experts (largest logits, ties to the lower index; -inf never) or None for a NaN or +inf row."""
    out = []
    for row in logits:
        if np.isnan(row).any() or np.isposinf(row).any():
            out.append(None)
        else:
            out.append([e for e in np.lexsort((np.arange(row.size), -row))[:k] if row[e] > -np.inf])
    return out


def _reference(x, up, down, logits, k, normalize):
    xv = _values(*x)
    lg = logits.cpu().numpy().astype(np.float64)
    T, D, F = xv.shape[0], xv.shape[1], up[0].shape[1] // 2
    y = np.zeros((T, D))
    chosen = _choice(lg, k)
    for e in sorted({e for c in chosen if c for e in c}):
        tok = [t for t in range(T) if chosen[t] and e in chosen[t]]
        c = xv[tok] @ _values(up[0][e], up[1][e]).T
        cb = oracle.bf16_from_f32(c.astype(np.float32))
        q, s, _ = oracle.swiglu_mx_quantize(cb)
        h = oracle.fp8_value(q, oracle.E4M3) * np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), 32, axis=1)
        o = h @ _values(down[0][e], down[1][e]).T
        for i, t in enumerate(tok):
            m = max(lg[t][j] for j in chosen[t])
            over = [lg[t][j] for j in chosen[t]] if normalize else lg[t]
            y[t] += np.exp(lg[t][e] - m) / np.exp(np.asarray(over) - m).sum() * o[i]
    for t in range(T):
        if chosen[t] is None:
            y[t] = np.nan
    return y


def _near(got, want, F):
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(g), np.isnan(want))
    for t in range(want.shape[0]):
        if np.isnan(want[t]).any():
            continue
        d = np.abs(g[t] - want[t])
        rms = np.sqrt((want[t] ** 2).mean())
        assert np.linalg.norm(d) <= (2.0 ** -8 + 0.25 / F ** 0.5) * np.linalg.norm(want[t]), t
        assert np.all(d <= 2.0 ** -7 * np.abs(want[t]) + rms / F ** 0.5), t


@pytest.mark.parametrize("T,E,k,D,F,normalize", [
    (1, 64, 8, 2048, 1024, True), (1, 1, 1, 32, 32, True), (2, 8, 2, 96, 160, False), (3, 64, 8, 512, 256, True),
    (7, 64, 9, 544, 96, True), (8, 64, 8, 256, 128, False), (16, 8, 2, 1056, 224, True), (17, 5, 5, 128, 64, True),
    (33, 40, 3, 320, 416, False), (64, 16, 4, 256, 288, True), (64, 2, 1, 512, 64, True), (5, 1000, 32, 64, 32, False),
    (64, 130, 7, 64, 64, True),
])
def test_against_plain(T, E, k, D, F, normalize):
    need_gpu()
    say("few-token experts", T, E, k, D, F, normalize)
    x, up, down, logits = _operands(T, E, D, F, k)
    y = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down, normalize=normalize)
    again = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down, normalize=normalize)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    _near(y, _reference(x, up, down, logits, k, normalize), F)


@pytest.mark.parametrize("T,E", [(1, 4), (16, 4), (50, 3)])
def test_whole_numbers_keep_the_product_bound(T, E):
    """Operands of small whole numbers: c and h are exact, and y = h W_down^T within the GEMM bound (one expert a token)."""
    need_gpu()
    say("few-token experts, whole numbers", T, E)
    D, F = 96, 128
    rng = np.random.default_rng(T)
    whole = lambda *s: torch.from_numpy(rng.integers(-2, 3, s).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
    x, up, down = _mx(whole(T, D)), _mx(whole(E, 2 * F, D)), _mx(whole(E, D, F))
    logits = workloads.normal_f32((T, E), 1.0, 52, 90 + T, DEV)
    y = mxq.moe_mx_few_tokens(*x, logits, 1, *up, *down)
    torch.cuda.synchronize()
    got = y.float().cpu().numpy().astype(np.float64)
    xv = _values(*x)
    for t, c in enumerate(_choice(logits.cpu().numpy(), 1)):
        e = c[0]
        cb = oracle.bf16_from_f32((xv[t] @ _values(up[0][e], up[1][e]).T).astype(np.float32)[None])
        q, s, _ = oracle.swiglu_mx_quantize(cb)
        h = (oracle.fp8_value(q, oracle.E4M3) * np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), 32, axis=1))[0]
        w = _values(down[0][e], down[1][e])
        assert np.all(np.abs(got[t] - w @ h) <= 2.0 ** -7 * np.abs(w @ h) + 2.0 ** -20 * (np.abs(w) @ np.abs(h))), t


def test_against_the_grouped_path():
    """The same tokens through grouped_scaled_gemm, swiglu_mx_quantize and grouped_scaled_gemm on padded expert groups."""
    need_gpu()
    T, E, k, D, F = 24, 16, 4, 512, 256
    say("few-token experts against the grouped path", T, E, k, D, F)
    x, up, down, logits = _operands(T, E, D, F, 5)
    y = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down)
    chosen = _choice(logits.cpu().numpy(), k)
    off, rows, who = [0], [], []
    for e in range(E):
        tok = [t for t in range(T) if e in chosen[t]]
        rows += tok + [-1] * (-len(tok) % 32)
        who += [e] * (len(rows) - off[-1])
        off.append(len(rows))
    idx = torch.tensor([max(t, 0) for t in rows], device=DEV)
    offs = torch.tensor(off, dtype=torch.int64, device=DEV)
    c = mxq.grouped_scaled_gemm(x[0][idx].contiguous(), x[1][idx].contiguous(), offs, *up)
    h = mxq.swiglu_mx_quantize(c)
    o = mxq.grouped_scaled_gemm(h.q_row, h.s_row, offs, *down)
    torch.cuda.synchronize()
    of, lg = o.float().cpu().numpy().astype(np.float64), logits.cpu().numpy().astype(np.float64)
    want = np.zeros((T, D))
    for r, (t, e) in enumerate(zip(rows, who)):
        if t >= 0:
            l = lg[t][chosen[t]]
            want[t] += np.exp(lg[t][e] - l.max()) / np.exp(l - l.max()).sum() * of[r]
    g = y.float().cpu().numpy().astype(np.float64)
    # each side rounds: the grouped path every expert's output to bf16 (2^-9 of it), this one the sum; and a moved code
    for t in range(T):
        assert np.linalg.norm(g[t] - want[t]) <= (2.0 ** -7 + 0.25 / F ** 0.5) * np.linalg.norm(want[t])


@pytest.mark.parametrize("T,E,k", [(3, 64, 8), (20, 16, 4)])
def test_masked_tied_and_refused_logits(T, E, k):
    """Masks that leave fewer than k experts or none, equal logits, one hot expert for all, a NaN and a +inf logit."""
    need_gpu()
    say("few-token experts, masks", T, E, k)
    D, F = 160, 96
    x, up, down, _ = _operands(T, E, D, F, 6)
    inf = float("inf")
    for kind in ("masked", "empty row", "ties", "one expert", "nan", "inf", "lowest"):
        logits = workloads.normal_f32((T, E), 1.5, 52, 77, DEV)
        if kind == "masked":
            logits[0] = -inf
            logits[0, E - 1] = 0.5
            logits[1, : E - 3] = -inf
        elif kind == "empty row":
            logits[0] = -inf
            logits[T - 1] = -inf
        elif kind == "ties":
            logits[:] = 1.0
            logits[1, ::2] = 2.0
        elif kind == "one expert":
            logits[:, 5] = 30.0
        elif kind == "nan":
            logits[1, E // 2] = float("nan")
        elif kind == "inf":
            logits[2, 0] = inf
        else:
            logits[0] = torch.finfo(torch.float32).min
            logits[1, 1:] = torch.finfo(torch.float32).min
        y = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down)
        torch.cuda.synchronize()
        want = _reference(x, up, down, logits, k, True)
        _near(y, want, F)
        if kind == "empty row":
            assert bool((y[0] == 0).all()) and bool((y[T - 1] == 0).all())


def test_graph_and_side_stream():
    """Captured in a graph and replayed on new inputs, with eager work between the replays; and on a side stream."""
    need_gpu()
    T, E, k, D, F = 4, 64, 8, 256, 128
    say("few-token experts, graph")
    x, up, down, logits = _operands(T, E, D, F, 7)
    ws = torch.empty(mxq.moe_few_tokens_workspace_bytes(T, E, k, D, F), dtype=torch.uint8, device=DEV)
    out = torch.empty((T, D), dtype=torch.bfloat16, device=DEV)
    mxq.moe_mx_few_tokens(*x, logits, k, *up, *down, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxq.moe_mx_few_tokens(*x, logits, k, *up, *down, out=out, workspace=ws)
    for rep in range(3):
        logits.copy_(workloads.normal_f32((T, E), 1.5, 52, 200 + rep, DEV))
        ws.fill_(0xA5 if rep else 0x5A)                          # the workspace needs no particular contents
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), rep
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down)
    side.synchronize()
    assert torch.equal(y.view(torch.int16), eager.view(torch.int16))


@pytest.mark.parametrize("T,E,k,D,F", [
    (2, 8, 2, 4128, 64), (1, 6, 3, 4096, 2112), (16, 24, 3, 4128, 64), (20, 24, 2, 64, 2208), (5, 40, 4, 2304, 2080),
    (40, 20, 2, 4096, 96), (9, 32, 3, 6176, 4256),
])
def test_long_contractions(T, E, k, D, F):
    """Contractions past the 2048 values that a workgroup or a wave has in hand at once, whole and with a rest."""
    need_gpu()
    say("few-token experts, long contractions", T, E, k, D, F)
    x, up, down, logits = _operands(T, E, D, F, 11)
    y = mxq.moe_mx_few_tokens(*x, logits, k, *up, *down)
    torch.cuda.synchronize()
    _near(y, _reference(x, up, down, logits, k, True), F)


def test_weights_past_2_31_bytes():
    """Expert weights of 2.2e9 bytes: tokens sent to the last expert."""
    need_gpu()
    E, D, F = 520, 2048, 1024
    say("few-token experts, weights past 2^31 bytes")
    up_q = torch.zeros((E, 2 * F, D), dtype=torch.uint8, device=DEV)
    up_s = torch.full((E, 2 * F, D // 32), 127, dtype=torch.uint8, device=DEV)
    down_q = torch.zeros((E, D, F), dtype=torch.uint8, device=DEV)
    down_s = torch.full((E, D, F // 32), 127, dtype=torch.uint8, device=DEV)
    x, up, down, logits = _operands(2, 1, D, F, 8)
    up_q[E - 1], up_s[E - 1], down_q[E - 1], down_s[E - 1] = up[0][0], up[1][0], down[0][0], down[1][0]
    logits = torch.full((2, E), -5.0, device=DEV)
    logits[:, E - 1] = 1.0
    y = mxq.moe_mx_few_tokens(*x, logits, 1, up_q, up_s, down_q, down_s)
    torch.cuda.synchronize()
    _near(y, _reference(x, up, down, torch.ones((2, 1)), 1, True), F)
    del up_q, down_q
    torch.cuda.empty_cache()
