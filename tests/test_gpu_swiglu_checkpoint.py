"""SwiGLU with an 8-bit checkpoint and its backward, against the CPU oracle byte for byte: the forward's h is
swiglu_mx_quantize's, the checkpoint is the oracle's quantize of c, and the backward is the oracle's backward on the
values the checkpoint stands for (bf16 holds them exactly)."""
import numpy as np
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
import oracle
from gpu_util import DEV, need_gpu, say, u16, u8
from mxfp8_precision_numerics_amd import workloads

pytestmark = pytest.mark.gpu


def _same_codes(got, want):
    got, want = u8(got), np.asarray(want)
    nan = (want & 0x7F) == 0x7F
    return np.array_equal((got & 0x7F) == 0x7F, nan) and np.array_equal(got[~nan], want[~nan])


def _values(q, s):
    v = oracle.fp8_value(u8(q), oracle.E4M3).astype(np.float64)
    b = u8(s).astype(np.int64)
    return v * np.repeat(np.where(b == 255, np.nan, np.ldexp(1.0, b - 127)), 32, axis=1)


@pytest.mark.parametrize("rows,F,std,rule", [(1, 32, 1.0, mxq.RCEIL), (37, 96, 10.0, mxq.RCEIL), (5, 1440, 2.0, mxq.FLOOR),
                                             (1000, 1024, 1.5, mxq.RCEIL), (33, 4128, 45.0, mxq.RCEIL),
                                             (16500, 256, 1.5, mxq.RCEIL)])
def test_forward(rows, F, std, rule):
    need_gpu()
    say("swiglu checkpoint forward", rows, F, std, rule)
    c = workloads.normal_bf16((rows, 2 * F), std, 51, 1, DEV)
    h, ck = mxq.swiglu_mx_quantize_checkpoint(c, rule)
    ref = mxq.swiglu_mx_quantize(c, rule)
    torch.cuda.synchronize()
    q, s, _ = oracle.swiglu_mx_quantize(u16(c), rule)
    assert np.array_equal(u8(h.s_row), s) and np.array_equal(u8(h.q_row), q)
    assert torch.equal(h.q_row, ref.q_row) and torch.equal(h.s_row, ref.s_row)
    o = oracle.mx_quantize(u16(c), rule, colwise=False)
    assert np.array_equal(u8(ck.q_row), o[0]) and np.array_equal(u8(ck.s_row), o[1])


def test_forward_extremes():
    need_gpu()
    say("swiglu checkpoint extremes")
    vals = np.array([0.0, -0.0, 1e-30, -1e-30, 88.0, -104.5, 200.0, 3.0e38, -3.0e38, np.inf, -np.inf, 1.0, np.nan], np.float32)
    c = oracle.bf16_from_f32(np.resize(vals, (16, 256)).astype(np.float32))
    t = torch.from_numpy(c.view(np.int16)).view(torch.bfloat16).to(DEV)
    h, ck = mxq.swiglu_mx_quantize_checkpoint(t)
    torch.cuda.synchronize()
    q, s, _ = oracle.swiglu_mx_quantize(c)
    o = oracle.mx_quantize(c, colwise=False)
    assert np.array_equal(u8(h.s_row), s) and _same_codes(h.q_row, q)
    assert np.array_equal(u8(ck.s_row), o[1]) and _same_codes(ck.q_row, o[0])


@pytest.mark.parametrize("rows,F,rule,row,col,hid", [
    (32, 32, mxq.RCEIL, True, True, True), (96, 160, mxq.RCEIL, True, True, True), (416, 1440, mxq.RCEIL, True, True, True),
    (64, 128, mxq.FLOOR, True, True, True), (7, 96, mxq.RCEIL, True, False, False), (160, 1024, mxq.RCEIL, False, True, False),
    (160, 1056, mxq.RCEIL, False, False, True), (224, 4096, mxq.RCEIL, True, False, True), (2080, 256, mxq.RCEIL, True, True, True),
])
def test_backward(rows, F, rule, row, col, hid):
    need_gpu()
    say("swiglu checkpoint backward", rows, F, rule, row, col, hid)
    c = workloads.normal_bf16((rows, 2 * F), 1.5, 51, 2, DEV)
    dh = workloads.normal_bf16((rows, F), 1e-3, 51, 3, DEV)
    ck = mxq.mx_quantize(c, colwise=False)
    dc, h = mxq.swiglu_backward_mx_checkpoint(ck, dh, rowwise=row, colwise=col, hidden=hid, rule=rule)
    torch.cuda.synchronize()
    ch = _values(ck.q_row, ck.s_row).astype(np.float32)
    cb = oracle.bf16_from_f32(ch)
    assert np.array_equal(oracle.bf16_to_f32(cb), ch)
    o = oracle.swiglu_bwd_mx_quantize(cb, u16(dh), rule, row, col)
    for got, want in zip(dc, o[:4]):
        assert (got is None) == (want is None)
        assert got is None or np.array_equal(u8(got), want)
    if hid:
        _, _, hf = oracle.swiglu_mx_quantize(cb, rule, want_h=True)
        w = oracle.mx_quantize_f32(hf, rule, False, True)
        assert np.array_equal(u8(h.q_col), w[2]) and np.array_equal(u8(h.s_col), w[3])
    else:
        assert h is None


@pytest.mark.parametrize("std,rule", [(1.5, mxq.RCEIL), (1e-4, mxq.FLOOR)])
def test_backward_many_tiles(std, rule):
    """Enough tiles for groups of four down a column, the last group and the last tile across being partial; with small
    values no block's scale is in the kernel's table."""
    need_gpu()
    rows, F = 8224, 1056
    say("swiglu checkpoint backward, many tiles", rows, F, std, rule)
    ck = mxq.mx_quantize(workloads.normal_bf16((rows, 2 * F), std, 51, 8, DEV), colwise=False)
    dh = workloads.normal_bf16((rows, F), 1e-3, 51, 9, DEV)
    dc, h = mxq.swiglu_backward_mx_checkpoint(ck, dh, rule=rule)
    torch.cuda.synchronize()
    cb = oracle.bf16_from_f32(_values(ck.q_row, ck.s_row).astype(np.float32))
    o = oracle.swiglu_bwd_mx_quantize(cb, u16(dh), rule, True, True)
    assert all(np.array_equal(u8(got), want) for got, want in zip(dc, o[:4]))
    _, _, hf = oracle.swiglu_mx_quantize(cb, rule, want_h=True)
    w = oracle.mx_quantize_f32(hf, rule, False, True)
    assert np.array_equal(u8(h.q_col), w[2]) and np.array_equal(u8(h.s_col), w[3])


def test_backward_nan_block():
    need_gpu()
    say("swiglu checkpoint NaN block")
    rows, F = 32, 96
    c = workloads.normal_bf16((rows, 2 * F), 1.5, 51, 4, DEV)
    dh = workloads.normal_bf16((rows, F), 1e-3, 51, 5, DEV)
    ck = mxq.mx_quantize(c, colwise=False)
    ck.s_row[3, 1] = 255                                         # gate columns 32 .. 63 of row 3
    dc, h = mxq.swiglu_backward_mx_checkpoint(ck, dh)
    torch.cuda.synchronize()
    s = u8(dc.s_row)
    assert s[3, 1] == 255 and s[3, 4] == 255 and s[3, 0] != 255 and s[2, 1] != 255
    assert np.all(u8(h.s_col)[32:64, 0] == 255) and np.all(u8(h.s_col)[:32, 0] != 255)


def test_gradient_against_differences():
    """The row orientation of dc against central differences of L = sum dh silu(g) u in 64 bits, single values at a time
    summed over random sign directions: within E4M3's half step of each value (2^-4 of it, or 2^-10 of 448 block scales
    where it is subnormal)."""
    need_gpu()
    say("swiglu differences")
    rows, F = 16, 64
    c = workloads.normal_bf16((rows, 2 * F), 1.5, 51, 6, DEV)
    dh = workloads.normal_bf16((rows, F), 1.0, 51, 7, DEV)
    ck = mxq.mx_quantize(c, colwise=False)
    dc, _ = mxq.swiglu_backward_mx_checkpoint(ck, dh, colwise=False, hidden=False)
    torch.cuda.synchronize()
    x = _values(ck.q_row, ck.s_row)
    d = dh.float().cpu().numpy().astype(np.float64)
    got = _values(dc.q_row, dc.s_row)
    step = np.repeat(np.ldexp(1.0, u8(dc.s_row).astype(np.int64) - 127), 32, axis=1)

    def h(v):
        return v[:, :F] / (1.0 + np.exp(-v[:, :F])) * v[:, F:]

    e = 1e-5
    for half in (0, 1):                                          # h depends on each (g, u) pair alone
        v = np.zeros_like(x)
        v[:, half * F:(half + 1) * F] = e
        diff = d * (h(x + v) - h(x - v)) / (2 * e)
        mine = got[:, half * F:(half + 1) * F]
        tol = 2.0 ** -4 * np.abs(diff) + 2.0 ** -10 * step[:, half * F:(half + 1) * F] + 1e-8
        assert np.all(np.abs(mine - diff) <= tol)


def test_past_2_31_elements():
    """1,081,344 x 1024 hidden values (c holds 2.2e9): the last rows of the forward and the backward."""
    need_gpu()
    rows, F = 1_081_344, 1024
    say("swiglu checkpoint past 2^31 elements", rows, F)
    c = workloads.normal_bf16((8192, 2 * F), 1.5, 51, 8, DEV).repeat(132, 1)
    c[-64:] *= 2
    h, ck = mxq.swiglu_mx_quantize_checkpoint(c)
    torch.cuda.synchronize()
    t = rows - 64
    q, s, _ = oracle.swiglu_mx_quantize(u16(c[t:]))
    assert np.array_equal(u8(h.q_row[t:]), q) and np.array_equal(u8(h.s_row[t:]), s)
    o = oracle.mx_quantize(u16(c[t:]), colwise=False)
    assert np.array_equal(u8(ck.q_row[t:]), o[0]) and np.array_equal(u8(ck.s_row[t:]), o[1])
    dh = c[:, :F].contiguous()
    del c, h
    say("backward past 2^31 elements")
    dc, hc = mxq.swiglu_backward_mx_checkpoint(ck, dh)
    torch.cuda.synchronize()
    cb = oracle.bf16_from_f32(_values(ck.q_row[t:], ck.s_row[t:]).astype(np.float32))
    o = oracle.swiglu_bwd_mx_quantize(cb, u16(dh[t:]))
    got = (dc.q_row[t:], dc.s_row[t:], dc.q_col[:, t:], dc.s_col[:, t // 32:])
    assert all(np.array_equal(u8(a), b) for a, b in zip(got, o[:4]))
    _, _, hf = oracle.swiglu_mx_quantize(cb, want_h=True)
    w = oracle.mx_quantize_f32(hf, oracle.RCEIL, False, True)
    assert np.array_equal(u8(hc.q_col[:, t:]), w[2])
    del dc, hc, ck, dh
    torch.cuda.empty_cache()
