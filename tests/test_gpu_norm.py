"""RMSNorm with residual addition and MXFP8 output, and its backward from the 8-bit checkpoint, against plain 64-bit
formulas and the CPU oracle's quantizer.

Forward: the residual sum is one rounding, so it is compared bit for bit. rstd is within 2^-18 of the 64-bit value: the
sum of squares (all positive) passes at most 32 sequential and 11 joining additions, so its relative error is below
44 * 2^-24, of which rstd takes half, plus 4 roundings of its own. The codes are then those of the oracle's fp32 quantizer
on fl(fl(h rstd) gamma) with the kernel's own rstd, byte for byte.
Backward: dx is within bf16's rounding plus the fp32 error of the projection term, dgamma within the depth of its sum."""
import numpy as np
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
import oracle
from gpu_util import DEV, need_gpu, say, u16, u8
from mxfp8_precision_numerics_amd import workloads

pytestmark = pytest.mark.gpu

EPS = 1e-6
U = 2.0 ** -24


def _f32(t):
    return t.detach().float().cpu().numpy()


def _gamma(cols, k=0):
    return 1.0 + 0.2 * workloads.normal_f32((cols,), 1.0, 50, 100 + k, DEV)


def _stream_like(rows, cols, k):
    """N(0, 1) values with a few columns 20 times as large."""
    x = workloads.normal_f32((rows, cols), 1.0, 50, k, DEV)
    x[:, :: max(1, cols // 3)] *= 20.0
    return x.to(torch.bfloat16)


def _same_codes(got, want):
    """Equal bytes, a NaN code (S.1111.111) of either sign matching another."""
    got, want = u8(got), np.asarray(want)
    nan = (want & 0x7F) == 0x7F
    return np.array_equal((got & 0x7F) == 0x7F, nan) and np.array_equal(got[~nan], want[~nan])


def _check_forward(x, res, gamma, out, rule, rowwise, colwise, ck):
    h = x if res is None else (x.cpu().float() + res.cpu().float()).to(torch.bfloat16)
    if res is not None:
        assert np.array_equal(u16(out.sum), u16(h)), "sum"
    hf = _f32(h)
    rstd = _f32(out.rstd)
    with np.errstate(all="ignore"):
        want = 1.0 / np.sqrt((hf.astype(np.float64) ** 2).mean(1) + EPS)
        ok = np.isfinite(want) & (np.abs(hf).max(1) < 1e15)
        assert np.all(np.abs(rstd[ok] - want[ok]) <= 2.0 ** -18 * want[ok]), "rstd"
        y = (hf * rstd[:, None]) * _f32(gamma)
    q = oracle.mx_quantize_f32(y, rule, rowwise, colwise)
    if rowwise:
        assert np.array_equal(u8(out.mx.s_row), q[1]) and _same_codes(out.mx.q_row, q[0]), "row"
    if colwise:
        assert np.array_equal(u8(out.mx.s_col), q[3]) and _same_codes(out.mx.q_col, q[2]), "col"
    if ck:
        c = oracle.mx_quantize(u16(h), rule, colwise=False)
        assert np.array_equal(u8(out.checkpoint.s_row), c[1]) and _same_codes(out.checkpoint.q_row, c[0]), "checkpoint"
    else:
        assert out.checkpoint is None


@pytest.mark.parametrize("rows,cols,residual,rowwise,colwise,ck,rule", [
    (1, 32, True, True, False, False, mxq.RCEIL),
    (1, 2048, True, True, False, True, mxq.RCEIL),
    (7, 96, False, True, False, True, mxq.RCEIL),
    (3, 544, True, True, False, False, mxq.FLOOR),
    (32, 512, True, True, True, True, mxq.RCEIL),
    (33, 1056, True, True, False, True, mxq.RCEIL),
    (96, 1024, False, True, True, True, mxq.FLOOR),
    (160, 2048, True, False, True, True, mxq.RCEIL),
    (352, 2080, True, True, True, True, mxq.RCEIL),
    (64, 4096, True, True, True, False, mxq.RCEIL),
    (1120, 4128, True, True, True, True, mxq.RCEIL),
    (64, 8192, False, True, True, True, mxq.RCEIL),
    (96, 12288, True, True, True, True, mxq.RCEIL),
    (32, 16416, True, True, True, True, mxq.RCEIL),
    (32, 32768, True, True, True, True, mxq.RCEIL),
])
def test_forward(rows, cols, residual, rowwise, colwise, ck, rule):
    need_gpu()
    say("rmsnorm forward", rows, cols, residual, rowwise, colwise, ck, rule)
    x = _stream_like(rows, cols, 1)
    res = _stream_like(rows, cols, 2) if residual else None
    gamma = _gamma(cols)
    out = mxq.rmsnorm_mx_quantize(x, gamma, EPS, residual=res, rowwise=rowwise, colwise=colwise, checkpoint=ck, rule=rule)
    torch.cuda.synchronize()
    _check_forward(x, res, gamma, out, rule, rowwise, colwise, ck)


def test_forward_extreme_rows():
    """Rows of zeros, of one value, holding NaN and infinities, of subnormals, and of squares beyond fp32 (rstd 0)."""
    need_gpu()
    say("rmsnorm extreme rows")
    rows, cols = 64, 160
    x = _stream_like(rows, cols, 3)
    x[1] = 0.0
    x[2] = 3.0
    x[5, 7] = float("nan")
    x[9, 150] = float("inf")
    x[11, 0] = float("-inf")
    x[12] = 1e-39
    x[13] = 3e38
    x[14] = -1e-20
    gamma = _gamma(cols)
    gamma[40] = 0.0
    gamma[41] = -2.0
    out = mxq.rmsnorm_mx_quantize(x, gamma, EPS)
    torch.cuda.synchronize()
    _check_forward(x, None, gamma, out, mxq.RCEIL, True, True, True)
    r = _f32(out.rstd)
    assert np.isnan(r[5]) and r[9] == 0.0 and r[11] == 0.0 and r[13] == 0.0
    assert np.all(u8(out.mx.q_row)[1] & 0x7F == 0)
    assert np.all((u8(out.mx.q_row)[5] & 0x7F) == 0x7F) and np.all(u8(out.mx.s_row)[5] == 255)


@pytest.mark.parametrize("which", ["x", "residual"])
def test_forward_in_place_and_on_a_side_stream(which):
    need_gpu()
    say("rmsnorm in place", which)
    rows, cols = 96, 2048
    x, res, gamma = _stream_like(rows, cols, 4), _stream_like(rows, cols, 5), _gamma(cols)
    ref = mxq.rmsnorm_mx_quantize(x, gamma, EPS, residual=res)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    xs, rs = x.clone(), res.clone()
    mine = mxq.RMSNormOut(mxq.MXTensor(*[torch.empty_like(t) for t in ref.mx]), xs if which == "x" else rs,
                          torch.empty_like(ref.rstd),
                          mxq.MXTensor(torch.empty_like(ref.checkpoint.q_row), torch.empty_like(ref.checkpoint.s_row), None, None))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        mxq.rmsnorm_mx_quantize(xs, gamma, EPS, residual=rs, out=mine)
    side.synchronize()
    assert torch.equal(mine.sum.view(torch.int16), ref.sum.view(torch.int16)) and torch.equal(mine.rstd, ref.rstd)
    assert all(torch.equal(a, b) for a, b in zip(mine.mx, ref.mx))
    assert torch.equal(mine.checkpoint.q_row, ref.checkpoint.q_row)


def _values(q, s):
    """float64 values of an MXFP8 row orientation; a block with scale byte 0xFF is NaN."""
    v = oracle.fp8_value(u8(q), oracle.E4M3).astype(np.float64)
    b = u8(s).astype(np.int64)
    f = np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    return v * np.repeat(f, 32, axis=1)


def _backward_ref(dy, ck, rstd, gamma, dres):
    """dx, dgamma and their error bounds, in float64."""
    dyf, g = _f32(dy).astype(np.float64), _f32(gamma).astype(np.float64)
    rs = _f32(rstd).astype(np.float64)[:, None]
    xh = _values(ck.q_row, ck.s_row) * rs
    t = dyf * g
    cols = xh.shape[1]
    m = (t * xh).sum(1, keepdims=True) / cols
    d = 0.0 if dres is None else _f32(dres).astype(np.float64)
    dx = rs * (t - xh * m) + d
    # m: at most 32 sequential and 11 joining additions, 4 roundings a term; then 6 roundings of the two terms
    mabs = np.abs(t * xh).sum(1, keepdims=True) / cols
    tol = 2.0 ** -8 * np.abs(dx) + rs * (np.abs(xh) * mabs * 64 * U + 8 * U * (np.abs(t) + np.abs(xh * m))) + 4 * U * np.abs(d)
    # dgamma: rows / 512 sequential additions a workgroup, 64 + 8 joining ones, 2 roundings a term
    tol_g = (dyf.shape[0] / 512 + 128) * U * np.abs(dyf * xh).sum(0) + 1e-45
    return dx, tol, (dyf * xh).sum(0), tol_g


@pytest.mark.parametrize("rows,cols,residual,accumulate", [
    (1, 32, True, False), (1, 2048, False, False), (5, 96, True, True), (333, 1056, True, False), (513, 512, False, True),
    (600, 2048, True, False), (40, 4128, True, False), (1030, 8192, True, False), (70, 12288, True, True),
    (9, 16384, False, False), (17, 32768, True, False),
])
def test_backward(rows, cols, residual, accumulate):
    need_gpu()
    say("rmsnorm backward", rows, cols, residual, accumulate)
    x, gamma = _stream_like(rows, cols, 6), _gamma(cols, 1)
    fwd = mxq.rmsnorm_mx_quantize(x, gamma, EPS, colwise=False)
    dy = workloads.normal_bf16((rows, cols), 1e-3, 50, 7, DEV)
    dres = workloads.normal_bf16((rows, cols), 1e-3, 50, 8, DEV) if residual else None
    base = workloads.normal_f32((cols,), 1.0, 50, 9, DEV)
    acc = base.clone() if accumulate else None
    dx, dg = mxq.rmsnorm_backward_mx_checkpoint(dy, fwd.checkpoint, fwd.rstd, gamma, residual_grad=dres, accumulate=acc)
    torch.cuda.synchronize()
    want, tol, want_g, tol_g = _backward_ref(dy, fwd.checkpoint, fwd.rstd, gamma, dres)
    assert np.all(np.abs(_f32(dx) - want) <= tol), "dx"
    if accumulate:
        assert dg is acc
        b = _f32(base).astype(np.float64)
        want_g, tol_g = want_g + b, tol_g + 2 * U * (np.abs(b) + np.abs(want_g))
    assert np.all(np.abs(_f32(dg) - want_g) <= tol_g), "dgamma"
    # the same call again gives the same bits, in place too, and dgamma can be left out
    again, dg2 = mxq.rmsnorm_backward_mx_checkpoint(dy, fwd.checkpoint, fwd.rstd, gamma, residual_grad=dres)
    place = dy.clone()
    mine, none = mxq.rmsnorm_backward_mx_checkpoint(place, fwd.checkpoint, fwd.rstd, gamma, residual_grad=dres,
                                                    want_dgamma=False, out=place)
    torch.cuda.synchronize()
    assert none is None and torch.equal(again.view(torch.int16), dx.view(torch.int16))
    assert torch.equal(mine.view(torch.int16), dx.view(torch.int16))
    if not accumulate:
        assert torch.equal(dg2, dg)


def test_backward_against_differences():
    """Where the checkpoint is exact (h on the MXFP8 grid), dx and dgamma are the derivatives of
    L = sum dy y(h) + sum dr h: compared with central differences of L in 64 bits along random directions. The bound is
    dx's rounding to bf16 (2^-9 a value, doubled) and the differences' own h^2 term."""
    need_gpu()
    say("rmsnorm differences")
    rows, cols = 12, 256
    q = mxq.mx_quantize(_stream_like(rows, cols, 10), colwise=False)
    h = _values(q.q_row, q.s_row)
    x = torch.from_numpy(h).to(torch.bfloat16).to(DEV)
    assert np.array_equal(_f32(x).astype(np.float64), h)
    gamma = _gamma(cols, 2)
    fwd = mxq.rmsnorm_mx_quantize(x, gamma, EPS, colwise=False)
    dy = workloads.normal_bf16((rows, cols), 1.0, 50, 11, DEV)
    dr = workloads.normal_bf16((rows, cols), 1.0, 50, 12, DEV)
    dx, dg = mxq.rmsnorm_backward_mx_checkpoint(dy, fwd.checkpoint, fwd.rstd, gamma, residual_grad=dr)
    torch.cuda.synchronize()
    g, dyf, drf = (_f32(t).astype(np.float64) for t in (gamma, dy, dr))

    def loss(hh, gg):
        y = hh / np.sqrt((hh ** 2).mean(1, keepdims=True) + EPS) * gg
        return (dyf * y).sum() + (drf * hh).sum()

    rng = np.random.default_rng(7)
    e = 1e-4
    dxf, dgf = _f32(dx).astype(np.float64), _f32(dg).astype(np.float64)
    for _ in range(6):
        v = rng.choice([-1.0, 1.0], size=h.shape)
        diff = (loss(h + e * v, g) - loss(h - e * v, g)) / (2 * e)
        assert abs((dxf * v).sum() - diff) <= 2.0 ** -8 * np.abs(dxf).sum() + 1e-5
        w = rng.choice([-1.0, 1.0], size=g.shape)
        diff = (loss(h, g + e * w) - loss(h, g - e * w)) / (2 * e)
        assert abs((dgf * w).sum() - diff) <= 1e-5 * np.abs(dgf).sum()


def test_backward_nan_block_and_empty():
    need_gpu()
    say("rmsnorm backward NaN block, empty")
    rows, cols = 4, 96
    x, gamma = _stream_like(rows, cols, 13), _gamma(cols, 3)
    fwd = mxq.rmsnorm_mx_quantize(x, gamma, EPS, colwise=False)
    fwd.checkpoint.s_row[2, 1] = 255
    dy = workloads.normal_bf16((rows, cols), 1e-3, 50, 14, DEV)
    dx, dg = mxq.rmsnorm_backward_mx_checkpoint(dy, fwd.checkpoint, fwd.rstd, gamma)
    torch.cuda.synchronize()
    assert bool(torch.isnan(dx[2]).all()) and not bool(torch.isnan(dx[[0, 1, 3]]).any())
    assert bool(torch.isnan(dg[32:64]).all()) and not bool(torch.isnan(dg[:32]).any())
    empty = torch.empty((0, cols), dtype=torch.bfloat16, device=DEV)
    ck = mxq.MXTensor(torch.empty((0, cols), dtype=torch.uint8, device=DEV),
                      torch.empty((0, cols // 32), dtype=torch.uint8, device=DEV), None, None)
    none = torch.empty(0, dtype=torch.float32, device=DEV)
    _, dg = mxq.rmsnorm_backward_mx_checkpoint(empty, ck, none, gamma)
    acc = torch.ones(cols, device=DEV)
    mxq.rmsnorm_backward_mx_checkpoint(empty, ck, none, gamma, accumulate=acc)
    out = mxq.rmsnorm_mx_quantize(empty, gamma, EPS)
    torch.cuda.synchronize()
    assert bool((dg == 0).all()) and bool((acc == 1).all()) and out.rstd.numel() == 0


def test_past_2_31_elements():
    """98304 x 32768 values (3.2e9): the last rows against the oracle, both orientations and the checkpoint; then the
    backward's last rows."""
    need_gpu()
    rows, cols = 98304, 32768
    say("rmsnorm past 2^31 elements", rows, cols)
    x = workloads.normal_bf16((1024, cols), 1.0, 50, 15, DEV).repeat(96, 1)
    x[-40:] *= 3
    gamma = _gamma(cols, 4)
    out = mxq.rmsnorm_mx_quantize(x, gamma, EPS)
    torch.cuda.synchronize()
    tail = rows - 64
    part = mxq.RMSNormOut(mxq.MXTensor(out.mx.q_row[tail:], out.mx.s_row[tail:], out.mx.q_col[:, tail:].contiguous(),
                                       out.mx.s_col[:, tail // 32:].contiguous()), None, out.rstd[tail:],
                          mxq.MXTensor(out.checkpoint.q_row[tail:], out.checkpoint.s_row[tail:], None, None))
    _check_forward(x[tail:], None, gamma, part, mxq.RCEIL, True, True, True)
    say("backward past 2^31 elements")
    ck, rstd = out.checkpoint, out.rstd
    dy = x                                                      # any gradient serves
    dx, _ = mxq.rmsnorm_backward_mx_checkpoint(dy, ck, rstd, gamma)
    torch.cuda.synchronize()
    ckt = mxq.MXTensor(ck.q_row[tail:].contiguous(), ck.s_row[tail:].contiguous(), None, None)
    want, tol, _, _ = _backward_ref(dy[tail:], ckt, rstd[tail:], gamma, None)
    assert np.all(np.abs(_f32(dx[tail:]) - want) <= tol)
    del x, out, dx, dy, ck, part
    torch.cuda.empty_cache()
