"""The norm and its backward through every width's kernel: rows that fill more than one step of the grid, partial chunks, rows
of zeros, infinities and NaN in each form, buffers in place, and row slices of larger tensors. Tolerances as derived in
test_gpu_norm.py, whose checks these are."""
import numpy as np
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
from gpu_util import DEV, need_gpu, say, u8
from mxfp8_precision_numerics_amd import workloads
from test_gpu_norm import EPS, U, _backward_ref, _check_forward, _f32, _gamma, _stream_like

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,residual", [
    (4110, 96, True), (4110, 512, False),          # 8 rows a workgroup, 512 workgroups
    (2060, 992, True), (2060, 544, False),         # 4 rows
    (1040, 2048, False), (1040, 1056, True),       # 2 rows
    (530, 3104, True), (530, 4096, False),         # a row a workgroup, 8 waves
    (530, 4128, False), (515, 8192, True),         # 16 waves, 256 workgroups
    (300, 8224, True), (300, 12288, False),        # 12 waves, two chunks a lane
    (270, 12320, False), (260, 16384, True),       # 16 waves
    (260, 16416, True), (259, 20000, False),       # four chunks a lane
])
def test_backward_over_more_than_one_step(rows, cols, residual):
    need_gpu()
    say("rmsnorm backward, steps", rows, cols, residual)
    x, gamma = _stream_like(rows, cols, 20), _gamma(cols, 5)
    x[rows // 2] = 0.0
    fwd = mxq.rmsnorm_mx_quantize(x, gamma, EPS, colwise=False)
    dy = workloads.normal_bf16((rows, cols), 1e-3, 50, 21, DEV)
    dres = workloads.normal_bf16((rows, cols), 1e-3, 50, 22, DEV) if residual else None
    dx, dg = mxq.rmsnorm_backward_mx_checkpoint(dy, fwd.checkpoint, fwd.rstd, gamma, residual_grad=dres)
    torch.cuda.synchronize()
    want, tol, want_g, tol_g = _backward_ref(dy, fwd.checkpoint, fwd.rstd, gamma, dres)
    # a workgroup adds rows / 256 rows where it has 12 or 16 waves
    tol_g = tol_g + rows / 256 * U * (tol_g / ((rows / 512 + 128) * U))
    assert np.all(np.abs(_f32(dx) - want) <= tol), "dx"
    assert np.all(np.abs(_f32(dg) - want_g) <= tol_g), "dgamma"
    again = mxq.rmsnorm_backward_mx_checkpoint(dy, fwd.checkpoint, fwd.rstd, gamma, residual_grad=dres)
    for place in (dy, dres):                       # in place of either gradient
        if place is None:
            continue
        mine = place.clone()
        got, dg2 = mxq.rmsnorm_backward_mx_checkpoint(mine if place is dy else dy, fwd.checkpoint, fwd.rstd, gamma,
                                                      residual_grad=mine if place is dres else dres, out=mine)
        torch.cuda.synchronize()
        assert got is mine and torch.equal(mine.view(torch.int16), dx.view(torch.int16)) and torch.equal(dg2, dg)
    assert torch.equal(again[0].view(torch.int16), dx.view(torch.int16)) and torch.equal(again[1], dg)


@pytest.mark.parametrize("rows,cols,residual,rowwise,ck,rule", [
    (32, 32, True, True, True, mxq.RCEIL), (96, 160, True, False, True, mxq.FLOOR), (64, 480, False, True, False, mxq.RCEIL),
    (1056, 512, True, True, True, mxq.RCEIL), (64, 544, True, True, True, mxq.RCEIL), (96, 992, True, False, False, mxq.RCEIL),
    (160, 1024, True, True, False, mxq.RCEIL), (64, 1056, True, True, True, mxq.RCEIL), (32, 8224, True, True, False, mxq.RCEIL),
])
def test_forward_both_orientations(rows, cols, residual, rowwise, ck, rule):
    need_gpu()
    say("rmsnorm forward, column form", rows, cols, residual, rowwise, ck, rule)
    x, res = _stream_like(rows, cols, 23), _stream_like(rows, cols, 24) if residual else None
    gamma = _gamma(cols, 6)
    out = mxq.rmsnorm_mx_quantize(x, gamma, EPS, residual=res, rowwise=rowwise, checkpoint=ck, rule=rule)
    torch.cuda.synchronize()
    _check_forward(x, res, gamma, out, rule, rowwise, True, ck)


@pytest.mark.parametrize("cols", [160, 544, 1056, 2080, 8224, 12320])
@pytest.mark.parametrize("colwise", [False, True])
def test_extreme_rows_in_every_form(cols, colwise):
    """Rows of zeros, of one value, holding NaN and infinities, of subnormals, and of squares beyond fp32 (rstd 0)."""
    need_gpu()
    say("rmsnorm extreme rows", cols, colwise)
    x = _stream_like(64, cols, 25)
    x[1] = 0.0
    x[2] = 3.0
    x[5, 7] = float("nan")
    x[9, cols - 10] = float("inf")
    x[11, 0] = float("-inf")
    x[12] = 1e-39
    x[13] = 3e38
    x[14] = -1e-20
    x[15, cols - 1] = float("nan")
    x[15, 0] = float("inf")
    gamma = _gamma(cols, 7)
    gamma[40], gamma[41] = 0.0, -2.0
    out = mxq.rmsnorm_mx_quantize(x, gamma, EPS, colwise=colwise)
    torch.cuda.synchronize()
    _check_forward(x, None, gamma, out, mxq.RCEIL, True, colwise, True)
    r, q, s = _f32(out.rstd), u8(out.mx.q_row) & 0x7F, u8(out.mx.s_row)
    assert np.isnan(r[5]) and np.isnan(r[15]) and r[9] == 0.0 and r[11] == 0.0 and r[13] == 0.0
    assert np.all(q[1] == 0) and np.all(q[5] == 0x7F) and np.all(s[5] == 255) and np.all(q[15] == 0x7F)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("cols,colwise", [(160, True), (992, True), (992, False), (4128, True), (12320, False)])
def test_in_place(which, cols, colwise):
    need_gpu()
    say("rmsnorm in place", which, cols, colwise)
    rows = 96
    x, res, gamma = _stream_like(rows, cols, 26), _stream_like(rows, cols, 27), _gamma(cols, 8)
    ref = mxq.rmsnorm_mx_quantize(x, gamma, EPS, residual=res, colwise=colwise)
    xs, rs = x.clone(), res.clone()
    new = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    out = mxq.RMSNormOut(mxq.MXTensor(*map(new, ref.mx)), xs if which == "x" else rs, new(ref.rstd),
                         mxq.MXTensor(*map(new, ref.checkpoint)))
    mxq.rmsnorm_mx_quantize(xs, gamma, EPS, residual=rs, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out.sum.view(torch.int16), ref.sum.view(torch.int16)) and torch.equal(out.rstd, ref.rstd)
    for a, b in zip(list(out.mx) + list(out.checkpoint), list(ref.mx) + list(ref.checkpoint)):
        assert b is None or torch.equal(a, b)


@pytest.mark.parametrize("cols", [96, 1056, 4128])
def test_row_slices(cols):
    """Rows out of the middle of larger tensors, inputs and outputs: the same bytes, and nothing written beside them."""
    need_gpu()
    say("rmsnorm slices", cols)
    rows, lo, n = 160, 64, 64                       # rows of 3 scale bytes: 64 of them start on 16 bytes
    x, res, gamma = _stream_like(rows, cols, 28), _stream_like(rows, cols, 29), _gamma(cols, 9)
    cut = slice(lo, lo + n)
    ref = mxq.rmsnorm_mx_quantize(x[cut].clone(), gamma, EPS, residual=res[cut].clone(), colwise=False)
    big = mxq.rmsnorm_mx_quantize(x, gamma, EPS, residual=res, colwise=False)
    for t in (big.mx.q_row, big.mx.s_row, big.checkpoint.q_row, big.checkpoint.s_row, big.rstd, big.sum):
        t.fill_(7)
    view = mxq.RMSNormOut(mxq.MXTensor(big.mx.q_row[cut], big.mx.s_row[cut], None, None), big.sum[cut], big.rstd[cut],
                          mxq.MXTensor(big.checkpoint.q_row[cut], big.checkpoint.s_row[cut], None, None))
    mxq.rmsnorm_mx_quantize(x[cut], gamma, EPS, residual=res[cut], out=view)
    dy = workloads.normal_bf16((rows, cols), 1e-3, 50, 30, DEV)
    dx, dg = mxq.rmsnorm_backward_mx_checkpoint(dy[cut].clone(), ref.checkpoint, ref.rstd, gamma)
    out = torch.full_like(dy, 7)
    dx2, dg2 = mxq.rmsnorm_backward_mx_checkpoint(dy[cut], view.checkpoint, view.rstd, gamma, out=out[cut])
    torch.cuda.synchronize()
    for a, b in ((view.mx.q_row, ref.mx.q_row), (view.mx.s_row, ref.mx.s_row), (view.sum, ref.sum), (view.rstd, ref.rstd),
                 (view.checkpoint.q_row, ref.checkpoint.q_row), (view.checkpoint.s_row, ref.checkpoint.s_row), (dx2, dx), (dg2, dg)):
        assert torch.equal(a, b)
    for t in (big.mx.q_row, big.mx.s_row, big.checkpoint.q_row, big.checkpoint.s_row, big.rstd, big.sum, out):
        assert bool((t[:lo] == 7).all()) and bool((t[lo + n:] == 7).all())
