"""The norm's sum of squares on rows where the order of its additions shows.

A square of a bf16 value is exact in fp32, so rstd's error is that of the additions and of four operations after them.
Added in pairs, a sum of cols values passes ceil(log2 cols) roundings, each within u = 2^-24 of the partial sum, and all
terms are positive: relative error at most ceil(log2 cols) u. The division by cols and the addition of eps add one each,
the square root halves what came before it, and it and the reciprocal add one each:

    |rstd / exact - 1| <= (ceil(log2 cols) / 2 + 3) u        (second-order terms are below 1e-3 u)

The rows below hold a 1 at every eighth of their first columns and 2^-24 * 0.9 as square of every other value: added one
after the other behind a 1, each of these is lost (0.9 u is less than half the spacing 2 u of numbers above 1), and a
lane's 32 values lose 31 * 0.9 u of 1 + 31 * 0.9 u, half of which, 13.9 u, would show in rstd."""
import math

import numpy as np
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
from gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SMALL = 243.0 / 256.0 * 2.0 ** -12                                # a bf16 value, its square 0.9010 u


@pytest.mark.parametrize("rows,cols,ones,colwise,residual", [
    (5, 2048, 512, False, False), (3, 8192, 2048, False, True), (2, 12288, 4096, False, False), (2, 32768, 8192, False, False),
    (32, 1024, 512, True, False), (32, 992, 512, True, True), (32, 2048, 512, True, False), (1, 512, 512, False, False),
])
def test_rstd_of_rows_with_many_small_squares(rows, cols, ones, colwise, residual):
    need_gpu()
    say("rmsnorm sums", rows, cols, ones, colwise, residual)
    x = torch.full((rows, cols), SMALL, dtype=torch.bfloat16)
    x[:, :ones:8] = 1.0
    x[rows - 1] *= 4.0                                            # the same bits one and a half decades up
    res = torch.zeros_like(x).to(DEV) if residual else None
    eps = 2.0 ** -40
    out = mxq.rmsnorm_mx_quantize(x.to(DEV), torch.ones(cols, device=DEV), eps, residual=res, colwise=colwise)
    torch.cuda.synchronize()
    want = 1.0 / np.sqrt((x.double().numpy() ** 2).mean(1) + eps)
    off = np.abs(out.rstd.double().cpu().numpy() / want - 1.0) / U
    say("rstd off by", off.max(), "u")
    assert np.all(off <= math.ceil(math.log2(cols)) / 2 + 3 + 1e-3)


def test_more_rows_than_the_column_form_takes():
    """8388648 rows in the row orientation (the column one ends at 8388480): every row equals its like in a short call."""
    need_gpu()
    rows, cols, n = 128 * 65536 + 40, 32, 65536
    say("rmsnorm rows", rows, cols)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    few = torch.randn((n, cols), generator=g, device=DEV).to(torch.bfloat16)
    gamma = 1.0 + 0.1 * torch.randn(cols, generator=g, device=DEV)
    x = few.repeat(rows // n + 1, 1)[:rows].contiguous()
    out = mxq.rmsnorm_mx_quantize(x, gamma, 1e-6, colwise=False)
    want = mxq.rmsnorm_mx_quantize(few, gamma, 1e-6, colwise=False)
    torch.cuda.synchronize()
    for a, b in ((out.rstd, want.rstd), (out.mx.q_row, want.mx.q_row), (out.mx.s_row, want.mx.s_row),
                 (out.checkpoint.q_row, want.checkpoint.q_row), (out.checkpoint.s_row, want.checkpoint.s_row)):
        for r in range(0, rows, n):
            assert torch.equal(a[r:r + n], b[:min(n, rows - r)]), r


@pytest.mark.parametrize("rows,cols,colwise", [
    (4096, 2048, False), (2048, 8192, False), (1024, 12288, False), (512, 16384, False), (64, 32768, True), (4096, 512, True),
    (2048, 992, True), (2048, 96, False), (1024, 4128, True),
])
def test_rstd_is_the_exact_value_rounded(rows, cols, colwise):
    """Eight squares are added in pairs in fp32 (three roundings, at most 3 u, half of which reaches rstd), everything after
    that in 64 bits (below 1e-3 u), and rstd is rounded once: |rstd / exact - 1| <= 2.5 u + 1e-3 u."""
    need_gpu()
    say("rmsnorm rstd", rows, cols, colwise)
    g = torch.Generator(device=DEV)
    g.manual_seed(cols)
    x = torch.randn((rows, cols), generator=g, device=DEV) * torch.exp2(torch.arange(rows, device=DEV) % 23 - 11)[:, None]
    x = x.to(torch.bfloat16)
    x[:, :: cols // 4] *= 20.0
    x[0] = SMALL
    x[0, ::8] = 1.0
    out = mxq.rmsnorm_mx_quantize(x, torch.ones(cols, device=DEV), 1e-6, colwise=colwise, checkpoint=False)
    torch.cuda.synchronize()
    eps = float(torch.tensor(1e-6, dtype=torch.float32))
    want = 1.0 / (x.double().square().mean(1) + eps).sqrt()
    off = (out.rstd.double() / want - 1.0).abs() / U
    say("rstd off by", float(off.max()), "u, root mean square", float(off.square().mean().sqrt()))
    assert float(off.max()) <= 2.5 + 1e-3
