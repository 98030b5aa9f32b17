"""The int8 operators on operands without rows or columns."""
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [0, 1, 7, 3000])
def test_rows_without_values_have_scale_zero(rows):
    need_gpu()
    x = torch.empty(rows, 0, dtype=torch.bfloat16, device=DEV)
    out = mxq.Int8Tensor(torch.empty(rows, 0, dtype=torch.int8, device=DEV), torch.full((rows,), 99.0, device=DEV))
    assert mxq.int8_quantize_tokens(x, out=out) is out and not out.scale.any()
    assert mxq.int8_quantize_tokens(x).q.shape == (rows, 0)


@pytest.mark.parametrize("swiglu", [False, True])
def test_products_without_rows_or_columns(swiglu):
    need_gpu()
    a, sa = torch.ones(5, 64, dtype=torch.int8, device=DEV), torch.ones(5, device=DEV)
    b, sb = torch.ones(8, 64, dtype=torch.int8, device=DEV), torch.ones(8, device=DEV)
    n = 4 if swiglu else 8
    off = torch.tensor([0, 2, 5], device=DEV)
    assert mxq.int8_scaled_gemm(a[:0], sa[:0], b, sb, swiglu=swiglu).shape == (0, n)
    assert mxq.int8_scaled_gemm(a, sa, b[:0], sb[:0], swiglu=swiglu).shape == (5, 0)
    assert mxq.int8_grouped_gemm(a[:0], sa[:0], off * 0, torch.stack([b, b]), torch.stack([sb, sb]), swiglu=swiglu).shape == (0, n)
    assert mxq.int8_grouped_gemm(a, sa, off, torch.stack([b, b])[:, :0], torch.stack([sb, sb])[:, :0],
                                 swiglu=swiglu).shape == (5, 0)
    out = torch.full((5, n), 7.0, dtype=torch.bfloat16, device=DEV)                # no group holds a row: nothing is written
    mxq.int8_grouped_gemm(a, sa, off * 0, torch.stack([b, b]), torch.stack([sb, sb]), swiglu=swiglu, out=out)
    assert bool((out == 7.0).all())
