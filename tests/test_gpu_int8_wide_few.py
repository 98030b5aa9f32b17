"""The int8 products of up to 16 tokens with weights of 256 MB and more but few rows: the one-tile-a-CU kernel with few blocks of B."""
import pytest
import torch

import int8_plan as P
import mxfp8_precision_numerics_amd as mxq
from gpu_util import say
from test_gpu_int8 import _check, _gen, _operands, _sums

pytestmark = pytest.mark.gpu
SHAPES = [(5, 8200, 31232), (16, 8196, 40000), (9, 16384, 16000), (12, 10002, 30016)]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dense(M, N, K, swiglu, tmp_path):
    g = _gen(M * 31 + N * 7 + K)
    assert P.variant(P.load(str(tmp_path)), M, N // 2 if swiglu else N, K, swiglu=swiglu) == ("wide", 16, True, swiglu)
    a, sa, b, sb = _operands(g, M, N, K)
    if swiglu:
        sa = sa * 0.001
    say("int8_scaled_gemm", M, N, K, swiglu)
    _check(mxq.int8_scaled_gemm(a, sa, b, sb, swiglu=swiglu), _sums(a, b), sa, sb, swiglu)
