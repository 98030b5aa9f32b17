"""Refusals of the int8 operators (no GPU needed): the status codes of the C ABI before anything is enqueued, and the
binding's checks. Fake aligned pointers are never dereferenced."""
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
from mxfp8_precision_numerics_amd import _lib

P, MIS, ODD = 0x10000, 0x10008, 0x10001


def test_quantize_validation():
    f = _lib.load().int8_quantize_tokens

    def call(x=P, rows=4, cols=64, q=P, s=P):
        return f(x, rows, cols, q, s, None)

    assert call(x=None) == 1 and call(q=None) == 1 and call(s=None) == 1
    assert call(cols=48) == 2 and call(rows=-1) == 2 and call(cols=-32) == 2
    assert call(rows=1 << 26, cols=64) == 2 and call(rows=1 << 24, cols=2080) == 2 and call(rows=1 << 22, cols=8224) == 2
    assert call(x=MIS) == 3 and call(q=MIS) == 3 and call(s=ODD) == 3
    assert call(rows=0, x=None, q=None, s=None) == 0 and call(cols=0) == 0


@pytest.mark.parametrize("grouped", [False, True])
def test_gemm_validation(grouped):
    lib = _lib.load()

    def call(a=P, sa=P, off=P, G=4, M=64, b=P, sb=P, N=64, K=64, swiglu=0, c=P, ldc=64):
        if grouped:
            return lib.int8_grouped_gemm(a, sa, off, G, M, b, sb, N, K, swiglu, c, ldc, None)
        return lib.int8_scaled_gemm(a, sa, b, sb, M, N, K, swiglu, c, ldc, None)

    for name in ("a", "sa", "b", "sb", "c") + (("off",) if grouped else ()):
        assert call(**{name: None}) == 1
    assert call(K=0) == 2 and call(K=48) == 2 and call(K=131072) == 2 and call(K=-32) == 2
    assert call(M=-1) == 2 and call(N=-1) == 2 and call(ldc=63) == 2 and call(N=63, swiglu=1, ldc=64) == 2
    assert call(swiglu=1, ldc=31) == 2
    assert call(M=1 << 30, N=1 << 20, ldc=1 << 20) == 2                  # more tiles than one launch holds
    assert call(a=MIS) == 3 and call(b=MIS) == 3 and call(sa=ODD) == 3 and call(sb=ODD) == 3 and call(c=ODD) == 3
    assert call(M=0, a=None, c=None) == 0 and call(N=0, b=None, c=None) == 0
    if grouped:
        assert call(G=0) == 2 and call(G=4097) == 2 and call(off=MIS) == 3


def test_binding_checks():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        mxq.int8_quantize_tokens(x.bfloat16())                           # not on a device
    with pytest.raises(ValueError):
        mxq.int8_scaled_gemm(x.to(torch.int8), torch.ones(4), x.to(torch.int8), torch.ones(4))
    with pytest.raises(ValueError):
        mxq.int8_grouped_gemm(x.to(torch.int8), torch.ones(4), torch.zeros(2, dtype=torch.int64),
                              x.to(torch.int8)[None], torch.ones(1, 4))
