"""Refusals of the 8-bit block operators (no GPU needed): the status codes of the C ABI before anything is enqueued,
and the binding's checks. Fake aligned pointers are never dereferenced."""
import ctypes as C

import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
from mxfp8_precision_numerics_amd import _lib

P, MIS = 0x10000, 0x10001


def test_rmsnorm_validation():
    f = _lib.load().rmsnorm_mx_quantize

    def call(x=P, res=P, g=P, rows=64, cols=64, eps=1e-6, total=P, rstd=P, qr=P, sr=P, qc=P, sc=P, cq=P, cs=P, rule=0):
        return f(x, res, g, rows, cols, C.c_float(eps), total, rstd, qr, sr, qc, sc, cq, cs, rule, None)

    assert call(x=None) == 1 and call(g=None) == 1 and call(rstd=None) == 1
    assert call(res=None) == 1 and call(total=None) == 1                # a residual and its sum come together
    assert call(sr=None) == 1 and call(qc=None) == 1 and call(cq=None) == 1
    assert call(qr=None, sr=None, qc=None, sc=None) == 1
    assert call(cols=48) == 2 and call(cols=32800) == 2 and call(rows=-32) == 2 and call(rows=48) == 2
    assert call(rows=128 * 65536) == 2
    assert call(x=MIS) == 3 and call(g=MIS) == 3 and call(cs=MIS) == 3 and call(total=MIS) == 3
    assert call(rule=2) == 4
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(eps=eps) == 4
    assert call(rows=0) == 0 and call(cols=0) == 0


def test_rmsnorm_backward_validation():
    lib = _lib.load()
    f = lib.rmsnorm_backward_mx_checkpoint
    ws = lib.mxq_workspace_bytes(b"rmsnorm_backward", 64)
    assert ws >= 512 * 64 * 4

    def call(dy=P, dr=P, cq=P, cs=P, rstd=P, g=P, rows=64, cols=64, dx=P, dg=P, acc=0, w=P, n=ws):
        return f(dy, dr, cq, cs, rstd, g, rows, cols, dx, dg, acc, w, n, None)

    for name in ("dy", "cq", "cs", "rstd", "g", "dx"):
        assert call(**{name: None}) == 1
    assert call(cols=40) == 2 and call(cols=32800) == 2 and call(rows=-1) == 2
    assert call(dx=MIS) == 3 and call(dr=MIS) == 3 and call(dg=MIS) == 3 and call(w=MIS) == 3
    assert call(w=None) == 5 and call(n=ws - 1) == 5
    assert call(cols=0) == 0 and call(rows=0, dg=None, w=None, n=0) == 0


def test_swiglu_checkpoint_validation():
    lib = _lib.load()
    f, b = lib.swiglu_mx_quantize_checkpoint, lib.swiglu_backward_mx_checkpoint
    assert f(None, 4, 64, P, P, P, P, 0, None) == 1 and f(P, 4, 64, P, P, None, P, 0, None) == 1
    assert f(P, 4, 48, P, P, P, P, 0, None) == 2 and f(P, -4, 64, P, P, P, P, 0, None) == 2
    assert f(MIS, 4, 64, P, P, P, P, 0, None) == 3 and f(P, 4, 64, P, P, P, P, 9, None) == 4
    assert f(None, 0, 64, None, None, None, None, 0, None) == 0
    assert b(None, P, P, 64, 64, P, P, P, P, P, P, 0, None) == 1
    assert b(P, P, P, 64, 64, None, None, None, None, None, None, 0, None) == 1
    assert b(P, P, P, 64, 64, P, None, P, P, P, P, 0, None) == 1
    assert b(P, P, P, 48, 64, P, P, None, None, P, P, 0, None) == 2     # the hidden column form needs rows % 32
    assert b(P, P, P, 64, 40, P, P, P, P, P, P, 0, None) == 2
    assert b(P, P, MIS, 64, 64, P, P, P, P, P, P, 0, None) == 3 and b(P, P, P, 64, 64, P, P, P, P, P, P, 5, None) == 4
    assert b(None, None, None, 0, 64, P, P, P, P, P, P, 0, None) == 0


def test_moe_few_tokens_validation():
    lib = _lib.load()
    f, size = lib.moe_mx_few_tokens, lib.moe_mx_few_tokens_workspace_bytes
    ws = size(4, 64, 8, 256, 128)
    assert ws > 4 * 8 * 128
    for bad in ((65, 64, 8), (-1, 64, 8), (4, 0, 1), (4, 1025, 8), (4, 64, 0), (4, 4, 5), (4, 64, 33)):
        assert size(*bad, 256, 128) == 0
    assert size(4, 64, 8, -1, 128) == 0 and size(4, 64, 8, 256, 1 << 21) == 0

    def call(x=P, l=P, T=4, E=64, k=8, u=P, d=P, D=256, F=128, y=P, w=P, n=ws):
        return f(x, P, l, T, E, k, 1, u, P, d, P, D, F, y, w, n, None)

    for name in ("x", "l", "u", "d", "y"):
        assert call(**{name: None}) == 1
        assert call(**{name: MIS}) == 3
    for bad in (dict(T=65), dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(E=4, k=5), dict(D=48), dict(F=40),
                dict(D=0), dict(F=0), dict(D=-32), dict(D=1 << 21)):
        assert call(**bad) == 2, bad
    assert call(w=None) == 5 and call(n=ws - 1) == 5 and call(w=MIS) == 3
    assert call(T=0) == 0


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros((64, 64), dtype=torch.bfloat16)
    u = torch.zeros((64, 64), dtype=torch.uint8)
    s = torch.zeros((64, 2), dtype=torch.uint8)
    ck = mxq.MXTensor(u, s, None, None)
    for call in (lambda: mxq.rmsnorm_mx_quantize(x, torch.ones(64), 1e-6),
                 lambda: mxq.rmsnorm_backward_mx_checkpoint(x, ck, torch.ones(64), torch.ones(64)),
                 lambda: mxq.swiglu_mx_quantize_checkpoint(x), lambda: mxq.swiglu_backward_mx_checkpoint(ck, x[:, :32]),
                 lambda: mxq.moe_mx_few_tokens(u, s, torch.zeros(64, 2), 1, u[None], s[None], u[None], s[None])):
        with pytest.raises(ValueError, match="device tensor"):
            call()
