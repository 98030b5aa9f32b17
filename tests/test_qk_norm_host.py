"""Refusals of qk_norm_rope and its backward (no GPU needed), and the 64-bit formulas that the GPU tests compare with:
their gradient against differences."""
import ctypes as C

import numpy as np
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
from mxfp8_precision_numerics_amd import _lib
from qk_reference import backward, forward

P, MIS, ODD = 0x10000, 0x10008, 0x10001


def _forward(x=P, ld=256, T=8, hq=2, hk=1, dim=64, gq=P, gk=P, eps=1e-6, pos=P, axes=1, inv=P, rot=64, pair=None, inter=0,
             q=P, qt=128, qh=64, k=P, kt=64, kh=64):
    return _lib.load().qk_norm_rope(x, ld, T, hq, hk, dim, gq, gk, C.c_float(eps), pos, axes, inv, rot, pair, inter, q, qt,
                                    qh, k, kt, kh, None)


def _backward(dq=P, qt=128, qh=64, dk=P, kt=64, kh=64, x=P, ld=256, T=8, hq=2, hk=1, dim=64, gq=P, gk=P, eps=1e-6, pos=P,
              axes=1, inv=P, rot=64, pair=None, inter=0, dx=P, ldd=192, dgq=P, dgk=P, acc=0, ws=P, n=None):
    lib = _lib.load()
    n = lib.mxq_workspace_bytes(b"qk_norm_backward", dim) if n is None else n
    return lib.qk_norm_rope_backward(dq, qt, qh, dk, kt, kh, x, ld, T, hq, hk, dim, gq, gk, C.c_float(eps), pos, axes, inv,
                                     rot, pair, inter, dx, ldd, dgq, dgk, acc, ws, n, None)


@pytest.mark.parametrize("f", [_forward, _backward])
def test_validation(f):
    x, q, k = ("x", "q", "k") if f is _forward else ("x", "dq", "dk")
    for name in (x, q, k, "pos", "inv", "gq", "gk"):
        assert f(**{name: None}) == 1, name
    for bad in (dict(dim=24, rot=16), dict(dim=272, rot=64), dict(dim=0, rot=0), dict(rot=8), dict(rot=80), dict(rot=-16),
                dict(axes=0), dict(axes=5), dict(T=-1), dict(T=(1 << 25) + 1), dict(hq=-1), dict(hk=65537), dict(ld=184),
                dict(ld=260), dict(qt=56), dict(qh=60), dict(qh=68), dict(kt=-64), dict(pair=bytes([1] * 32)),
                dict(axes=3, pair=bytes([2] * 31 + [3]))):
        assert f(**bad) == 2, bad
    for name in (x, q, k, "gq", "gk"):
        assert f(**{name: MIS}) == 3, name
    assert f(pos=0x10004) == 3 and f(inv=ODD) == 3
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert f(eps=eps) == 4
    more = {} if f is _forward else dict(dgq=None, dgk=None, ws=None, n=0)
    assert f(T=0, **{x: None, q: None, k: None}, **more) == 0 and f(hq=0, hk=0, **more) == 0


def test_backward_validation():
    assert _backward(dx=None) == 1 and _backward(dgq=None) == 1 and _backward(dgk=None) == 1
    assert _backward(ldd=184) == 2 and _backward(ldd=196) == 2
    assert _backward(dx=MIS) == 3 and _backward(dgq=MIS) == 3 and _backward(ws=MIS) == 3
    assert _backward(gq=None, gk=None) == 4                               # no norm has no gamma
    n = _lib.load().mxq_workspace_bytes(b"qk_norm_backward", 64)
    assert n > 0 and _backward(ws=None) == 5 and _backward(n=n - 1) == 5
    assert _lib.load().mxq_workspace_bytes(b"qk_norm_backward", 512) == 0


def test_binding_checks():
    qkv, inv, pos = torch.zeros(4, 192).bfloat16(), torch.ones(32), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        mxq.qk_norm_rope(qkv, 2, 1, 64, pos, inv)                         # not on a device
    with pytest.raises(ValueError):
        mxq.qk_norm_rope_backward(qkv.view(4, 3, 64), qkv.view(4, 3, 64), None, pos, inv)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
def test_formula_gradient_against_differences(norm, interleaved):
    """The 64-bit gradient formulas against central differences of the 64-bit forward, along random directions: the
    difference quotient with step h is off by h^2 f''' / 6, below 1e-7 here, and by rounding, about 1e-15 / h."""
    g = torch.Generator().manual_seed(5)
    T, hq, hk, dim, rot = 3, 2, 1, 32, 16
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    qkv = r(T, (hq + hk) * dim)
    gq, gk = (1 + 0.2 * r(dim), 1 + 0.2 * r(dim)) if norm else (None, None)
    pos, inv, axis = torch.randint(0, 50, (2, T), generator=g), torch.rand(rot // 2, generator=g), [0, 1] * (rot // 4)
    dq, dk = r(T, hq, dim), r(T, hk, dim)

    def loss(x, a, b):
        q, k = forward(x, hq, hk, dim, pos, inv, a, b, 1e-6, axis, interleaved)
        return float((q * dq).sum() + (k * dk).sum())

    dx, dgq, dgk = backward(dq, dk, qkv, pos, inv, gq, gk, 1e-6, axis, interleaved)[:3]
    h = 1e-4
    v = r(*qkv.shape)
    diff = (loss(qkv + h * v, gq, gk) - loss(qkv - h * v, gq, gk)) / (2 * h)
    assert abs(diff - float((dx * v).sum())) < 1e-5
    if norm:
        v = r(dim)
        assert abs((loss(qkv, gq + h * v, gk) - loss(qkv, gq - h * v, gk)) / (2 * h) - float((dgq * v).sum())) < 1e-5
        assert abs((loss(qkv, gq, gk + h * v) - loss(qkv, gq, gk - h * v)) / (2 * h) - float((dgk * v).sum())) < 1e-5


def test_gradients_of_both_gammas_in_one_buffer_are_refused():
    for dgk in (P, P + 16, P + 4 * 64 - 16, P - 16):
        for acc in (0, 1):
            assert _backward(dgk=dgk, acc=acc) == 4, (hex(dgk), acc)


@pytest.mark.parametrize("kind", [list, bytes, np.array, torch.tensor, lambda v: torch.tensor(v, dtype=torch.uint8)])
def test_pair_axis_from_any_sequence(kind):
    """An array of 64-bit numbers is a sequence of its numbers, not of their bytes."""
    want = [0] * 8 + [1] * 12 + [2] * 12
    pos, inv = torch.zeros(3, 4, dtype=torch.int64), torch.ones(32)
    axes, rot, got = mxq._expect_rotation(4, pos, inv, kind(want), None, None, 64, pos.device)
    assert (axes, rot, list(got)) == (3, 64, want)
    with pytest.raises(ValueError):
        mxq._expect_rotation(4, pos, inv, kind(want[1:]), None, None, 64, pos.device)
