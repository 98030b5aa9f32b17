"""qk_norm_rope and its backward against the 64-bit formulas.

Tolerances, in units of u = 2^-24 (half a step of fp32): a sum of squares passes at most 8 roundings, its mean 2, rsqrt 2, so
rstd is within 7 u; n = (x rstd) gamma within 9 u; cos and sin within 2 u of 1; the turn's two products and sum add 2. So an
output is within 13 u < 2^-20 of its pair's |a| + |b|, and its rounding to bf16 adds 2^-8 of itself. A gradient's turned dy
is within 4 u of its pair, t = d gamma, the mean and the difference add under 28: 2^-19 of the terms' magnitudes, and bf16's
2^-8. A dgamma adds at most 64 terms a lane here, then at most 16 partial sums: 2^-17 of the terms' magnitudes."""
import math
from fractions import Fraction

import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
import qk_reference as ref
from gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _case(T, hq, hk, dim, rot, axes=1, norm=True, seed=0, extra=0, far=1000):
    need_gpu()
    g = torch.Generator(device=DEV).manual_seed(seed * 1009 + T + hq + dim)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    c = dict(T=T, hq=hq, hk=hk, dim=dim)
    c["qkv"] = (2.0 * n(T, (hq + hk) * dim + extra)).bfloat16()
    c["pos"] = torch.randint(0, far, (axes, T), generator=g, device=DEV)
    c["inv"] = (10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) / max(1, rot // 2))).float()
    c["axis"] = None if axes == 1 else [i % axes for i in range(rot // 2)]
    c["gq"], c["gk"] = (1 + 0.3 * n(dim), 1 + 0.3 * n(dim)) if norm else (None, None)
    c["dq"], c["dk"] = n(T, hq, dim).bfloat16(), n(T, hk, dim).bfloat16()
    return c


def _run(c, interleaved=False, out=None):
    return mxq.qk_norm_rope(c["qkv"], c["hq"], c["hk"], c["dim"], c["pos"], c["inv"], c["gq"], c["gk"], EPS,
                            pair_axis=c["axis"], interleaved=interleaved, out=out)


def _check(c, got, interleaved=False):
    args = (c["qkv"], c["hq"], c["hk"], c["dim"], c["pos"], c["inv"], c["gq"], c["gk"], EPS, c["axis"], interleaved)
    for y, want, size in zip(got, ref.forward(*args), ref.magnitude(*args)):
        off = (y.double() - want).abs()
        assert bool((off <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size + 1e-37).all()), float(off.max())


def _run_back(c, interleaved=False, **more):
    return mxq.qk_norm_rope_backward(c["dq"], c["dk"], c["qkv"], c["pos"], c["inv"], c["gq"], c["gk"], EPS,
                                     pair_axis=c["axis"], interleaved=interleaved, **more)


def _check_back(c, r, interleaved=False, dgamma=True):
    dx, gq, gk, sx, sq, sk = ref.backward(c["dq"], c["dk"], c["qkv"], c["pos"], c["inv"], c["gq"], c["gk"], EPS, c["axis"],
                                          interleaved)
    off = (r.dqk[:, :dx.shape[1]].double() - dx).abs()
    assert bool((off <= 2.0 ** -8 * dx.abs() + 2.0 ** -19 * sx + 1e-37).all()), float(off.max())
    if c["gq"] is None or not dgamma:
        assert r.dgamma_q is None and r.dgamma_k is None
        return
    for got, want, size in ((r.dgamma_q, gq, sq), (r.dgamma_k, gk, sk)):
        assert bool(((got.double() - want).abs() <= 2.0 ** -17 * size + 1e-37).all())


SHAPES = [(1, 16, 16, 128, 128), (1, 1, 1, 64, 64), (1, 96, 96, 128, 128), (3, 5, 2, 128, 128), (7, 8, 1, 64, 32),
          (5, 3, 3, 96, 96), (2, 7, 2, 80, 64), (9, 4, 2, 192, 64), (4, 6, 2, 256, 256), (11, 2, 1, 16, 16), (6, 3, 1, 32, 16),
          (13, 9, 0, 48, 48), (13, 0, 9, 112, 96), (333, 16, 4, 128, 128), (65, 40, 8, 160, 0), (1000, 2, 2, 128, 64),
          (3000, 12, 4, 128, 128)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,hq,hk,dim,rot", SHAPES)
def test_forward_and_backward(T, hq, hk, dim, rot, norm, interleaved):
    c = _case(T, hq, hk, dim, rot, norm=norm)
    say("qk_norm_rope", T, hq, hk, dim, rot, norm, interleaved)
    _check(c, _run(c, interleaved), interleaved)
    say("qk_norm_rope_backward", T, hq, hk, dim, rot, norm, interleaved)
    _check_back(c, _run_back(c, interleaved), interleaved)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_several_axes(axes, interleaved):
    c = _case(77, 6, 2, 128, 96, axes=axes)
    _check(c, _run(c, interleaved), interleaved)
    _check_back(c, _run_back(c, interleaved), interleaved)


def test_far_positions():
    """Angles of positions up to 2^40, and below zero: an angle in 32 bits would be off by whole turns."""
    c = _case(64, 4, 2, 128, 128, far=1 << 40)
    c["pos"][0, :8] = -c["pos"][0, :8]
    c["pos"][0, 8:12] = torch.tensor([0, 1, (1 << 31) - 1, 1 << 31], device=DEV)
    # the reference's own 64-bit angle is good to 2^-53 of itself: 2^-13 here, so it is formed exactly instead
    pos, inv = c["pos"][0].tolist(), c["inv"].tolist()
    two_pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592, 10 ** 63) * 2
    ang = []
    for p in pos:
        row = []
        for f in inv:
            a = Fraction(p) * Fraction(f)
            row.append(float(a - math.floor(a / two_pi) * two_pi))
        ang.append(row)
    a = torch.tensor(ang, dtype=torch.float64, device=DEV)
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    got = _run(c)
    for y, x, g in zip(got, ref._split(c["qkv"], 4, 2, 128), (c["gq"], c["gk"])):
        n = ref._one(x, g, EPS)[1]
        want, size = ref.turn(n, cos, sin, False), ref._both(n.abs(), cos, False)
        assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all())


def test_views_strides_and_in_place():
    c = _case(37, 6, 2, 128, 128, extra=2 * 128)
    q, k = _run(c)
    _check(c, (q, k))
    # head-major outputs, and rows of a cache whose other rows stay
    qh = torch.zeros(6, 37, 128, dtype=torch.bfloat16, device=DEV)
    cache = torch.full((64, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    _run(c, out=(qh.transpose(0, 1), cache[20:57]))
    assert torch.equal(qh.transpose(0, 1), q) and torch.equal(cache[20:57], k)
    assert bool((cache[:20] == 7.0).all()) and bool((cache[57:] == 7.0).all())
    # in place, the values behind the heads left as they were
    x = c["qkv"].clone()
    d = dict(c, qkv=x)
    _run(d, out=(x[:, :768].view(37, 6, 128), x[:, 768:1024].view(37, 2, 128)))
    assert torch.equal(x[:, :768].view(37, 6, 128), q) and torch.equal(x[:, 768:1024].view(37, 2, 128), k)
    assert torch.equal(x[:, 1024:], c["qkv"][:, 1024:])
    # the backward from head-major gradients, into wider rows
    r = _run_back(c)
    _check_back(c, r)
    wide = torch.full((37, 1280), 7.0, dtype=torch.bfloat16, device=DEV)
    e = dict(c, dq=c["dq"].transpose(0, 1).contiguous().transpose(0, 1), dk=c["dk"].transpose(0, 1).contiguous().transpose(0, 1))
    s = _run_back(e, out=wide)
    assert torch.equal(wide[:, :1024], r.dqk) and bool((wide[:, 1024:] == 7.0).all())
    assert torch.equal(s.dgamma_q, r.dgamma_q) and torch.equal(s.dgamma_k, r.dgamma_k)
    x = c["qkv"].clone()                                                  # over the input itself
    s = _run_back(dict(c, qkv=x), out=x)
    assert torch.equal(x[:, :1024], r.dqk) and torch.equal(x[:, 1024:], c["qkv"][:, 1024:])


def test_dgamma_forms():
    c = _case(50, 6, 2, 64, 64)
    r = _run_back(c)
    s = _run_back(c, want_dgamma=False)
    assert torch.equal(s.dqk, r.dqk) and s.dgamma_q is None
    gq, gk = torch.full((64,), 3.0, device=DEV), torch.full((64,), -2.0, device=DEV)
    t = _run_back(c, accumulate=(gq, gk))
    assert t.dgamma_q is gq and torch.allclose(gq - 3.0, r.dgamma_q, atol=1e-4) and torch.allclose(gk + 2.0, r.dgamma_k, atol=1e-4)
    ws = torch.empty(mxq.workspace_bytes("qk_norm_backward", 64), dtype=torch.uint8, device=DEV)
    u = _run_back(c, workspace=ws)
    assert torch.equal(u.dgamma_q, r.dgamma_q) and torch.equal(u.dgamma_k, r.dgamma_k)
    e = {**c, "T": 0, "qkv": c["qkv"][:0], "pos": c["pos"][:, :0].contiguous(), "dq": c["dq"][:0], "dk": c["dk"][:0]}
    v = _run_back(e)
    assert v.dqk.shape == (0, 512) and not v.dgamma_q.any() and not v.dgamma_k.any()
    gq.fill_(3.0)
    _run_back(e, accumulate=(gq, gk))
    assert bool((gq == 3.0).all())
    assert _run(e)[0].shape == (0, 6, 64)


def test_many_tokens_dgamma():
    """More tokens than one pass of the grid holds: every wave takes several."""
    c = _case(20000, 3, 1, 64, 64)
    _check(c, _run(c))
    _check_back(c, _run_back(c))


@pytest.mark.parametrize("norm", [True, False])
def test_non_finite_values_stay_in_their_place(norm):
    """With a norm an infinity or NaN spoils its own head; without, its own pair, and past the rotation itself alone."""
    c = _case(9, 4, 2, 96, 64, norm=norm)
    clean = [t.clone() for t in _run(c)]
    x = c["qkv"].view(9, 6, 96)
    x[2, 1, 3], x[4, 3, 80], x[5, 5, 40], x[6, 0, 95] = float("nan"), float("inf"), -float("inf"), float("nan")
    q, k = _run(c)
    full = torch.cat([q, k], 1)
    want = torch.cat(clean, 1)
    touched = torch.zeros_like(full, dtype=torch.bool)
    for t, h, d in ((2, 1, 3), (4, 3, 80), (5, 5, 40), (6, 0, 95)):
        if norm:
            touched[t, h] = True
        else:
            touched[t, h, d] = True
            if d < 64:
                touched[t, h, d + 32 if d < 32 else d - 32] = True
    assert torch.equal(full[~touched], want[~touched])
    if norm:
        assert bool(torch.isnan(full[2, 1]).all()) and bool(torch.isnan(full[6, 0]).all())
    else:
        assert float(full[4, 3, 80]) == float("inf") and not bool(torch.isfinite(full[2, 1, 3]))


def test_zero_heads():
    c = _case(4, 2, 1, 64, 64)
    c["qkv"].zero_()
    q, k = _run(c)
    assert not q.any() and not k.any()
    _check_back(c, _run_back(c))
