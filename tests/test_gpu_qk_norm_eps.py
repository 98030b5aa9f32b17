"""The smallest eps of the head norms, 2^-126: zero heads stay zero, and heads of tiny values keep the formula."""
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
import qk_reference as ref
from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -126


def test_smallest_eps():
    need_gpu()
    T, hq, hk, dim = 5, 3, 2, 64
    g = torch.Generator(device=DEV).manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    qkv = n(T, hq + hk, dim)
    qkv[0], qkv[1, 1], qkv[2] = 0.0, 0.0, qkv[2] * 2.0 ** -66             # squares around 2^-132: subnormal, below eps
    qkv = qkv.bfloat16().view(T, -1)
    pos, inv = torch.arange(T, device=DEV) * 7, (1e4 ** (-torch.arange(dim // 2, device=DEV) / (dim // 2))).float()
    gq, gk = 1 + 0.3 * n(dim), 1 + 0.3 * n(dim)
    args = (qkv, hq, hk, dim, pos, inv, gq, gk, EPS)
    # a subnormal square is off by up to half of 2^-149, which is 2^-23 of eps: with the 13 roundings of ordinary heads below 2^-19
    for y, want, size in zip(mxq.qk_norm_rope(*args), ref.forward(*args), ref.magnitude(*args)):
        assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * size).all())
    q, k = mxq.qk_norm_rope(*args)
    assert not q[0].any() and not k[0].any() and not q[1, 1].any()
    # gradients of ordinary size: dx up to 2^63 of them, and no zero head puts a NaN into dgamma
    dq, dk = n(T, hq, dim).bfloat16(), n(T, hk, dim).bfloat16()
    r = mxq.qk_norm_rope_backward(dq, dk, qkv, pos, inv, gq, gk, EPS)
    dx, wq, wk, sx, sq, sk = ref.backward(dq, dk, qkv, pos, inv, gq, gk, EPS)
    assert bool(((r.dqk.double() - dx).abs() <= 2.0 ** -8 * dx.abs() + 2.0 ** -18 * sx).all())
    for got, want, size in ((r.dgamma_q, wq, sq), (r.dgamma_k, wk, sk)):
        assert bool(((got.double() - want).abs() <= 2.0 ** -17 * size).all())
