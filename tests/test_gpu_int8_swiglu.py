"""SwiGLU of the int8 products over the whole range of gates, in every kernel (which one a shape takes is asserted from the plan).

g and u are the fp32 values that the interface names, reproduced here bit for bit, so what is left to allow is, for g >= -87, silu's
(13 + 2 |g|) 2^-24 and the product's rounding, 2^-24 of the result each, and the rounding to bf16, 2^-8; 2^-22 covers the products of
these. Below -87 silu may also be 0, which is off by less than 2^-119 |u|. Up values are about 2^60, so no result is subnormal as long
as silu is above 2^-180."""
import pytest
import torch

import int8_plan as P
import mxfp8_precision_numerics_amd as mxq
from gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu
FAR = 105.0


def _operands(g, M, F, K, groups=None):
    """Codes of every value, and scales that spread the gates over -FAR .. FAR, a third of them within a few units."""
    lead = () if groups is None else (groups,)
    c = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)  # noqa: E731
    r = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    unit = 5461.0 * K ** 0.5                                              # a sum's standard deviation
    sa = (0.5 + r(M)) / unit
    gate = torch.where(r(*lead, F) < 0.33, 2.0, 50.0) * (0.2 + r(*lead, F))
    up = (0.5 + r(*lead, F)) * 2.0 ** 60
    return c(M, K), sa, c(*lead, 2 * F, K), torch.cat([gate, up], -1).contiguous()


def _check(c, a, sa, b, sb):
    y = ((a.double() @ b.double().t()).float() * sa[:, None]) * sb[None]
    F = y.shape[1] // 2
    gate, up = y[:, :F].double(), y[:, F:].double()
    h = gate / (1.0 + torch.exp(-gate)) * up
    tol = h.abs() * (2.0 ** -8 + 2.0 ** -22 + (14.0 + 2.0 * gate.abs()) * 2.0 ** -24)
    tol = torch.where(gate < -87.0, tol + 2.0 ** -119 * up.abs(), tol)
    bad = torch.isnan(y[:, :F]) | torch.isnan(y[:, F:])
    assert torch.equal(torch.isnan(c), bad)
    assert bool(((c.double() - h).abs() <= tol)[~bad].all())
    return gate[~bad]


DENSE = [(1, 100, 2048, P.FEW), (16, 130, 544, P.FEW), (61, 1000, 256, P.FEW), (130, 6150, 160, P.MIDDLE),
         (257, 8193, 96, P.MIDDLE), (16, 18432, 7008, P.WIDE), (61, 25001, 1952, P.WIDE), (100, 12290, 4000, P.WIDE),
         (1030, 4100, 288, P.LARGE), (1030, 4099, 96, P.LARGE), (2100, 8200, 512, P.LARGE)]


@pytest.mark.parametrize("M,F,K,kind", DENSE)
def test_dense(M, F, K, kind, tmp_path):
    need_gpu()
    assert P.plan(P.load(str(tmp_path)), M, F, K, swiglu=True)[0] == kind
    g = torch.Generator(device=DEV).manual_seed(M + F + K)
    a, sa, b, sb = _operands(g, M, F, K)
    say("int8_scaled_gemm swiglu", M, F, K)
    gates = _check(mxq.int8_scaled_gemm(a, sa, b, sb, swiglu=True), a, sa, b, sb)
    if M > 1:
        assert float(gates.min()) < -FAR and float(gates.max()) > FAR and bool((gates.abs() < 1.0).any())
    # rows and channels whose scale is NaN or zero: those are NaN or zero, the others as ever
    sa[M // 2], sb[3], sb[F + 4] = float("nan"), float("nan"), float("nan")
    sb[5], sb[F + 6] = 0.0, 0.0
    if M > 2:
        sa[0] = 0.0
    _check(mxq.int8_scaled_gemm(a, sa, b, sb, swiglu=True), a, sa, b, sb)


GROUPED = [(8, 130, 256, [0, 3, 3, 20, 21, 21, 40, 41, 60], P.FEW), (5, 2000, 160, [0, 100, 101, 101, 240, 300], P.MIDDLE),
           (3, 1030, 416, [0, 1, 1700, 3001], P.LARGE), (9, 1501, 64, [0, 0, 255, 511, 767, 1023, 1400, 1401, 2200, 2200], P.LARGE)]


@pytest.mark.parametrize("G,F,K,off,kind", GROUPED)
def test_grouped(G, F, K, off, kind, tmp_path):
    need_gpu()
    rows = off[-1]
    assert P.plan(P.load(str(tmp_path)), rows, F, K, G, True)[0] == kind
    g = torch.Generator(device=DEV).manual_seed(G + F + K)
    a, sa, b, sb = _operands(g, rows, F, K, G)
    sa[off[-1] - 1], sa[0] = float("nan"), 0.0
    say("int8_grouped_gemm swiglu", G, rows, F, K)
    c = mxq.int8_grouped_gemm(a, sa, torch.tensor(off, device=DEV), b, sb, swiglu=True)
    for e in range(G):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            _check(c[lo:hi], a[lo:hi], sa[lo:hi], b[e], sb[e])


def test_each_gate():
    """One gate a channel, from -125 to 125 in steps of a quarter, by a product of one code."""
    need_gpu()
    gates = torch.arange(-500, 501, device=DEV).float() / 4
    F = len(gates)
    a = torch.zeros(4, 32, dtype=torch.int8, device=DEV)
    a[:, 0] = torch.tensor([1, -1, 0, 1], device=DEV)
    b = torch.zeros(2 * F, 32, dtype=torch.int8, device=DEV)
    b[:, 0] = 1
    sa, sb = torch.ones(4, device=DEV), torch.cat([gates, torch.full((F,), 2.0 ** 60, device=DEV)])
    _check(mxq.int8_scaled_gemm(a, sa, b, sb, swiglu=True), a, sa, b, sb)
