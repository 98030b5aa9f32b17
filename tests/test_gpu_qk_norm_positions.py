"""Positions at the end of the range for which the angles' bound is stated: |position| <= 2^53, |position * inv_freq| < 2^50. The pairs
are (1, 0), so the outputs are cos and sin themselves, rounded to bf16 once: 2^-9 for values up to 1, and 2^-23 of the bound."""
import math
from fractions import Fraction

import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
from gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
TWO_PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592, 10 ** 63) * 2


def test_farthest_positions():
    need_gpu()
    pos = [2 ** 53, 2 ** 53 - 1, -2 ** 53, 2 ** 52 + 1, -(2 ** 53 - 3), 2 ** 50 + 7, 12345678912345, 2 ** 31]
    inv = torch.tensor([2.0 ** -4 * (1 - 2.0 ** -24), 0.1, 0.07, 1e-3, 1e-9, 2.0 ** -40, 0.11, 1e-5], dtype=torch.float32, device=DEV)
    inv = torch.where(inv > 2.0 ** -4, inv / 2, inv)                      # 2^53 of the largest stays below 2^50
    x = torch.zeros(len(pos), 16, dtype=torch.bfloat16, device=DEV)
    x[:, :8] = 1.0
    q, _ = mxq.qk_norm_rope(x, 1, 0, 16, torch.tensor(pos, device=DEV), inv)
    for t, p in enumerate(pos):
        for i, f in enumerate(inv.tolist()):
            a = Fraction(p) * Fraction(f)
            assert abs(a) < 2 ** 50
            a = float(a - math.floor(a / TWO_PI) * TWO_PI)
            for got, want in ((float(q[t, 0, i]), math.cos(a)), (float(q[t, 0, 8 + i]), math.sin(a))):
                assert abs(got - want) <= 2.0 ** -9 + 2.0 ** -23, (p, f)
