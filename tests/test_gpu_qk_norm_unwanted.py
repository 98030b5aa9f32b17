"""Buffers for the gammas' gradients that are given but not wanted, or without a norm: nothing is added to them."""
import pytest
import torch

from gpu_util import DEV
from test_gpu_qk_norm import _case, _check_back, _run_back

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", [True, False])
def test_unwanted_sums_are_left_alone(norm):
    c = _case(50, 6, 2, 64, 64, norm=norm)
    gq, gk = torch.full((64,), 3.0, device=DEV), torch.full((64,), -2.0, device=DEV)
    r = _run_back(c, accumulate=(gq, gk), want_dgamma=not norm)
    _check_back(c, r, dgamma=False)
    assert bool((gq == 3.0).all()) and bool((gk == -2.0).all())
