"""Caller buffers of the 8-bit block operators: what is refused before a launch, and what is accepted."""
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq
from gpu_util import DEV, need_gpu, say
from mxfp8_precision_numerics_amd import workloads

pytestmark = pytest.mark.gpu


def _moe(workspace):
    u8 = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device=DEV)  # noqa: E731  (1.0)
    sc = lambda *s: torch.full(s, 120, dtype=torch.uint8, device=DEV)  # noqa: E731
    T, E, D, F = 3, 8, 64, 32
    logits = workloads.normal_f32((T, E), 1.0, 54, 1, DEV)
    return mxq.moe_mx_few_tokens(u8(T, D), sc(T, D // 32), logits, 2, u8(E, 2 * F, D), sc(E, 2 * F, D // 32), u8(E, D, F),
                                 sc(E, D, F // 32), workspace=workspace)


def _norm_bwd(workspace):
    x = workloads.normal_bf16((6, 64), 1.0, 54, 2, DEV)
    gamma = torch.ones(64, device=DEV)
    f = mxq.rmsnorm_mx_quantize(x, gamma, 1e-6, colwise=False)
    return mxq.rmsnorm_backward_mx_checkpoint(x, f.checkpoint, f.rstd, gamma, workspace=workspace)[1]


@pytest.mark.parametrize("call,size", [(_moe, lambda: mxq.moe_few_tokens_workspace_bytes(3, 8, 2, 64, 32)),
                                       (_norm_bwd, lambda: mxq.workspace_bytes("rmsnorm_backward", 64))])
def test_workspaces(call, size):
    """On the host, with gaps or too short: refused. Of another type than bytes: its bytes count."""
    need_gpu()
    say("workspaces", call.__name__)
    n = size()
    want = call(None)
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            call(bad)
    with pytest.raises(mxq.MXQError):
        call(torch.empty(n - 4, dtype=torch.uint8, device=DEV))
    for good in (torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty((n + 3) // 4, device=DEV)):
        assert torch.equal(call(good), want)


def test_no_sum_without_a_residual():
    """Buffers reused from a call with a residual: without one the result names no sum (x itself is the norm's input)."""
    need_gpu()
    say("norm buffers reused without a residual")
    x, r = workloads.normal_bf16((32, 64), 1.0, 54, 3, DEV), workloads.normal_bf16((32, 64), 1.0, 54, 4, DEV)
    gamma = torch.ones(64, device=DEV)
    first = mxq.rmsnorm_mx_quantize(x, gamma, 1e-6, residual=r)
    old = first.sum.clone()
    again = mxq.rmsnorm_mx_quantize(x, gamma, 1e-6, out=first)
    want = mxq.rmsnorm_mx_quantize(x, gamma, 1e-6)
    assert again.sum is None and torch.equal(first.sum, old)
    assert again.mx.q_row is first.mx.q_row and all(torch.equal(a, b) for a, b in zip(again.mx, want.mx))
