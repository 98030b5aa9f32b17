"""Routed int8 products with offsets that break the rule, at sizes that take the large tiles (which kernel takes them is asserted
from the plan): wrong rows, but every call ends and nothing outside the output is touched."""
import pytest
import torch

import int8_plan as P
import mxfp8_precision_numerics_amd as mxq
from gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("what", ["alternating", "backwards", "astray"])
def test_large_tiles(what, swiglu, tmp_path):
    need_gpu()
    G, rows, K = 65, 4161, 96
    N = 1400 if swiglu else 700
    assert P.plan(P.load(str(tmp_path)), rows, 700, K, G, swiglu)[:2] == ((P.LARGE, 492) if swiglu else (P.LARGE, 246))
    if what == "alternating":
        off = [0 if i % 2 == 0 else rows for i in range(G + 1)]
    elif what == "backwards":
        off = [rows - 64 * i for i in range(G + 1)]
    else:
        off = [-7] + [(1 << 40) if i % 3 == 0 else 61 * i for i in range(1, G + 1)]
    g = torch.Generator(device=DEV).manual_seed(1)
    a = torch.randint(-128, 128, (rows, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
    b = torch.randint(-128, 128, (G, N, K), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
    sa, sb = torch.rand(rows, generator=g, device=DEV), torch.rand(G, N, generator=g, device=DEV)
    whole = torch.full((rows + 64, 700), 7.0, dtype=torch.bfloat16, device=DEV)
    say("int8_grouped_gemm with offsets", what, swiglu)
    mxq.int8_grouped_gemm(a, sa, torch.tensor(off, device=DEV), b, sb, swiglu=swiglu, out=whole[32:32 + rows])
    torch.cuda.synchronize()
    assert bool((whole[:32] == 7.0).all()) and bool((whole[32 + rows:] == 7.0).all())
