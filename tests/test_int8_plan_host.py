"""Which int8 kernel takes which call: the shapes beside the rules' figures, and that the GPU tests' shapes reach every compiled form, so
that a changed rule does not leave one untested."""
import itertools

import pytest

import int8_plan as P
import test_gpu_int8 as T
import test_gpu_int8_wide_few as W


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return P.load(str(tmp_path_factory.mktemp("plan")))


@pytest.mark.parametrize("M,N,K,G,swiglu,kind", [
    (1, 6144, 2048, 0, False, P.FEW), (64, 256, 4096, 0, False, P.FEW), (256, 2048, 8192, 0, False, P.FEW),
    (100, 6144, 2048, 0, False, P.FEW), (61, 8192, 8192, 0, False, P.FEW), (16, 12288, 12288, 0, False, P.FEW),
    (16, 36864, 12288, 0, False, P.WIDE), (32, 12288, 12288, 0, False, P.WIDE), (61, 36864, 12288, 0, False, P.WIDE),
    (128, 36864, 12288, 0, False, P.WIDE), (129, 12288, 12288, 0, False, P.MIDDLE), (130, 12288, 12288, 0, False, P.MIDDLE),
    (200, 6144, 2048, 0, False, P.MIDDLE), (400, 12288, 12288, 0, False, P.MIDDLE), (512, 12288, 12288, 0, False, P.LARGE),
    (160, 36864, 12288, 0, False, P.LARGE), (4096, 36864, 12288, 0, False, P.LARGE), (128, 2048, 2048, 64, True, P.FEW),
    (16 * 64, 2048, 2048, 64, True, P.MIDDLE), (64 * 64, 2048, 2048, 64, True, P.MIDDLE), (72 * 64, 2048, 2048, 64, True, P.LARGE),
    (131072, 2048, 2048, 64, True, P.LARGE), (131072, 2048, 1024, 64, False, P.LARGE)])
def test_kernel_of(lib, M, N, K, G, swiglu, kind):
    assert P.plan(lib, M, N // 2 if swiglu else N, K, G, swiglu)[0] == kind


def test_every_form_is_tested(lib):
    reached = set()
    for swiglu in (False, True):
        cols = lambda N: (N + 1) // 2 if swiglu else N  # noqa: E731
        for M, N, K in T.SHAPES + T.WIDE + W.SHAPES:
            reached.add(P.variant(lib, M, cols(N), K, 0, swiglu))
        for G, N, K, off in T.GROUPS:
            reached.add(P.variant(lib, off[-1] if off else 2 * G, cols(N), K, G, swiglu))
        for G, K in ((64, 96), (130, 288), (200, 544)):                   # test_large_grouped_tiles_in_turn, 130 rows a group
            reached.add(P.variant(lib, 130 * G, cols(2064), K, G, swiglu))
    both = (False, True)
    every = {("few", *v) for v in itertools.product((16, 32, 64), both, both)}
    every |= {("wide", *v) for v in itertools.product((16, 32, 64, 128), both, both)}
    every |= {("middle", *v) for v in itertools.product(both, both, both)}
    every |= {("large", *v) for v in itertools.product(both, both, both)}
    assert reached == every
