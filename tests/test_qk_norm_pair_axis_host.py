"""What pair_axis refuses (no GPU needed): numbers that are not whole, from a list or an array, and numbers that are no axis."""
import numpy as np
import pytest
import torch

import mxfp8_precision_numerics_amd as mxq


def _axes(pair_axis):
    pos, inv = torch.zeros(3, 4, dtype=torch.int64), torch.ones(16)
    return mxq._expect_rotation(4, pos, inv, pair_axis, None, None, 64, pos.device)[2]


@pytest.mark.parametrize("kind", [list, tuple, np.array, torch.tensor])
def test_fractions_are_refused(kind):
    for bad in ([0.0] * 16, [0] * 15 + [1.7], [0.5] * 16):
        with pytest.raises(TypeError):
            _axes(kind(bad))


@pytest.mark.parametrize("kind", [list, np.array, torch.tensor])
def test_numbers_outside_a_byte_are_refused(kind):
    for bad in ([0] * 15 + [-1], [0] * 15 + [256]):
        with pytest.raises(ValueError):
            _axes(kind(bad))


@pytest.mark.parametrize("kind", [bytearray, memoryview, lambda v: np.array(list(v), np.int32), lambda v: torch.tensor(list(v)),
                                  lambda v: range(16)])
def test_other_sequences(kind):
    want = bytes(range(16))
    assert _axes(kind(want)) == want
