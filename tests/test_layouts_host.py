"""Whether two tensors of an entry have one layout (no GPU): the stride of a
dimension of one element says nothing about where an element is."""

import pytest
import torch

from muon_newton_schulz_03_b200 import _check_tensor

F32 = (torch.float32,)


def _strides(shape, strides):
    return torch.zeros(1000).as_strided(shape, strides)


@pytest.mark.parametrize("shape,a,b", [
    ((1, 5, 3), (15, 1, 5), (7, 1, 5)), ((5, 1, 3), (1, 99, 5), (1, 1, 5)), ((1, 4, 3, 2), (24, 1, 8, 4), (1, 1, 8, 4)),
    ((1, 1), (3, 9), (9, 3))])
def test_one_layout_by_other_strides(shape, a, b):
    with pytest.raises(ValueError, match="must be on cuda"):      # the device is what is left to refuse
        _check_tensor(_strides(shape, a), "x", F32, 0, _strides(shape, b))


@pytest.mark.parametrize("shape,a,b", [((1, 5, 3), (15, 1, 5), (15, 3, 1)), ((2, 2), (1, 2), (2, 1))])
def test_other_layouts(shape, a, b):
    with pytest.raises(ValueError, match="strides"):
        _check_tensor(_strides(shape, a), "x", F32, 0, _strides(shape, b))
