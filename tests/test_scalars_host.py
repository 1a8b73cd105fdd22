"""One-element tensors that the calls read on the device: what is read is the
memory, so a tensor whose value is its memory negated is no multiplier."""

import pytest
import torch

from muon_newton_schulz_03_b200 import _check_scalar


@pytest.mark.parametrize("bad", [torch._neg_view(torch.ones(1)), torch.conj(torch.ones(1, dtype=torch.complex64)).imag,
                                 torch.ones(1).to_sparse()])
def test_a_scalar_that_is_not_its_memory_is_refused(bad):
    assert bad.dtype == torch.float32 and bad.numel() == 1
    with pytest.raises(ValueError, match="one element, stored as it is"):
        _check_scalar(bad, "grad_scale", torch.float32, 0)
