"""The clipping bound's range, without a GPU: it is a 64-bit number, so nothing
that is negative or finite there turns into 0 or infinity on the way."""

import math

import pytest

from test_grad_ops_host import _clip, _norm


@pytest.mark.parametrize("call", [_norm, _clip])
@pytest.mark.parametrize("bound", [-1e-60, -5e-324, -math.inf, math.nan])
def test_a_negative_bound_is_refused_however_small(call, bound):
    rc, text = call(max_norm=bound)
    assert rc == 1 and "max_norm" in text


@pytest.mark.parametrize("call", [_norm, _clip])
@pytest.mark.parametrize("bound", [0.0, 1e-60, 1e60, math.inf])
def test_bounds_of_any_size_are_taken(call, bound):
    assert call(max_norm=bound) == (1, "handle is NULL")
