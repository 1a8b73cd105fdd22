"""The operators on lists of gradients at the ends of their arguments' ranges,
against their definitions in 64 bits (tolerances: see test_gpu_grad_ops)."""

import math

import pytest
import torch

import muon_newton_schulz_03_b200 as muon

from gpu_helpers import DEV
from test_gpu_grad_ops import U, exact_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def opt():
    with muon.Muon(device=0) as o:
        yield o


# -- the bound is a 64-bit number --------------------------------------------

# 700,000 elements take several kernels, 1000 one.
@pytest.mark.parametrize("n", [1000, 700_000])
def test_a_bound_above_the_range_of_fp32(opt, n):
    g = torch.full((n,), 3e38, device=DEV)
    want, _ = exact_norm([g])                     # about 9.5e39 and 2.5e41: beyond fp32 too
    bound = 1e39
    norm, scale = opt.grad_norm([g], max_norm=bound)
    assert norm.item() == math.inf and abs(scale.item() - bound / want) <= 1.001 * U * (bound / want)
    opt.clip_grads([g], bound)
    s = bound / want * float(torch.tensor(3e38))
    assert ((g.double() - s).abs() <= 3 * U * s).all()      # the multiplier and the product
    g[7] = math.nan                               # a bound, so NaN shows
    assert math.isnan(opt.grad_norm([g], max_norm=bound)[1].item())
    assert opt.grad_norm([g], max_norm=math.inf)[1].item() == 1.0


@pytest.mark.parametrize("n", [1, 200_000])
@pytest.mark.parametrize("bound", [0.1, 1.0 + 2.0 ** -24, 1.0 - 2.0 ** -26, 1e-3])
def test_the_multiplier_is_one_rounding_off(opt, n, bound):
    # A norm that is exact in fp64, so that nothing but the multiplier's own rounding is left.
    g = torch.zeros(n, device=DEV)
    g[-1] = 1.5
    s = bound / (1.5 + 1e-6)
    got = opt.grad_norm([g], max_norm=bound)[1].item()
    assert abs(got - s) <= 1.0001 * U * s


# -- a positive eps below fp32's range ---------------------------------------

@pytest.mark.parametrize("step", [1, 1000, "device"])
@pytest.mark.parametrize("eps", [1e-30, 1e-44, 1e-46, 1e-60, 5e-324])
def test_entries_without_gradients_only_decay_whatever_eps(opt, eps, step):
    # Rows of an embedding that no token named: 0 / (0 + eps) = 0 in the definition.
    n, lr, wd = 3000, 1e-2, 0.1
    p, g, m, v = (torch.zeros(n, device=DEV) for _ in range(4))
    p += 0.75
    g[1000] = 0.5
    t = torch.tensor(1, device=DEV) if step == "device" else step
    opt.adamw_step([p], [g], [m], [v], lr=lr, step=t, eps=eps, wd=wd)
    rest = torch.arange(n, device=DEV) != 1000
    want = 0.75 * (1 - lr * wd)
    assert ((p[rest].double() - want).abs() <= 3 * U * want).all()       # the factor, the product, the sum
    assert (m[rest] == 0).all() and (v[rest] == 0).all()
    assert math.isfinite(p[1000].item()) and p[1000] != p[0]
