"""The operators on lists of gradients at the ends of their arguments' ranges,
against their definitions in 64 bits (tolerances: see test_gpu_grad_ops)."""

import math
import os
import subprocess
import sys

import pytest
import torch

import muon_newton_schulz_03_b200 as muon

from gpu_helpers import DEV
from test_gpu_grad_ops import BF16, F32, U, clip_of, exact_norm, norm_tol, tensors

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


# -- one tensor of many units among small ones --------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_per_tensor_norms_of_a_table_and_vectors(opt, dtype, kind):
    ts = tensors([700, 1, 90_000_001, 0, 5000, 33], (dtype,), seed=80, offset=1, scale=0.1)
    norm, _, per = opt.grad_norm(ts, norm_type=kind, per_tensor=True)
    want, want_per = exact_norm(ts, kind)
    tol = norm_tol(ts, kind)
    assert abs(norm.item() - want) <= tol * want
    assert all(abs(x - w) <= tol * w for x, w in zip(per.tolist(), want_per))


# -- captured calls between other streams' work --------------------------------

@pytest.mark.parametrize("n", [1000, 300_001])
def test_captured_after_a_join_of_two_streams(opt, n):
    # The call's kernels follow two branches of the graph at once, and another branch follows them.
    g = [torch.zeros(n, device=DEV) for _ in range(2)]
    p, m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    src = torch.zeros((), device=DEV)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        g[0].copy_(src.expand(n))
        with torch.cuda.stream(side):
            g[1].copy_((2 * src).expand(n))
        main.wait_stream(side)
        norm, scale = opt.grad_norm(g, max_norm=1.0)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            seen = norm + scale
        opt.adamw_step([p], [g[0]], [m], [v], lr=1e-3, step=1, wd=0.0, grad_scale=scale)
        main.wait_stream(side)
    for x in (0.25, 3.0, 1.0):
        src.fill_(x)
        m.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = x * math.sqrt(5.0 * n)
        s = clip_of(want, 1.0)
        assert abs(norm.item() - want) <= 1.001 * U * want and abs(scale.item() - s) <= 1.001 * U * s
        assert seen.item() == (norm + scale).item()
        first = 0.1 * s * x                                    # m' = (1 - beta1) s g
        assert ((m.double() - first).abs() <= 5 * U * first).all()
    del graph


FIRST = """
import math, torch
import muon_newton_schulz_03_b200 as muon
o = muon.Muon(device=0)
n = {n}
t = [torch.full((n,), 0.5, device="cuda") for _ in range(4)]
one = torch.ones(1, dtype=torch.int64, device="cuda")
graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=stream):
    norm, scale = o.grad_norm(t, max_norm=1.0)
    o.clip_grads(t[:1], 0.25)
    o.adamw_step(t[1:2], t[:1], t[2:3], t[3:], lr=1e-3, step=one, grad_scale=scale)
graph.replay()
torch.cuda.synchronize()
assert abs(norm.item() - math.sqrt(n)) <= 1e-6 * math.sqrt(n), norm.item()
assert (t[1] != 0.5).all()
del graph
print("captured")
"""


@pytest.mark.parametrize("n", [1000, 300_001])
def test_the_first_calls_of_a_process_are_captured(n):
    r = subprocess.run([sys.executable, "-c", FIRST.format(n=n)], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
