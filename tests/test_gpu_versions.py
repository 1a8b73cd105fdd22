"""What the calls write in place counts as written to autograd: the tensors'
version counters move, so that a backward pass over a graph that saved the old
values raises instead of computing with the new ones. What is only read, and
the entries of a skipped row, keep theirs."""

import pytest
import torch

import muon_newton_schulz_03_b200 as muon

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def opt():
    with muon.Muon(device=0) as o:
        yield o


def versions(*lists):
    return [[t._version for t in ts] for ts in lists]


def state(sizes):
    return [[torch.full((n,), 0.25, device=DEV) for n in sizes] for _ in range(4)]


# One kernel, several kernels, more tensors than a launch takes.
SIZES = [[100, 7], [200_000, 3], [5] * 800]


@pytest.mark.parametrize("sizes", SIZES)
def test_adamw_moves_what_it_writes(opt, sizes):
    p, g, m, v = state(sizes)
    kept = [torch.zeros(3, device=DEV) for _ in range(3)]
    before, kept_before = versions(p, g, m, v), versions(kept)
    opt.adamw_step(p + kept[:1], g + [None], m + kept[1:2], v + kept[2:], lr=1e-3, step=1)
    after = versions(p, g, m, v)
    for k in (0, 2, 3):
        assert all(a > b for a, b in zip(after[k], before[k]))
    assert after[1] == before[1] and versions(kept) == kept_before


@pytest.mark.parametrize("sizes", SIZES)
def test_clip_moves_what_it_writes(opt, sizes):
    g, out = state(sizes)[:2]
    before = versions(g, out)
    opt.clip_grads(g + [None], 0.1, out=out + [None])
    after = versions(g, out)
    assert after[0] == before[0] and all(a > b for a, b in zip(after[1], before[1]))
    opt.clip_grads(g + [None], 0.1)
    assert all(t._version > b for t, b in zip(g, before[0]))
    opt.clip_grads(out, 0.1, out=list(out))             # in place through another list
    assert all(t._version > b for t, b in zip(out, after[1]))


def test_the_norm_and_refused_calls_move_nothing(opt):
    p, g, m, v = state([100, 7])
    before = versions(p, g, m, v)
    opt.grad_norm(g, max_norm=1.0, per_tensor=True)
    for call in (lambda: opt.clip_grads(g, -1.0), lambda: opt.clip_grads([g[0], g[0]], 1.0),
                 lambda: opt.adamw_step(p, g, m, v, lr=1e-3, step=0),
                 lambda: opt.adamw_step(p, g, m, [v[0], v[1][:6]], lr=1e-3, step=1)):
        with pytest.raises((muon.MuonError, ValueError)):
            call()
    assert versions(p, g, m, v) == before


@pytest.mark.parametrize("what", ["param", "grad"])
def test_a_graph_over_old_values_raises(opt, what):
    w = torch.full((50,), 0.5, device=DEV, requires_grad=True)
    loss = (w * w).sum()
    if what == "param":
        opt.adamw_step([w], [torch.ones(50, device=DEV)], [torch.zeros(50, device=DEV)], [torch.zeros(50, device=DEV)],
                       lr=1e-3, step=1)
    else:
        (g,) = torch.autograd.grad(loss, w, create_graph=True)
        loss = (g * g * w).sum()                       # saves the gradient
        opt.clip_grads([g.detach()], 0.1)              # which shares its counter
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_have_no_counter(opt):
    with torch.inference_mode():
        p, g, m, v = state([33, 200_000])
    opt.adamw_step(p, g, m, v, lr=1e-3, step=1)
    opt.clip_grads(g, 0.1)
    with torch.inference_mode():
        opt.adamw_step(p, g, m, v, lr=1e-3, step=2)
    assert all((t != 0.25).all() for t in p + g)


@pytest.mark.parametrize("buffers", [1, 3, 9])
def test_tensors_that_share_a_counter(opt, buffers):
    # Views share their buffer's counter, in turn from several of them; a detached one and its source too.
    bases = [torch.full((4000,), 0.25, device=DEV) for _ in range(buffers)]
    views = [bases[i % buffers][(i // buffers) * 100:(i // buffers) * 100 + 60] for i in range(27)]
    before = versions(bases)[0]
    opt.clip_grads(views, 0.1)
    assert all(t._version > b for t, b in zip(bases, before))
    w = torch.full((50,), 0.5, device=DEV, requires_grad=True)
    before = w._version
    opt.clip_grads([w.detach(), torch.ones(5, device=DEV)], 0.1)
    assert w._version > before


@pytest.mark.parametrize("call", ["step", "scaled", "schedule", "split"])
def test_the_muon_step_moves_what_it_writes(opt, call):
    P, G, M = ([torch.full((64, 96), 0.25, device=DEV) for _ in range(3)] for _ in range(3))
    G[1] = None
    before, gv = versions(P, M), G[0]._version
    kw = {"scaled": {"grad_scale": torch.ones(1, device=DEV)}, "split": {"row_splits": [32, None, [16, 48]]}}.get(call, {})
    if call == "schedule":
        opt.step_schedule(P, G, M, [muon.DEFAULT_COEFFS] * 2, lr=1e-3)
    else:
        opt.step(P, G, M, lr=1e-3, **kw)
    for old, new in zip(before, versions(P, M)):
        assert new[0] > old[0] and new[2] > old[2] and new[1] == old[1]
    assert G[0]._version == gv


def test_stages_and_qk_clip_move_what_they_write(opt):
    g, m, p, w = (torch.full((64, 96), 0.25, device=DEV) for _ in range(4))
    y, x, s = (muon.x_layout(64, 96, torch.bfloat16, DEV), muon.x_layout(64, 96, torch.bfloat16, DEV),
               torch.zeros(1, dtype=torch.float64, device=DEV))
    old = versions([g, m, y, x, s, p, w])[0]
    opt.momentum_norm([g], [m], [y], s)
    opt.newton_schulz([y], [x], [(64, 96)], sumsq=s)
    opt.apply([p], [x], 1e-3, 0.1)
    opt.qk_clip([w], [torch.full((4,), 200.0, device=DEV)], 16)
    new = versions([g, m, y, x, s, p, w])[0]
    assert new[0] == old[0] and all(b > a for a, b in zip(old[1:], new[1:]))
    opt.momentum_norm([None], [m], [y], s)
    opt.apply([p], [None], 1e-3, 0.1)
    assert m._version == new[1] and p._version == new[5]
