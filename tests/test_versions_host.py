"""What a step writes in place counts as written to autograd: the version
counters of its tensors move (no GPU: the host-buffer step over a C library
that does nothing)."""

import ctypes

import pytest
import torch

import muon_newton_schulz_03_b200 as muon


class _Lib:
    status = 0

    def __getattr__(self, name):
        return lambda *args: self.status


class _Stream:
    cuda_stream = 0


@pytest.fixture
def opt(monkeypatch):
    monkeypatch.setattr(muon, "check", lambda rc: _raise(rc) if rc else None)
    o = object.__new__(muon.Muon)
    o._lib, o._h, o._hv, o.device, o.ns_precision = _Lib(), ctypes.c_void_p(1), 1, 0, "bf16"
    yield o
    o._h = None


def _raise(rc):
    raise RuntimeError(rc)


def test_step_host_moves_what_it_writes(opt):
    P, G, M = ([torch.zeros(3, 4) for _ in range(3)] for _ in range(3))
    with torch.inference_mode():
        P.append(torch.zeros(2, 2)), G.append(torch.zeros(2, 2)), M.append(torch.zeros(2, 2))   # no counter
    G[1] = None
    before = [[t._version for t in ts[:3] if t is not None] for ts in (P, G, M)]
    opt.step_host(P, G, M, lr=0.1, stream=_Stream())
    for ts, old in ((P, before[0]), (M, before[2])):
        assert ts[0]._version > old[0] and ts[2]._version > old[2]
        assert ts[1]._version == old[1]                              # skipped
    assert [t._version for t in G[:3] if t is not None] == before[1]


def test_a_failed_call_moves_nothing(opt):
    P, G, M = ([torch.zeros(3, 4)] for _ in range(3))
    opt._lib.status = 3
    with pytest.raises(RuntimeError):
        opt.step_host(P, G, M, lr=0.1, stream=_Stream())
    assert P[0]._version == M[0]._version == 0


def test_a_graph_over_old_parameters_raises(opt):
    w = torch.ones(3, 4, requires_grad=True)
    loss = (w * w).sum()
    opt.step_host([w], [torch.ones(3, 4)], [torch.zeros(3, 4)], lr=0.1, stream=_Stream())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_iterators_are_lists_too(opt):
    P, G, M = ([torch.zeros(3, 4), torch.zeros(2, 2)] for _ in range(3))
    opt.step_host(iter(P), (g for g in G), iter(M), lr=0.1, stream=_Stream())
    assert all(t._version > 0 for t in P + M) and all(t._version == 0 for t in G)
