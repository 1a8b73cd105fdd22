"""Which stream a call takes when it is given none (no GPU): the current one of
the handle's device, in every method, whatever the current device is. The norm's
multiplier and the step that reads it are then ordered by their stream."""

import ctypes

import pytest
import torch

import muon_newton_schulz_03_b200 as muon

STREAMS = {0: 0x1000, 1: 0x2000}     # each device's current stream


class _Stream:
    def __init__(self, device):
        self.cuda_stream = STREAMS[device]


class _Lib:
    """Takes every C call and keeps the streams that the calls were given."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            at = 1 if name == "muon_get_status" else len(args) - 1     # (handle, stream, results) there
            self.streams.append(args[at].value)
            return 0
        return call


@pytest.fixture
def opt(monkeypatch):
    # Device 0 is current, the handle is on device 1.
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream(0 if device is None else device))
    o = object.__new__(muon.Muon)
    o._lib, o._h, o._hv, o.device, o.ns_precision = _Lib(), ctypes.c_void_p(1), 1, 1, "bf16"
    yield o
    o._h = None


CALLS = {
    "step": lambda o, **kw: o.step([], [], [], lr=0.1, **kw),
    "step_schedule": lambda o, **kw: o.step_schedule([], [], [], [muon.DEFAULT_COEFFS], lr=0.1, **kw),
    "step_host": lambda o, **kw: o.step_host([], [], [], lr=0.1, **kw),
    "qk_clip": lambda o, **kw: o.qk_clip([], [], 1, **kw),
    "newton_schulz": lambda o, **kw: o.newton_schulz([], [], [], **kw),
    "apply": lambda o, **kw: o.apply([], [], 0.1, 0.1, **kw),
    "status": lambda o, **kw: o.status(**kw),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_default_stream_is_the_handles_devices(opt, name):
    CALLS[name](opt)
    assert opt._lib.streams == [STREAMS[1]]


def test_default_stream_of_momentum_norm(opt, monkeypatch):
    monkeypatch.setattr(opt, "_check_sumsq", lambda *a: None, raising=False)
    opt.momentum_norm([], [], [], torch.zeros(1, dtype=torch.float64))
    assert opt._lib.streams == [STREAMS[1]]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_given_stream_is_taken_as_it_is(opt, name):
    CALLS[name](opt, stream=_Stream(0))
    assert opt._lib.streams == [STREAMS[0]]


def test_the_scaled_step_takes_the_same_stream(opt, monkeypatch):
    monkeypatch.setattr(muon, "_check_scalar", lambda t, what, dtype, device: 0x40)
    opt.step([], [], [], lr=0.1, grad_scale=torch.ones(1))
    assert opt._lib.streams == [STREAMS[1]]
