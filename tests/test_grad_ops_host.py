"""Operators on lists of gradients, without a GPU: what the C calls and the
binding refuse, before anything is launched.

The C entry points look at the handle last, so with a NULL handle a good call
says "handle is NULL" and a bad one says what is wrong with it.
"""

import ctypes
import math

import pytest
import torch

import muon_newton_schulz_03_b200 as muon
from muon_newton_schulz_03_b200 import _bad_lists, _check_scalar, _dense, _grad_dtypes, _norm_kind, _sequence

GRAD_SCRATCH_DOUBLES = 65536   # MUON_GRAD_SCRATCH_BYTES(count) = 8 * (65536 + count)
BASE = 1 << 20      # made-up device addresses: nothing reads them
SCRATCH = 8 * (GRAD_SCRATCH_DOUBLES + 16)


def _ptrs(xs):
    return (ctypes.c_void_p * len(xs))(*xs)


def _i64(xs):
    return (ctypes.c_int64 * len(xs))(*xs)


def _i32(xs):
    return (ctypes.c_int32 * len(xs))(*xs)


def _norm(ptrs=(BASE, BASE + 4096), numels=(10, 20), dtypes=(0, 1), count=None, kind=0, max_norm=1.0, out=BASE,
          per=None, scratch=BASE, nbytes=SCRATCH):
    lib = muon.load()
    rc = lib.muon_grad_norm(None, _ptrs(ptrs), _i64(numels), _i32(dtypes), len(ptrs) if count is None else count, kind,
                            max_norm, out, per, scratch, nbytes, None)
    return rc, lib.muon_last_error().decode()


def _clip(src=(BASE, BASE + 4096), dst=(BASE, BASE + 4096), numels=(10, 20), st=(0, 1), dt=(0, 1), kind=0,
          max_norm=1.0, out=BASE + 65536, nbytes=SCRATCH):
    lib = muon.load()
    rc = lib.muon_clip_grads(None, _ptrs(src), _ptrs(dst), _i64(numels), _i32(st), _i32(dt), len(src), kind, max_norm,
                             out, BASE, nbytes, None)
    return rc, lib.muon_last_error().decode()


def _adamw(p=(BASE,), g=(BASE + 4096,), m=(BASE + 8192,), v=(BASE + 12288,), numels=(100,), dtypes=(0,), lr=1e-3,
           b1=0.9, b2=0.999, eps=1e-8, wd=0.1, step=1, step_dev=None, scale=None):
    lib = muon.load()
    rc = lib.muon_adamw_step(None, _ptrs(p), _ptrs(g), _ptrs(m), _ptrs(v), _i64(numels), _i32(dtypes), len(p), lr, b1,
                             b2, eps, wd, step, step_dev, scale, None)
    return rc, lib.muon_last_error().decode()


@pytest.mark.parametrize("kw", [
    {}, {"kind": 1}, {"max_norm": math.inf}, {"max_norm": 0.0}, {"per": BASE}, {"ptrs": (None, BASE)},
    {"scratch": None, "nbytes": 0}, {"numels": (131072, 0), "scratch": None, "nbytes": 0}, {"numels": (200_000, 1)},
    {"numels": (0, 0)}, {"ptrs": (), "numels": (), "dtypes": ()}, {"ptrs": (BASE, BASE)}, {"ptrs": (BASE + 4, BASE + 2)}])
def test_norm_accepts(kw):
    assert _norm(**kw) == (1, "handle is NULL")


@pytest.mark.parametrize("kw,msg", [
    ({"count": -1}, "count"), ({"numels": (10, -1)}, "tensors[1]"), ({"numels": (10, 1 << 41)}, "tensors[1]"),
    ({"numels": (1 << 40, 1 << 40)}, "2^40"), ({"dtypes": (0, 3)}, "tensors[1]"), ({"dtypes": (-1, 0)}, "tensors[0]"),
    ({"ptrs": (BASE + 2, BASE)}, "tensors[0] is not aligned"), ({"ptrs": (BASE, BASE + 1)}, "tensors[1] is not aligned"),
    ({"kind": 2}, "norm_kind"), ({"max_norm": -1.0}, "max_norm"), ({"max_norm": math.nan}, "max_norm"),
    ({"out": None}, "out"), ({"out": BASE + 2}, "out"), ({"per": BASE + 1}, "per_tensor"), ({"numels": (131072, 1), "scratch": None}, "scratch"),
    ({"numels": (200_000, 1), "scratch": BASE + 4}, "scratch"),
    ({"numels": (200_000, 1), "nbytes": 8 * GRAD_SCRATCH_DOUBLES}, "scratch holds")])
def test_norm_refuses(kw, msg):
    rc, text = _norm(**kw)
    assert rc == 1 and msg in text


@pytest.mark.parametrize("kw", [
    {}, {"dst": (BASE + 8192, BASE + 12288)}, {"dst": (BASE + 8192, BASE + 12288), "dt": (1, 0)},
    {"src": (None, BASE), "dst": (None, BASE)}, {"numels": (0, 20), "dst": (None, BASE + 4096)}])
def test_clip_accepts(kw):
    assert _clip(**kw) == (1, "handle is NULL")


@pytest.mark.parametrize("kw,msg", [
    ({"src": (BASE, BASE), "dst": (BASE, BASE)}, "overlaps"),                       # the same tensor twice
    ({"dst": (BASE + 8, BASE + 4096)}, "overlaps"),                                 # shifted copy onto itself
    ({"dst": (BASE + 4096, BASE + 8192)}, "overlaps"),                              # onto another source
    ({"dst": (BASE + 8192, BASE + 8196)}, "overlaps"),                              # two results
    ({"dst": (BASE, None)}, "dst[1] is NULL"), ({"dt": (1, 1)}, "dst[0] is src in another dtype"),
    ({"dt": (0, 5)}, "dst[1]"), ({"dst": (BASE, BASE + 4097)}, "dst[1] is not aligned"), ({"max_norm": -0.5}, "max_norm")])
def test_clip_refuses(kw, msg):
    rc, text = _clip(**kw)
    assert rc == 1 and msg in text


@pytest.mark.parametrize("kw", [{}, {"g": (None,)}, {"numels": (0,), "p": (None,)}, {"step": 0, "step_dev": BASE},
                                {"scale": BASE + 4}, {"b1": 0.0, "b2": 0.0, "eps": 0.0, "wd": 0.0}])
def test_adamw_accepts(kw):
    assert _adamw(**kw) == (1, "handle is NULL")


@pytest.mark.parametrize("kw,msg", [
    ({"p": (None,)}, "params[0] is NULL"), ({"m": (BASE + 8194,)}, "exp_avgs[0] is not aligned"),
    ({"v": (None,)}, "exp_avg_sqs[0]"), ({"m": (BASE,)}, "overlaps"), ({"g": (BASE + 396,)}, "overlaps"),
    ({"v": (BASE + 8192 + 399 // 4 * 4,)}, "overlaps"), ({"lr": math.nan}, "lr"), ({"wd": math.inf}, "wd"),
    ({"b1": 1.0}, "beta1"), ({"b2": -0.1}, "beta1 and beta2"), ({"eps": -1e-8}, "eps"), ({"step": 0}, "step"),
    ({"step_dev": BASE + 4}, "step_dev"), ({"scale": BASE + 2}, "grad_scale"), ({"dtypes": (7,)}, "grads[0]")])
def test_adamw_refuses(kw, msg):
    rc, text = _adamw(**kw)
    assert rc == 1 and msg in text


def test_step_scaled_refuses_a_null_handle():
    lib = muon.load()
    assert lib.muon_step_scaled(None, None, None, None, None, 1, 0.1, 0.9, 1, 0.0, 5, None, 1, None, None) == 1


# -- the binding: dtype, layout and shape are checked before the device, so
#    tensors in host memory reach every check
#    of the function that names the reason (the compiled reader refuses any host
#    tensor at once; its own checks are tested on the device)

def _marshal(ts, *more, device=0):
    """What the binding does with a list: the reader refuses it, then the reason is raised."""
    reader = muon.load_lists()
    if not more:
        assert reader.grad_norm(0, device, ts, 0, 1.0, False) is None
    else:
        assert reader.adamw_step(0, device, ts, *(list(more) * 3)[:3], 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, None) is None
    _bad_lists(device, [("grads", ts, _grad_dtypes())] + [(f"more{k}", m, (torch.float32,))
                                                          for k, m in enumerate(more)])


@pytest.mark.parametrize("bad,exc,msg", [
    (torch.zeros(4, dtype=torch.float64), TypeError, "grads[1] must have dtype"),
    (torch.zeros(4, dtype=torch.int32), TypeError, "grads[1] must have dtype"),
    (torch.zeros(4, 6)[:, :3], ValueError, "grads[1] must be dense"),
    (torch.zeros(8)[::2], ValueError, "grads[1] must be dense"),
    (torch.zeros(1).expand(5), ValueError, "grads[1] must be dense"),
    (torch.zeros(3, 3).to_sparse(), ValueError, "grads[1] must be a strided tensor"),
    (3.0, TypeError, "grads[1] must be a tensor"),
    (torch.zeros(4), ValueError, "grads[1] must be on cuda:0")])
def test_binding_refuses(bad, exc, msg):
    with pytest.raises(exc) as e:
        _marshal([None, bad])
    assert msg in str(e.value)


@pytest.mark.parametrize("partner,exc,msg", [
    (torch.zeros(5, 3), ValueError, "more0[0] shape"), (torch.zeros(3, 5, dtype=torch.bfloat16), TypeError, "more0[0]"),
    (torch.zeros(5, 3).t(), ValueError, "more0[0] has strides"), (None, TypeError, "more0[0] must be a tensor")])
def test_binding_refuses_partners(partner, exc, msg, monkeypatch):
    real = muon._check_tensor

    def no_device(t, what, dtypes, device, like=None):   # the first list's tensor counts as on the device
        if like is None:
            return
        real(t, what, dtypes, device, like)

    monkeypatch.setattr(muon, "_check_tensor", no_device)
    with pytest.raises(exc) as e:
        _marshal([torch.zeros(3, 5)], [partner])
    assert msg in str(e.value)


def test_binding_refuses_other_lengths_and_norms():
    with pytest.raises(ValueError):
        _marshal([None, None], [None])
    with pytest.raises(ValueError):
        _norm_kind(1)
    assert _norm_kind(2) == _norm_kind(2.0) == 0 and _norm_kind(math.inf) == 1


@pytest.mark.parametrize("t", [torch.zeros(2), torch.zeros(1, dtype=torch.float64), torch.zeros(1)])
def test_binding_refuses_scalars(t):
    with pytest.raises(ValueError):
        _check_scalar(t, "grad_scale", torch.float32, 0)
    assert _check_scalar(None, "grad_scale", torch.float32, 0) is None


@pytest.mark.parametrize("t,ok", [
    (torch.zeros(3, 4), True), (torch.zeros(3, 4).t(), True), (torch.zeros(2, 3, 4).permute(2, 0, 1), True),
    (torch.zeros(2, 3, 4, 5).contiguous(memory_format=torch.channels_last), True), (torch.zeros(()), True),
    (torch.zeros(0, 4), True), (torch.zeros(4, 4)[:, :2], False), (torch.zeros(4, 4)[::2], False),
    (torch.zeros(3, 1).expand(3, 2), False), (torch.zeros(5, 4)[1:3], True), (torch.zeros(4, 4)[:, :1], False)])
def test_dense(t, ok):
    assert _dense(t) is ok


def test_reader_refuses_bad_arguments():
    reader = muon.load_lists()
    for bad in (5, None, [None]):
        assert reader.adamw_step(0, 0, bad, [], [], [], 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, None) is None
    with pytest.raises(TypeError):
        reader.grad_norm(0, 0)
    with pytest.raises(TypeError):
        reader.adamw_step(0, 0, [], [], [], [], "x", 0.9, 0.999, 1e-8, 0.0, 1, None)
    with pytest.raises(TypeError):
        reader.adamw_step(0, 0, [], [], [], [], 1e-3, 0.9, 0.999, 1e-8, 0.0, 1.5, None)
    for scale in (torch.ones(1), 1.0):           # not a CUDA tensor
        assert reader.adamw_step(0, 0, [], [], [], [], 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, scale) is None
    assert reader.adamw_step(0, 0, [], [], [], [], 1e-3, 0.9, 0.999, 1e-8, 0.0, torch.ones(1), None) is None
    with pytest.raises(TypeError):
        reader.clip_grads("handle", 0, [], [], 0, 1.0)


def test_a_bare_tensor_is_not_a_list():
    with pytest.raises(TypeError):
        _sequence(torch.zeros(3, 4))
    a = [torch.zeros(2)]
    assert _sequence(a) is a and _sequence(iter(a)) == a
    for bad in (1.0, torch.ones(2), torch.ones(1, dtype=torch.float64)):
        with pytest.raises(ValueError):
            _check_scalar(bad, "grad_scale", torch.float32, 0)
