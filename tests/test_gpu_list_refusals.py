"""What the compiled reader of tensor lists refuses of CUDA tensors: the type,
density, shape, strides and length checks behind its device check, which host
tensors never reach. Nothing is written by a refused call."""

import pytest
import torch

import muon_newton_schulz_03_b200 as muon

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def opt():
    with muon.Muon(device=0) as o:
        yield o


def full(*shape, dtype=torch.float32):
    return torch.full(shape, 0.5, dtype=dtype, device=DEV)


# name: (a tensor that is no entry of a list by itself, the error, words of its message)
SINGLE = {
    "float64": (lambda: full(4, 6, dtype=torch.float64), TypeError, "must have dtype"),
    "int32": (lambda: full(4, 6).int(), TypeError, "must have dtype"),
    "bool": (lambda: full(4, 6).bool(), TypeError, "must have dtype"),
    "complex": (lambda: full(4, 6, dtype=torch.complex64), TypeError, "must have dtype"),
    "columns": (lambda: full(4, 12)[:, :6], ValueError, "must be dense"),
    "every other row": (lambda: full(8, 6)[::2], ValueError, "must be dense"),
    "expanded": (lambda: full(1, 6).expand(4, 6), ValueError, "must be dense"),
    "overlapping": (lambda: full(9).as_strided((4, 6), (1, 1)), ValueError, "must be dense"),
    "sparse": (lambda: full(4, 6).to_sparse(), ValueError, "strided"),
    "negated view": (lambda: torch._neg_view(full(4, 6)), ValueError, "must be dense"),
    "host": (lambda: full(4, 6).cpu(), ValueError, "must be on cuda:0"),
    "number": (lambda: 0.5, TypeError, "must be a tensor"),
}

# name: (a partner of a 4 x 6 tensor, the error, words of its message)
PARTNER = {
    "shape": (lambda: full(6, 4), ValueError, "shape"),
    "fewer dimensions": (lambda: full(24), ValueError, "shape"),
    "longer": (lambda: full(4, 7), ValueError, "shape"),
    "transposed": (lambda: full(6, 4).t(), ValueError, "strides"),
    "none": (lambda: None, TypeError, "must be a tensor"),
    **{k: SINGLE[k] for k in ("float64", "columns", "expanded", "sparse", "host")},
}


def untouched(*lists):
    return all(t is None or not isinstance(t, torch.Tensor) or t.device.type == "cpu" or
               bool((t.to_dense() == t.new_tensor(0.5).to(t.dtype)).all()) for ts in lists for t in ts)


@pytest.mark.parametrize("name", sorted(SINGLE))
def test_an_entry_that_is_no_dense_cuda_tensor(opt, name):
    make, exc, words = SINGLE[name]
    bad, good = make(), full(4, 6)
    for call, what in ((lambda: opt.grad_norm([good, None, bad], max_norm=0.1), "tensors[2]"),
                       (lambda: opt.clip_grads([good, None, bad], 0.1), "grads[2]"),
                       (lambda: opt.adamw_step([good, None, full(4, 6)], [full(4, 6), None, bad],
                                               [full(4, 6), None, full(4, 6)], [full(4, 6), None, full(4, 6)], lr=0.1,
                                               step=1), "grads[2]")):
        with pytest.raises(exc) as e:
            call()
        assert what in str(e.value) and words in str(e.value)
    assert untouched([good])


@pytest.mark.parametrize("name", sorted(PARTNER))
@pytest.mark.parametrize("at", [0, 1, 2])
def test_a_partner_that_does_not_match(opt, name, at):
    make, exc, words = PARTNER[name]
    lists = [[full(4, 6), full(4, 6)] for _ in range(3)]
    lists[at][1] = make()
    g = [full(4, 6), full(4, 6, dtype=torch.bfloat16)]
    with pytest.raises(exc) as e:
        opt.adamw_step(lists[0], g, lists[1], lists[2], lr=0.1, step=1)
    assert ("params", "exp_avgs", "exp_avg_sqs")[at] + "[1]" in str(e.value) and words in str(e.value)
    with pytest.raises(exc) as e:
        opt.clip_grads(g, 0.1, out=lists[at])
    assert "out[1]" in str(e.value) and words in str(e.value)
    assert untouched(g, *lists)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_state_in_16_bits(opt, dtype, at):
    lists = [[full(4, 6)] for _ in range(3)]
    lists[at][0] = full(4, 6, dtype=dtype)
    with pytest.raises(TypeError) as e:
        opt.adamw_step(lists[0], [full(4, 6)], lists[1], lists[2], lr=0.1, step=1)
    assert "must have dtype" in str(e.value) and untouched(*lists)


@pytest.mark.parametrize("at", [0, 1, 2, 3])
def test_lists_of_other_lengths(opt, at):
    lists = [[full(4, 6), full(4, 6)] for _ in range(4)]
    for other in (lists[at][:1], lists[at] + [full(4, 6)]):
        args = lists[:at] + [other] + lists[at + 1:]
        with pytest.raises(ValueError) as e:
            opt.adamw_step(*args, lr=0.1, step=1)
        assert "entries" in str(e.value)
    with pytest.raises(ValueError):
        opt.clip_grads(lists[0], 0.1, out=lists[1][:1])
    assert untouched(*lists)


def test_a_transposed_row_against_contiguous_ones(opt):
    # The first of a row sets the layout: all of it transposed is taken, one of it is not.
    t = [full(6, 4).t() for _ in range(4)]
    opt.adamw_step([t[0]], [t[1]], [t[2]], [t[3]], lr=0.1, step=1)
    for at in range(4):
        row = [full(6, 4).t() for _ in range(4)]
        row[at] = full(4, 6)
        with pytest.raises(ValueError) as e:
            opt.adamw_step(*([x] for x in row), lr=0.1, step=1)
        assert "strides" in str(e.value) and untouched(row)


def test_one_layout_by_other_strides_is_taken(opt):
    # A dimension of one element has any stride; the others say where the elements are.
    def make(first):
        t = full(15)
        t[:] = torch.arange(15, device=DEV) / 8
        return t.as_strided((1, 5, 3), (first, 1, 5))
    g, out = [make(15)], [make(7)]
    opt.clip_grads(g, 1.0, out=out)
    whole = g[0].clone()
    opt.clip_grads([whole], 1.0)
    assert torch.equal(out[0], whole)
    p, m, v = make(1), make(99), make(15)
    q, n, w = p.clone(), m.clone(), v.clone()
    opt.adamw_step([p], g, [m], [v], lr=0.1, step=2)
    opt.adamw_step([q], [g[0].clone()], [n], [w], lr=0.1, step=2)
    assert torch.equal(p, q) and torch.equal(m, n) and torch.equal(v, w)
