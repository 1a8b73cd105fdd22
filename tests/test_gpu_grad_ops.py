"""Operators on lists of gradients against their definitions in 64 bits.

Tolerances count roundings (u = 2^-24, half an fp32 step; half a step of the
written type for its last rounding):
* norm: fp32 gradients are summed in fp64, so the result is one rounding off;
  16-bit ones are added in sixteens in fp32 (two sums of eight, joined: their
  products are exact, so at most 8 roundings), 8 u on the sum and 4 u on its
  root, and one rounding more. Magnitudes are exact.
* multiplier: the norm's error and one rounding; clipped values: that, one
  fp32 product, one rounding to the written type (an absolute half step below
  its smallest normal number).
* AdamW: see ``adamw_bounds``.
"""

import math

import numpy as np
import pytest
import torch

import muon_newton_schulz_03_b200 as muon
from oracle import muon_oracle as O

from gpu_helpers import DEV, TOL_FP32_NS, rel, to64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SIZES = [1, 0, 3, 7, 8, 9, 31, 255, 2047, 2048, 2049, 8191, 8193, 100_003]


@pytest.fixture(scope="module")
def opt():
    with muon.Muon(device=0) as o:
        yield o


def tensors(sizes, dtypes, seed=0, offset=0, scale=1.0):
    """Views into one buffer per tensor, `offset` elements from its start."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        buf = torch.randn(n + offset + 8, generator=gen, device=DEV).mul_(scale).to(dtypes[i % len(dtypes)])
        out.append(buf[offset:offset + n])
    return out


def exact_norm(ts, kind=2.0):
    per = [t.double().abs().max().item() if t.numel() and kind == math.inf else t.double().norm().item() for t in ts]
    return (max(per, default=0.0) if kind == math.inf else math.sqrt(sum(x * x for x in per))), per


def norm_tol(ts, kind):
    if kind == math.inf:
        return 0.0
    return (5.0 if any(t.dtype != F32 for t in ts) else 1.0) * U * 1.001


def clip_of(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))


def half_step(dtype):
    """(relative, absolute) size of one rounding to a type."""
    f = torch.finfo(dtype)
    return f.eps / 2, f.tiny * f.eps / 2


def assert_clipped(got, src, s, tol_s, what=""):
    r, a = half_step(got.dtype)
    want = src.double() * s
    off = (got.double() - want).abs() - ((r + tol_s + 2 * U) * want.abs() + a)
    assert got.numel() == 0 or off.max().item() <= 0, f"{what}: {off.max().item():.3e} over the bound"


@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F16,), (F32, BF16, F16)])
@pytest.mark.parametrize("offset", [0, 1, 5])
def test_norm(opt, dtypes, kind, offset):
    ts = tensors(SIZES, dtypes, seed=3, offset=offset)
    norm, scale, per = opt.grad_norm(ts, max_norm=2.0, norm_type=kind, per_tensor=True)
    want, want_per = exact_norm(ts, kind)
    tol = norm_tol(ts, kind)
    assert abs(norm.item() - want) <= tol * want
    for i, (x, w) in enumerate(zip(per.tolist(), want_per)):
        assert abs(x - w) <= tol * w, (i, x, w)
    s = clip_of(want, 2.0)
    assert abs(scale.item() - s) <= (tol + 2 * U) * s
    assert norm.dtype == scale.dtype == per.dtype == F32 and norm.dim() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mag", [1e-30, 1e30])
def test_norm_beyond_the_range_of_fp32_squares(opt, dtype, mag):
    # 1e30 squared overflows fp32 and 1e-30 squared vanishes there.
    ts = tensors([5, 4097], (dtype,), seed=4, scale=mag)
    norm, _ = opt.grad_norm(ts)
    want, _ = exact_norm(ts)
    assert abs(norm.item() - want) <= 5.0 * U * 1.001 * want


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("n,at", [(1, 0), (9, 8), (20_000, 8192), (20_000, 19_999)])
def test_norm_of_nan_and_infinity(opt, dtype, kind, n, at):
    good, bad = tensors([300, n], (dtype,), seed=5)
    bad[at] = -math.inf
    norm, scale = opt.grad_norm([good, bad], max_norm=1.0, norm_type=kind)
    assert norm.item() == math.inf and scale.item() == 0.0
    good[7] = math.nan
    norm, scale, per = opt.grad_norm([good, bad], max_norm=1.0, norm_type=kind, per_tensor=True)
    assert math.isnan(norm.item()) and math.isnan(scale.item())
    assert math.isnan(per[0].item()) and per[1].item() == math.inf
    assert opt.grad_norm([bad])[1].item() == 1.0       # no bound, no clipping


def test_norm_of_nothing_and_skipped(opt):
    for ts in ([], [None], [None, torch.zeros(0, device=DEV)], [torch.zeros(1000, device=DEV)]):
        norm, scale, per = opt.grad_norm(ts, max_norm=1.0, per_tensor=True)
        assert norm.item() == 0.0 and scale.item() == 1.0 and per.tolist() == [0.0] * len(ts)
    a, b = tensors([50, 70], (F32,))
    norm, _, per = opt.grad_norm([a, None, b, None], per_tensor=True)
    want, (wa, wb) = exact_norm([a, b])
    assert abs(norm.item() - want) <= U * 1.001 * want and per[1].item() == per[3].item() == 0.0
    assert abs(per[2].item() - wb) <= U * 1.001 * wb


@pytest.mark.parametrize("count", [64, 65, 256, 257, 512, 513, 704, 705, 1088, 1089, 1536, 1537, 3100])
def test_lists_longer_than_a_launch(opt, count):
    rng = np.random.default_rng(count)
    ts = tensors(rng.integers(0, 40, count).tolist(), (BF16, F32), seed=6, offset=1)
    norm, scale, per = opt.grad_norm(ts, max_norm=1.0, per_tensor=True)
    want, want_per = exact_norm(ts)
    assert abs(norm.item() - want) <= norm_tol(ts, 2.0) * want
    np.testing.assert_allclose(per.cpu().numpy(), want_per, rtol=norm_tol(ts, 2.0), atol=0)
    before = [t.clone() for t in ts]
    opt.clip_grads(ts, 1.0)
    for t, b in zip(ts, before):
        assert_clipped(t, b, clip_of(want, 1.0), norm_tol(ts, 2.0) + U)


@pytest.mark.parametrize("count,total", [(512, 131_072), (512, 131_073), (513, 131_072), (1, 131_072), (1, 131_073),
                                         (256, 131_072), (257, 131_072)])
@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_around_the_small_lists_limits(opt, count, total, kind):
    # One kernel up to 512 tensors and 2^17 elements, several above; units of
    # 1024 elements, one more per tensor at most.
    sizes = [total // count] * (count - 1)
    sizes.append(total - sum(sizes))
    ts = tensors(sizes, (BF16, F32), seed=7, offset=3)
    before = [t.clone() for t in ts]
    norm, scale, per = opt.grad_norm(ts, max_norm=1.0, norm_type=kind, per_tensor=True)
    want, want_per = exact_norm(ts, kind)
    assert abs(norm.item() - want) <= norm_tol(ts, kind) * want
    np.testing.assert_allclose(per.cpu().numpy(), want_per, rtol=norm_tol(ts, kind), atol=0)
    opt.clip_grads(ts, 0.5 * want, norm_type=kind)
    for t, b in zip(ts, before):
        assert_clipped(t, b, clip_of(want, 0.5 * want), norm_tol(ts, kind) + U)


@pytest.mark.parametrize("src", [F32, BF16, F16])
@pytest.mark.parametrize("dst", [None, F32, BF16, F16])
@pytest.mark.parametrize("offsets", [(0, 0), (1, 1), (3, 6), (4, 0)])
def test_clip(opt, src, dst, offsets):
    ts = tensors(SIZES, (src,), seed=8, offset=offsets[0])
    before = [t.clone() for t in ts]
    want, _ = exact_norm(ts)
    bufs = [torch.full((t.numel() + 16,), 7.0, dtype=dst or src, device=DEV) for t in ts]
    outs = None if dst is None else [b[offsets[1]:offsets[1] + t.numel()] for b, t in zip(bufs, ts)]
    norm = opt.clip_grads(ts, 0.5 * want, out=outs)
    tol = norm_tol(ts, 2.0)
    assert abs(norm.item() - want) <= tol * want
    for i, b in enumerate(before):
        assert_clipped((outs or ts)[i], b, clip_of(want, 0.5 * want), tol + U, f"tensor {i}")
        if dst is not None:
            assert torch.equal(ts[i], b)                                 # the source stays
            o, n = offsets[1], b.numel()
            assert (bufs[i][:o] == 7).all() and (bufs[i][o + n:] == 7).all()   # nothing beside it is written


@pytest.mark.parametrize("dst", [None, BF16])
def test_clip_inside_the_bound_changes_nothing(opt, dst):
    ts = tensors(SIZES, (BF16,), seed=9)
    before = [t.clone() for t in ts]
    outs = None if dst is None else [torch.zeros_like(t) for t in ts]
    opt.clip_grads(ts, 1e4, out=outs)
    for t, b in zip(outs or ts, before):
        assert torch.equal(t, b)


def test_clip_to_zero_and_of_nonfinite(opt):
    t = tensors([1000], (F32,))[0]
    t[3] = math.inf
    opt.clip_grads([t], 1.0)
    assert math.isnan(t[3].item()) and (t[:3] == 0).all() and (t[4:] == 0).all()    # 0 * inf
    t = tensors([1000], (F32,))[0]
    opt.clip_grads([t], 0.0)
    assert (t == 0).all()


@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_permuted_and_shaped_tensors(opt, kind):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    x = torch.randn(6, 5, 4, 3, generator=gen, device=DEV)
    ts = [x.contiguous(memory_format=torch.channels_last), torch.randn(33, 17, generator=gen, device=DEV).t(),
          torch.randn((), generator=gen, device=DEV), torch.randn(1, 9, 1, generator=gen, device=DEV)]
    before = [t.clone() for t in ts]
    want, _ = exact_norm(ts, kind)
    norm = opt.clip_grads(ts, 0.25 * want, norm_type=kind)
    assert abs(norm.item() - want) <= U * 1.001 * want
    for t, b in zip(ts, before):
        assert_clipped(t, b, clip_of(want, 0.25 * want), 2 * U)


# -- AdamW ------------------------------------------------------------------

def adamw64(p, g, m, v, lr, step, betas, eps, wd, s, more=0):
    """The definition in 64 bits, and how far fp32 may be from it.

    m' = b1 m + (1 - b1) g: the constants, g's scaling, the product and the sum
    are 5 roundings of its two terms (which may cancel). v' has no cancelling
    terms: 7 roundings. The quotient's denominator: half of v's, the root, the
    correction, its product and eps: 7; the quotient, the step size and the
    product with it: 3 more. p': the decay factor, its product, the sum.
    A step number on the device: its factors are made in fp32, 4 roundings
    more in the step size and 2.5 in the correction (``more`` = 6.5)."""
    b1, b2 = betas
    g = g.double() * s
    m1 = b1 * m.double() + (1 - b1) * g
    v1 = b2 * v.double() + (1 - b2) * g * g
    den = (v1 / (1 - b2 ** step)).sqrt() + eps
    lr1 = lr / (1 - b1 ** step)
    d = lr1 * m1 / den
    p64 = p.double()
    p1 = p64 * (1 - lr * wd) - d
    tiny = torch.finfo(F32).tiny * torch.finfo(F32).eps
    tm = 5 * U * ((b1 * m.double()).abs() + ((1 - b1) * g).abs()) + tiny
    tv = 7 * U * v1 + tiny
    tp = 2 * U * p64.abs() + lr1 * tm / den + (10 + more) * U * d.abs() + U * p1.abs() + tiny
    # a v that fell below fp32's normal range moves the root by up to sqrt(tiny)
    tp = tp + torch.where(v1 < torch.finfo(F32).tiny, (d * math.sqrt(torch.finfo(F32).tiny) / den).abs(), 0.0 * d)
    return (p1, m1, v1), (tp, tm, tv)


def check_adamw(got, want, tol):
    for name, x, w, t in zip("pmv", got, want, tol):
        off = (x.double() - w).abs() - t
        assert x.numel() == 0 or off.max().item() <= 0, f"{name}: {off.max().item():.3e} over the bound"


def adam_state(sizes, gtypes, seed, offset=0, first=False):
    g = tensors(sizes, gtypes, seed, offset, 1e-2)
    p = tensors(sizes, (F32,), seed + 1, offset, 0.02)
    m = tensors(sizes, (F32,), seed + 2, offset, 0.0 if first else 1e-3)
    v = [t.square_() for t in tensors(sizes, (F32,), seed + 3, offset, 0.0 if first else 1e-2)]
    return p, g, m, v


@pytest.mark.parametrize("gtypes", [(F32,), (BF16,), (F16,), (BF16, F32, F16)])
@pytest.mark.parametrize("step,scale,offset", [(1, None, 0), (7, 0.3, 1), (100_000, 0.5, 4)])
def test_adamw(opt, gtypes, step, scale, offset):
    p, g, m, v = adam_state(SIZES, gtypes, 11, offset, first=step == 1)
    old = [[t.clone() for t in ts] for ts in (p, m, v)]
    gs = None if scale is None else torch.tensor([scale], device=DEV)
    hyper = dict(lr=3e-4, step=step, betas=(0.9, 0.95), eps=1e-8, wd=0.1)
    opt.adamw_step(p, g, m, v, grad_scale=gs, **hyper)
    s = 1.0 if gs is None else gs.item()
    for i in range(len(SIZES)):
        want, tol = adamw64(old[0][i], g[i], old[1][i], old[2][i], s=s, **hyper)
        check_adamw((p[i], m[i], v[i]), want, tol)


@pytest.mark.parametrize("offsets", [(0, 1, 2, 3), (0, 0, 0, 4), (1, 5, 1, 5)])
@pytest.mark.parametrize("gtype", [F32, BF16])
def test_adamw_with_unequal_alignments(opt, offsets, gtype):
    n = 5001
    ts = [tensors([n], (F32 if k != 1 else gtype,), 20 + k, o, 1e-2)[0] for k, o in enumerate(offsets)]
    p, g, m, v = ts
    v.square_()
    old = (p.clone(), m.clone(), v.clone())
    hyper = dict(lr=1e-3, step=3, betas=(0.9, 0.999), eps=1e-8, wd=0.0)
    opt.adamw_step([p], [g], [m], [v], **hyper)
    want, tol = adamw64(old[0], g, old[1], old[2], s=1.0, **hyper)
    check_adamw((p, m, v), want, tol)


@pytest.mark.parametrize("gtype,offset", [(F32, 0), (BF16, 3)])
def test_adamw_leaves_everything_else(opt, gtype, offset):
    n = 2049
    bufs = [torch.full((n + 32,), 5.0, device=DEV) for _ in range(3)]
    views = [b[offset:offset + n] for b in bufs]
    for x in views:
        x.fill_(0.25)
    g = torch.full((n + 32,), 0.5, device=DEV).to(gtype)[offset:offset + n]
    keep = torch.full((10,), 3.0, device=DEV)
    k2, k3 = keep.clone(), keep.clone()
    opt.adamw_step([views[0], keep], [g, None], [views[1], k2], [views[2], k3], lr=1e-3, step=2)
    for b in bufs:
        assert (b[:offset] == 5).all() and (b[offset + n:] == 5).all()
    # v' = 0.999 * 0.25 + 0.001 * 0.5^2 = 0.25, the old value; p and m move everywhere
    assert not (views[0] == 0.25).any() and not (views[1] == 0.25).any()
    assert ((views[2] - 0.25).abs() <= 7 * U * 0.25).all()
    assert (keep == 3).all() and (k2 == 3).all() and (k3 == 3).all()


@pytest.mark.parametrize("count", [64, 65, 257, 513, 705, 1500])
def test_adamw_of_many(opt, count):
    rng = np.random.default_rng(count)
    sizes = rng.integers(0, 50, count).tolist()
    p, g, m, v = adam_state(sizes, (F32, BF16), 31, 2)
    old = [[t.clone() for t in ts] for ts in (p, m, v)]
    hyper = dict(lr=1e-3, step=5, betas=(0.9, 0.95), eps=1e-6, wd=0.1)
    opt.adamw_step(p, g, m, v, **hyper)
    for i in range(count):
        want, tol = adamw64(old[0][i], g[i], old[1][i], old[2][i], s=1.0, **hyper)
        check_adamw((p[i], m[i], v[i]), want, tol)


def test_adamw_of_zero_and_nan_gradients(opt):
    p, g, m, v = adam_state([600], (F32,), 40, first=True)
    g[0].zero_()
    g[0][5] = math.nan
    p0 = p[0].clone()
    opt.adamw_step(p, g, m, v, lr=1e-2, step=1, wd=0.1)
    want, tol = adamw64(p0, torch.zeros_like(p0), m[0].new_zeros(600), m[0].new_zeros(600), 1e-2, 1, (0.9, 0.999),
                        1e-8, 0.1, 1.0)
    ok = torch.arange(600, device=DEV) != 5
    check_adamw((p[0][ok], m[0][ok], v[0][ok]), [w[ok] for w in want], [t[ok] for t in tol])
    assert all(math.isnan(t[0][5].item()) for t in (p, m, v))


def test_adamw_permuted(opt):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    p, g, m, v = (torch.randn(31, 45, generator=gen, device=DEV).t() for _ in range(4))
    v.abs_()
    old = (p.clone(), m.clone(), v.clone())
    opt.adamw_step([p], [g], [m], [v], lr=1e-3, step=2)
    want, tol = adamw64(old[0], g, old[1], old[2], 1e-3, 2, (0.9, 0.999), 1e-8, 0.1, 1.0)
    check_adamw((p, m, v), want, tol)


# -- streams, graphs, repeated and simultaneous calls ------------------------

def test_results_repeat_bit_for_bit(opt):
    ts = tensors([1_000_003, 17, 65_537], (BF16, F32), seed=50)
    first = opt.grad_norm(ts, max_norm=1.0, per_tensor=True)
    for _ in range(5):
        again = opt.grad_norm(ts, max_norm=1.0, per_tensor=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_calls_on_two_streams_at_once(opt):
    a = tensors([3_000_001, 5], (F32,), seed=51)
    b = tensors([2_000_003, 11, 7], (BF16,), seed=52)
    want = [exact_norm(x)[0] for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, ts in enumerate((a, b)):
            got[k].append(opt.grad_norm(ts, stream=streams[k])[0])
    torch.cuda.synchronize()
    for k, ts in enumerate((a, b)):
        assert all(abs(x.item() - want[k]) <= norm_tol(ts, 2.0) * want[k] for x in got[k])


@pytest.mark.parametrize("sizes", [[3000, 17], [2_000_003, 17]])
def test_calls_on_a_given_stream(opt, sizes):
    p, g, m, v = adam_state(sizes, (BF16,), 55, 1)
    old = [[t.clone() for t in ts] for ts in (p, m, v)]
    before = [t.clone() for t in g]
    out = [torch.empty_like(t) for t in g]
    want, _ = exact_norm(g)
    hyper = dict(lr=1e-3, step=4, betas=(0.9, 0.95), eps=1e-8, wd=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm, scale, per = opt.grad_norm(g, max_norm=0.5 * want, per_tensor=True, stream=side)
    opt.clip_grads(g, 0.5 * want, out=out, stream=side)
    opt.adamw_step(p, out, m, v, stream=side, **hyper)
    junk = [torch.full((70_000 + k,), 9.0, device=DEV) for k in range(50)]   # the current stream's memory moves on
    torch.cuda.current_stream().wait_stream(side)
    assert abs(norm.item() - want) <= norm_tol(g, 2.0) * want and per.numel() == len(g)
    for i, b in enumerate(before):
        assert_clipped(out[i], b, clip_of(want, 0.5 * want), norm_tol(g, 2.0) + U)
        w, tol = adamw64(old[0][i], out[i], old[1][i], old[2][i], s=1.0, **hyper)
        check_adamw((p[i], m[i], v[i]), w, tol)
    assert all((j == 9).all() for j in junk)
    assert abs(scale.item() - clip_of(want, 0.5 * want)) <= 7.0 * U


def test_one_gradient_for_two_parameters(opt):
    # Read twice, written never: allowed; it counts twice in the norm.
    p, g, m, v = adam_state([900, 900], (F32,), 56)
    g[1] = g[0]
    old = [[t.clone() for t in ts] for ts in (p, m, v)]
    norm, _ = opt.grad_norm(g)
    assert abs(norm.item() - math.sqrt(2.0) * exact_norm(g[:1])[0]) <= 2 * U * norm.item()
    opt.adamw_step(p, g, m, v, lr=1e-3, step=2)
    for i in range(2):
        w, tol = adamw64(old[0][i], g[0], old[1][i], old[2][i], 1e-3, 2, (0.9, 0.999), 1e-8, 0.1, 1.0)
        check_adamw((p[i], m[i], v[i]), w, tol)


def test_many_separate_tensors_in_any_order(opt):
    # Addresses in no order: the overlap check sorts them.
    sizes = np.random.default_rng(3).integers(1, 30_000, 300).tolist()
    p, g, m, v = adam_state(sizes, (F32, F16), 57)
    order = np.random.default_rng(4).permutation(len(sizes))
    p, g, m, v = ([ts[i] for i in order] for ts in (p, g, m, v))
    old = [[t.clone() for t in ts] for ts in (p, m, v)]
    opt.adamw_step(p, g, m, v, lr=1e-3, step=2)
    for i in range(0, len(p), 17):
        w, tol = adamw64(old[0][i], g[i], old[1][i], old[2][i], 1e-3, 2, (0.9, 0.999), 1e-8, 0.1, 1.0)
        check_adamw((p[i], m[i], v[i]), w, tol)
    with pytest.raises(muon.MuonError):
        opt.adamw_step(p + [p[150]], g + [g[150]], m + [m[150].clone()], v + [v[150].clone()], lr=1e-3, step=2)
    with pytest.raises(muon.MuonError):
        opt.clip_grads(g[:200] + [g[7][1:]], 1.0)


def test_two_captured_graphs_replayed_in_turn(opt):
    lists = [tensors([70_001, 40], (F32,), seed=53), tensors([900, 123_457], (BF16,), seed=54)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for ts in lists:
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            outs.append(opt.grad_norm(ts, max_norm=1.0, per_tensor=True))
        graphs.append(g)
    for k in (1, 0, 1, 0):
        for t in lists[k]:
            t.mul_(1.5)
        graphs[k].replay()
        graphs[1 - k].replay()
        torch.cuda.synchronize()
        for ts, (norm, scale, per) in zip(lists, outs):
            want, want_per = exact_norm(ts)
            assert abs(norm.item() - want) <= norm_tol(ts, 2.0) * want
            np.testing.assert_allclose(per.cpu().numpy(), want_per, rtol=norm_tol(ts, 2.0), atol=0)
    del graphs


def test_captured_training_tail(opt):
    # Clipped AdamW captured once and replayed with a step number on the
    # device, against the definition step by step.
    p, g, m, v = adam_state([5000, 33, 8193], (BF16,), 60, 1, first=True)
    state = [[t.double().clone() for t in ts] for ts in (p, m, v)]
    hyper = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8, wd=0.1)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    bound = 0.5 * exact_norm(g)[0]

    def tail():
        step.add_(1)
        _, scale = opt.grad_norm(g, max_norm=bound)
        opt.adamw_step(p, g, m, v, step=step, grad_scale=scale, **hyper)
        return scale

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        scale = tail()
    for t in range(1, 5):
        for x in g:
            x.copy_(torch.roll(x, 1) * -0.75)
        old = [[x.clone() for x in ts] for ts in (p, m, v)]
        graph.replay()
        torch.cuda.synchronize()
        assert step.item() == t
        norm = exact_norm(g)[0]
        assert abs(scale.item() - clip_of(norm, bound)) <= 7.0 * U * 1.001
        for i in range(len(p)):
            want, tol = adamw64(old[0][i], g[i], old[1][i], old[2][i], step=t, s=scale.item(), more=6.5, **hyper)
            check_adamw((p[i], m[i], v[i]), want, tol)
    del graph, state


@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.0, 0.95), (0.95, 0.0), (0.999, 0.99999)])
@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 9])
def test_adamw_with_the_step_on_the_device(opt, betas, step):
    p, g, m, v = adam_state([3001, 9], (F32, BF16), 61, 1, first=step == 1)
    old = [[t.clone() for t in ts] for ts in (p, m, v)]
    hyper = dict(lr=1e-3, betas=betas, eps=1e-8, wd=0.1)
    opt.adamw_step(p, g, m, v, step=torch.tensor(step, device=DEV), **hyper)
    for i in range(2):
        w, tol = adamw64(old[0][i], g[i], old[1][i], old[2][i], step=step, s=1.0, more=6.5, **hyper)
        check_adamw((p[i], m[i], v[i]), w, tol)


def test_refusals_on_the_device(opt):
    a, b = tensors([100, 100], (F32,))
    with pytest.raises(muon.MuonError):
        opt.clip_grads([a, a], 1.0)
    with pytest.raises(muon.MuonError):
        opt.clip_grads([a], 1.0, out=[a.view(BF16)[:100]])
    with pytest.raises(muon.MuonError):
        opt.adamw_step([a], [b], [a], [b.clone()], lr=1e-3, step=1)
    with pytest.raises(muon.MuonError):
        opt.adamw_step([a], [b], [b.clone()], [b.clone()], lr=1e-3, step=0)
    with pytest.raises(ValueError):
        opt.clip_grads([a], 1.0, out=[b[:50]])
    with pytest.raises(ValueError):
        opt.grad_norm([a.cpu()])
    with pytest.raises(muon.MuonError):
        opt.grad_norm([a], max_norm=-1.0)
    with pytest.raises(ValueError):
        opt.adamw_step([a], [b], [b.clone()], [b.clone()], lr=1e-3, step=torch.ones(1, device=DEV))


def test_a_closed_handle_is_refused():
    o = muon.Muon(device=0)
    a = torch.zeros(4, device=DEV)
    o.close()
    for call in (lambda: o.grad_norm([a]), lambda: o.clip_grads([a], 1.0),
                 lambda: o.adamw_step([a], [a.clone()], [a.clone()], [a.clone()], lr=1e-3, step=1)):
        with pytest.raises(muon.MuonError) as e:
            call()
        assert "handle is NULL" in str(e.value)


def test_lists_of_other_kinds(opt):
    a, b = tensors([100, 50], (F32,))
    want = exact_norm([a, b])[0]
    for ts in ((a, b), iter([a, b]), {"a": a, "b": b}.values()):
        assert abs(opt.grad_norm(ts)[0].item() - want) <= U * 1.001 * want


@pytest.mark.parametrize("dtype", [BF16])
def test_more_than_2_to_31_elements(opt, dtype):
    n = (1 << 31) + 4099
    g = torch.full((n,), 0.5, dtype=dtype, device=DEV)
    g[-1] = 64.0
    g[(1 << 31) + 1] = -32.0
    want = math.sqrt(0.25 * (n - 2) + 64.0 ** 2 + 32.0 ** 2)
    norm, _ = opt.grad_norm([g])
    assert abs(norm.item() - want) <= 5.0 * U * 1.001 * want
    assert opt.grad_norm([g], norm_type=math.inf)[0].item() == 64.0
    p = torch.full((n,), 1.0, device=DEV)
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    opt.adamw_step([p], [g], [m], [v], lr=1e-3, step=1, wd=0.0)
    opt.clip_grads([g], 0.25 * want)
    s = clip_of(want, 0.25 * want)
    for at in (0, 1 << 30, (1 << 31) + 1, n - 2, n - 1):
        g0 = {(1 << 31) + 1: -32.0, n - 1: 64.0}.get(at, 0.5)
        assert abs(g[at].item() - s * g0) <= (2.0 ** -8 + 8 * U) * abs(s * g0)
        w, t = adamw64(p.new_ones(1), torch.tensor([g0], device=DEV), m.new_zeros(1), m.new_zeros(1), 1e-3, 1,
                       (0.9, 0.999), 1e-8, 0.0, 1.0)
        check_adamw((p[at:at + 1], m[at:at + 1], v[at:at + 1]), w, t)


def test_a_module_s_parameters_and_gradients(opt):
    # Parameters as a program has them, gradients from a backward pass, the
    # tied one listed once; in and out of inference mode.
    torch.manual_seed(0)
    emb = torch.nn.Embedding(501, 48, device=DEV)
    net = torch.nn.Sequential(torch.nn.Linear(48, 33, device=DEV), torch.nn.LayerNorm(33, device=DEV),
                              torch.nn.Linear(33, 48, device=DEV))
    ids = torch.randint(0, 400, (64,), device=DEV)          # rows above 400 get zero gradients
    params = list(emb.parameters()) + list(net.parameters())
    m, v = [torch.zeros_like(p) for p in params], [torch.zeros_like(p) for p in params]
    for step in (1, 2):
        for p in params:
            p.grad = None
        torch.nn.functional.linear(net(emb(ids)), emb.weight).square().mean().backward()
        grads = [p.grad for p in params]
        old = [[t.detach().clone() for t in ts] for ts in (params, m, v)]
        want, _ = exact_norm(grads)
        with torch.inference_mode(step == 2):
            norm, scale = opt.grad_norm(grads, max_norm=0.5 * want)
            opt.adamw_step(params, grads, m, v, lr=1e-3, step=step, grad_scale=scale)
        assert abs(norm.item() - want) <= U * 1.001 * want
        for i in range(len(params)):
            w, tol = adamw64(old[0][i], grads[i], old[1][i], old[2][i], 1e-3, step, (0.9, 0.999), 1e-8, 0.1, scale.item())
            check_adamw((params[i].detach(), m[i], v[i]), w, tol)
    net(emb(ids)).sum().backward()                           # the next pass runs on the updated parameters


def test_mostly_zero_gradients(opt):
    # An embedding's: whole stretches of zeros, some signed, in 16 bits.
    for dtype in (BF16, F16):
        g = torch.zeros(300_000, dtype=dtype, device=DEV)
        g[1::2] = -0.0
        g[123_456] = 3.0
        g[200_001] = -4.0
        norm, _, per = opt.grad_norm([g, torch.zeros(5000, dtype=dtype, device=DEV)], per_tensor=True)
        assert norm.item() == 5.0 and per.tolist() == [5.0, 0.0]
        assert opt.grad_norm([g], norm_type=math.inf)[0].item() == 4.0


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_subnormal_gradients(opt, dtype):
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps      # the smallest magnitude
    g = torch.full((4099,), 3 * tiny, dtype=dtype, device=DEV)
    want = exact_norm([g])[0]
    tol = 5.0 * U * want + torch.finfo(F32).tiny * torch.finfo(F32).eps / 2   # and fp32's own last step
    assert abs(opt.grad_norm([g])[0].item() - want) <= tol
    assert opt.grad_norm([g], norm_type=math.inf)[0].item() == 3 * tiny


# -- the multiplier in the Muon step -----------------------------------------

@pytest.mark.parametrize("gtype", [F32, BF16])
@pytest.mark.parametrize("shapes", [[(256, 512), (384, 128), (5, 3)], [(64, 100)]])
def test_step_with_grad_scale_is_the_step_on_scaled_gradients(gtype, shapes):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(9)
    s = torch.tensor([0.37], device=DEV)
    p, g, m = ([torch.randn(*sh, generator=gen, device=DEV) for sh in shapes] for _ in range(3))
    g = [x.to(gtype) for x in g]
    with muon.Muon(device=0, deterministic=True) as o:
        runs = []
        for grads, kw in (([x.float() * s for x in g], {}), (g, {"grad_scale": s})):
            pp, mm = [x.clone() for x in p], [x.clone() for x in m]
            o.step(pp, grads, mm, lr=1e-2, **kw)
            runs.append(pp + mm)
        for a, b in zip(*runs):
            assert torch.equal(a, b)
        # a multiplier of 1 is the plain step
        runs = []
        for kw in ({}, {"grad_scale": torch.ones(1, device=DEV)}):
            pp, mm = [x.clone() for x in p], [x.clone() for x in m]
            o.step(pp, g, mm, lr=1e-2, **kw)
            o.step_schedule(pp, g, mm, [muon.DEFAULT_COEFFS] * 5, lr=1e-2, **kw)
            runs.append(pp + mm)
        for a, b in zip(*runs):
            assert torch.equal(a, b)


def test_whole_models_step_clipped_over_several_steps():
    # Two matrices for Muon, an embedding, a norm and a bias for AdamW, one
    # norm over all of them; against the oracle and the definition. The
    # matrices use the fp32 Newton-Schulz mode, at its gate.
    rng = np.random.default_rng(70)
    shapes2, others = [(96, 160), (160, 96)], [(501, 96), (96,), (7,)]
    lr, bound, wd = 1e-2, 1.0, 0.1
    beta = 0.95
    mk = lambda s, k: torch.tensor(rng.standard_normal(s) * k, dtype=F32, device=DEV)  # noqa: E731
    P, M = [mk(s, 0.05) for s in shapes2], [torch.zeros(s, device=DEV) for s in shapes2]
    p, m, v = [mk(s, 0.05) for s in others], [torch.zeros(s, device=DEV) for s in others], \
        [torch.zeros(s, device=DEV) for s in others]
    with muon.Muon(device=0, ns_precision="fp32") as o:
        for t in range(1, 4):
            G, g = [mk(s, 0.1) for s in shapes2], [mk(s, 0.1) for s in others]
            g[0] = g[0].to(BF16)
            oldP, oldM = [to64(x) for x in P], [to64(x) for x in M]
            old = [[x.clone() for x in ts] for ts in (p, m, v)]
            norm, scale = o.grad_norm(G + g, max_norm=bound)
            o.step(P, G, M, lr=lr, beta=beta, wd=wd, grad_scale=scale)
            o.adamw_step(p, g, m, v, lr=lr, step=t, wd=wd, grad_scale=scale)
            want, _ = exact_norm(G + g)
            assert want > bound and abs(norm.item() - want) <= norm_tol(G + g, 2.0) * want
            s = scale.item()
            for i in range(len(P)):
                ref = O.muon_step_matrix(oldP[i], s * to64(G[i]), oldM[i], lr=float(np.float32(lr)),
                                         beta=float(np.float32(beta)), wd=float(np.float32(wd)))
                assert rel(to64(M[i]), ref[1]) <= 1e-6
                assert rel(to64(P[i]) - oldP[i], ref[0] - oldP[i]) <= TOL_FP32_NS
            for i in range(len(p)):
                w, tol = adamw64(old[0][i], g[i], old[1][i], old[2][i], lr, t, (0.9, 0.999), 1e-8, wd, s)
                check_adamw((p[i], m[i], v[i]), w, tol)
        assert o.status() == (0, 0, 0)
