"""Cases of the gradient operators: global norm, clipping, and the AdamW update that takes the clip multiplier.

A training step of this package ends in the same three pieces whatever the model: the norm of every gradient taken
together, the multiplier min(1, max_norm / (norm + 1e-6)), and the updates. Matrices go to ``Muon.step``; embeddings,
heads, norms and biases go to ``Muon.adamw_step``. Gradients arrive in many tensors of very different sizes: separate
allocations (every start aligned), or views packed one behind the other in a flat buffer (any start).

A case is a dict:
  op       "norm", "clip" or "adamw"
  sizes    how the tensors' sizes are made: "vectors" (count equal ones), "ragged" (count of them, sizes spread over
           a factor of 1000, all odd ones possible), "layer" (count layers of the Llama-3-8B-shaped set), "experts"
           (count matrices of the MoE set), "table" (one rows x cols table and count vectors of cols)
  total    elements in all (ragged), or cols (vectors, table)
  dtype    of the gradients: "float32", "bfloat16", "float16", or "mixed" (the three in turn)
  packed   views one behind the other, or every tensor's start on a multiple of 64 elements
  norm     "l2" or "inf"
  out      clip only: "place", or the type of the tensors that receive the clipped gradients
  step     adamw only: the first pass's step number
"""

import math
import random

import torch

own = False

_DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
_LAYER = (4096 * 4096, 1024 * 4096, 1024 * 4096, 4096 * 4096, 14336 * 4096, 14336 * 4096, 4096 * 14336)
_EXPERT = 2048 * 7168
_NORM = 3.0                # the gradients' norm is about this, so that a bound of 1 clips
_MAX_NORM = 1.0
_LR, _BETAS, _EPS, _WD = 2e-4, (0.9, 0.95), 1e-8, 0.1


def _case(name, op, sizes, count, total, dtype, packed=False, norm="l2", out="place", step=1000, rows=0):
    return {"name": name, "op": op, "sizes": sizes, "count": count, "total": total, "rows": rows, "dtype": dtype,
            "packed": packed, "norm": norm, "out": out, "step": step, "shape_seed": 1}


def listed():
    return [
        # The vectors of a 12-layer model of width 768 (two norms a layer and a last one): latency alone.
        _case("norm_vectors", "norm", "vectors", 25, 768, "float32"),
        # The largest entry of a ragged set of all types in flat buffers, as a monitor logs it.
        _case("norm_ragged_inf", "norm", "ragged", 300, 20_000_003, "mixed", packed=True, norm="inf"),
        # Expert matrices with fp32 gradients.
        _case("norm_experts", "norm", "experts", 24, 0, "float32"),
        # Eight layers of the Llama-3-8B-shaped set, bf16 gradients: far larger than L2.
        _case("norm_layers", "norm", "layer", 8, 0, "bfloat16"),
        # The same vectors clipped in place.
        _case("clip_vectors", "clip", "vectors", 25, 768, "float32"),
        # fp16 gradients in a flat communication buffer, written clipped as fp32.
        _case("clip_bucket", "clip", "ragged", 200, 30_000_001, "float16", packed=True, out="float32"),
        # One layer's fp32 gradients, in place.
        _case("clip_layer", "clip", "layer", 1, 0, "float32"),
        # Four layers' bf16 gradients, in place.
        _case("clip_layers", "clip", "layer", 4, 0, "bfloat16"),
        # The vectors' first update.
        _case("adamw_vectors", "adamw", "vectors", 25, 768, "float32", step=1),
        # Many small and odd tensors of all gradient types, flat buffers.
        _case("adamw_ragged", "adamw", "ragged", 400, 10_000_019, "mixed", packed=True),
        # An embedding table with an odd number of rows, fp32 gradients.
        _case("adamw_table", "adamw", "table", 25, 768, "float32", rows=50_001),
        # A large embedding table, bf16 gradients, and the norms of 32 layers of its width.
        _case("adamw_large", "adamw", "table", 65, 4096, "bfloat16", rows=131_072),
    ]


def draw(rng):
    op = rng.choice(("norm", "clip", "adamw"))
    sizes = rng.choice(("vectors", "ragged", "ragged", "table"))
    dtype = rng.choice(("float32", "bfloat16", "float16", "mixed"))
    most = 1.2e8 if op == "adamw" else 3e8
    case = _case("", op, sizes, 0, 0, dtype, packed=rng.random() < 0.5, norm=rng.choice(("l2", "l2", "inf")),
                 out=rng.choice(("place", "place", "float32", "bfloat16")), step=rng.choice((1, 2, 17, 100_000)))
    del case["name"]
    case["shape_seed"] = rng.randrange(1 << 30)
    if sizes == "ragged":
        case["count"] = int(math.exp(rng.uniform(0, math.log(700))))
        case["total"] = max(4 * case["count"], int(math.exp(rng.uniform(math.log(2e4), math.log(most)))))
    else:
        case["count"] = int(math.exp(rng.uniform(math.log(2), math.log(200))))
        case["total"] = int(math.exp(rng.uniform(math.log(300), math.log(9000))))
        if sizes == "table":
            case["rows"] = int(math.exp(rng.uniform(math.log(50), math.log(most / case["total"]))))
    return case


def _sizes(case):
    kind, count, total = case["sizes"], case["count"], case["total"]
    if kind == "vectors":
        return [total] * count
    if kind == "layer":
        return list(_LAYER) * count
    if kind == "experts":
        return [_EXPERT] * count
    if kind == "table":
        return [case["rows"] * total] + [total] * count
    rng = random.Random(case["shape_seed"])
    w = [math.exp(rng.uniform(0, math.log(1000.0))) for _ in range(count)]
    return [max(1, int(total * x / sum(w))) for x in w]


def _dtypes(case):
    n = len(_sizes(case))
    if case["dtype"] == "mixed":
        three = (torch.float32, torch.bfloat16, torch.float16)
        return [three[i % 3] for i in range(n)]
    return [_DTYPES[case["dtype"]]] * n


def _layout(case):
    """(start, size) of every tensor in the flat buffer of its type, and the buffers' lengths by type."""
    at, where = {}, []
    for n, t in zip(_sizes(case), _dtypes(case)):
        start = at.get(t, 0)
        where.append((start, n))
        at[t] = start + (n if case["packed"] else (n + 63) // 64 * 64)
    return where, at


def _views(case, flats):
    return [flats[t][s:s + n] for (s, n), t in zip(_layout(case)[0], _dtypes(case))]


def _fill(case, gen, length, dtype, scale, uniform=False):
    """A buffer with values in the tensors and zeros between them."""
    out = torch.empty(length, dtype=dtype, device="cuda")
    for a in range(0, length, 1 << 27):
        b = min(length, a + (1 << 27))
        x = (torch.rand if uniform else torch.randn)(b - a, generator=gen, device="cuda")
        out[a:b] = x.mul_(scale).to(dtype)
    return out


def _blank(case, flats):
    if not case["packed"]:
        ends = {}
        for (s, n), t in zip(_layout(case)[0], _dtypes(case)):
            if t in ends and ends[t] < s:
                flats[t][ends[t]:s] = 0
            ends[t] = s + n
        for t, e in ends.items():
            flats[t][e:] = 0
    return flats


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lengths = _layout(case)[1]
    rms = _NORM / math.sqrt(sum(_sizes(case)))
    flats = _blank(case, {t: _fill(case, gen, n, t, rms) for t, n in lengths.items()})
    state = {"case": case, "flats": flats, "grads": _views(case, flats),
             "max_norm": _MAX_NORM * (rms if case["norm"] == "inf" else 1.0), "step": case["step"]}
    if case["op"] == "clip" and case["out"] != "place":
        state["outs"] = {t: torch.zeros(n, dtype=_DTYPES[case["out"]], device="cuda") for t, n in lengths.items()}
        state["out"] = _views(case, state["outs"])
    if case["op"] == "adamw":
        first = case["step"] == 1
        for k, scale, uniform in (("p", 0.02, False), ("m", 0.0 if first else 0.3 * rms, False),
                                  ("v", 0.0 if first else 2.0 * rms * rms, True)):
            state[k] = _blank(case, {t: _fill(case, gen, n, torch.float32, scale, uniform) for t, n in lengths.items()})
            state[k + "s"] = _views(case, state[k])
    return state


_HANDLE = []


def _opt():
    if not _HANDLE:
        import muon_newton_schulz_03_b200 as muon
        _HANDLE.append(muon.Muon(device=0))
    return _HANDLE[0]


# ---- the plain forms: 32 bits; elementwise work over whole buffers, not tensor by tensor ----

def _plain_norm(grads, kind, max_norm):
    if kind == "inf":
        per = torch.stack([g.abs().max().float() for g in grads])
        total = per.max()
    else:
        sums = torch.stack([g.float().square().sum() for g in grads])
        per, total = sums.sqrt(), sums.double().sum().sqrt()
    return total.float(), (max_norm / (total + 1e-6)).clamp(max=1.0).float(), per


def _plain_adamw(p, m, v, g, scale, step):
    b1, b2 = _BETAS
    g = g.float() * scale
    m.mul_(b1).add_(g, alpha=1.0 - b1)
    v.mul_(b2).add_(g.square_(), alpha=1.0 - b2)
    den = v.sqrt().div_(math.sqrt(1.0 - b2 ** step)).add_(_EPS)
    p.mul_(1.0 - _LR * _WD).sub_(m.div(den).mul_(_LR / (1.0 - b1 ** step)))


def _run_norm(s):
    c = s["case"]
    if own:
        norm, scale, per = _opt().grad_norm(s["grads"], max_norm=s["max_norm"], per_tensor=True,
                                            norm_type=math.inf if c["norm"] == "inf" else 2.0)
    else:
        norm, scale, per = _plain_norm(s["grads"], c["norm"], s["max_norm"])
    return {"norm": norm, "scale": scale, "per_tensor": per}


def _run_clip(s):
    c, bound = s["case"], s["max_norm"]
    to = s.get("outs", s["flats"])
    if own:
        norm = _opt().clip_grads(s["grads"], bound, out=s.get("out"),
                                 norm_type=math.inf if c["norm"] == "inf" else 2.0)
    else:
        norm, scale, _ = _plain_norm(s["grads"], c["norm"], bound)
        _ = [to[t].copy_(g.float() * scale) for t, g in s["flats"].items()]
    if "outs" not in s:
        s["max_norm"] = bound * 0.9995     # a bound that tightens: gradients clipped in place are clipped again
    return {"norm": norm, "grads": list(to.values())}


def _run_adamw(s):
    c, step = s["case"], s["step"]
    if own:
        norm, scale = _opt().grad_norm(s["grads"], max_norm=s["max_norm"],
                                       norm_type=math.inf if c["norm"] == "inf" else 2.0)
        _opt().adamw_step(s["ps"], s["grads"], s["ms"], s["vs"], lr=_LR, step=step, betas=_BETAS, eps=_EPS, wd=_WD,
                          grad_scale=scale)
    else:
        norm, scale, _ = _plain_norm(s["grads"], c["norm"], s["max_norm"])
        _ = [_plain_adamw(s["p"][t], s["m"][t], s["v"][t], g, scale, step) for t, g in s["flats"].items()]
    s["step"] = step + 1
    return {"norm": norm, **{k: list(s[k].values()) for k in ("p", "m", "v")}}


def run(state):
    return {"norm": _run_norm, "clip": _run_clip, "adamw": _run_adamw}[state["case"]["op"]](state)


def work(case):
    wide = {torch.float32: 4, torch.bfloat16: 2, torch.float16: 2}
    pairs = list(zip(_sizes(case), _dtypes(case)))
    n, read = sum(k for k, _ in pairs), sum(k * wide[t] for k, t in pairs)
    if case["op"] == "norm":
        return {"bytes": read + 4 * len(pairs) + 8, "flops": 2 * n}
    if case["op"] == "clip":
        wrote = read if case["out"] == "place" else n * wide[_DTYPES[case["out"]]]
        return {"bytes": read + wrote + 4, "flops": 3 * n}
    return {"bytes": read + 24 * n + 4, "flops": 18 * n}


def _exact_norm(s):
    """Norm of each tensor and of all, from the definition, in pieces that stay small."""
    parts = [[x.double() for x in g.split(1 << 26)] if g.numel() <= 1 << 26 else g.split(1 << 26) for g in s["grads"]]
    if s["case"]["norm"] == "inf":
        per = torch.stack([torch.stack([x.abs().amax().double() for x in ps]).amax() for ps in parts])
        return per, per.amax()
    sq = torch.stack([torch.stack([torch.dot(y, y) for y in (x.double() for x in ps)]).sum() for ps in parts])
    return sq ** 0.5, sq.sum() ** 0.5


def exact(case, seed):
    s = prepare(case, seed)
    per, norm = _exact_norm(s)
    scale = torch.minimum(torch.ones_like(norm), s["max_norm"] / (norm + 1e-6))
    if case["op"] == "norm":
        return {"norm": norm, "scale": scale, "per_tensor": per}
    if case["op"] == "clip":
        return {"norm": norm, "grads": [g.double() * scale for g in s["flats"].values()]}
    t, (b1, b2) = case["step"], _BETAS
    out = {"p": [], "m": [], "v": []}
    for k, g in s["flats"].items():
        new = {n: torch.empty(g.numel(), dtype=torch.float64, device="cuda") for n in out}
        for a in range(0, g.numel(), 1 << 26):
            i = slice(a, a + (1 << 26))
            gi = g[i].double() * scale
            new["m"][i] = b1 * s["m"][k][i].double() + (1 - b1) * gi
            new["v"][i] = b2 * s["v"][k][i].double() + (1 - b2) * gi * gi
            mhat, vhat = new["m"][i] / (1 - b1 ** t), new["v"][i] / (1 - b2 ** t)
            p = s["p"][k][i].double()
            new["p"][i] = p - _LR * _WD * p - _LR * mhat / (vhat ** 0.5 + _EPS)
        for n in out:
            out[n].append(new[n])
    return {"norm": norm, **out}
