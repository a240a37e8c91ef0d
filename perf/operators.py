"""The training-side operators of the library as measured cases: embedding
lookup and its gradient, layer norm and its gradient, and clipping by the
global gradient norm.

`listed()` names the cases, `draw(rng)` makes one more of the same ranges,
`prepare(case, seed)` makes a case's inputs on the GPU, `run(state)` is one
pass: the plain form (elementary torch operations in float32, rounded once at
the end) where `own` is false, the library's operators where it is true.
`exact` gives the same outputs from the definitions in 64 bits and `work` the
bytes and operations no implementation can do without.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
PAD = -1
EPS = 1e-5


def listed():
    return [
        # one short prompt entering a search encoder: latency alone
        {"name": "embed_prompt", "op": "embed", "n": 48, "dim": 512, "vocab": 32000, "table": "bf16", "out": "bf16",
         "bits": 64, "dist": "zipf", "pad": 0.0},
        # a training batch of packed text, float32 master table to bfloat16 activations
        {"name": "embed_batch", "op": "embed", "n": 131072, "dim": 1024, "vocab": 128000, "table": "f32",
         "out": "bf16", "bits": 64, "dist": "zipf", "pad": 0.06},
        # fine-tuning on a handful of short sequences: a small table's gradient
        {"name": "embed_grad_small", "op": "embed_grad", "n": 384, "dim": 256, "vocab": 5003, "dy": "f32",
         "grad": "f32", "bits": 32, "dist": "zipf", "pad": 0.2},
        # the gradient of a text vocabulary over one batch, frequent tokens holding most positions
        {"name": "embed_grad_text", "op": "embed_grad", "n": 65536, "dim": 1024, "vocab": 50001, "dy": "bf16",
         "grad": "f32", "bits": 64, "dist": "zipf", "pad": 0.06},
        # bytes as tokens: few rows, thousands of positions each, an odd width
        {"name": "embed_grad_bytes", "op": "embed_grad", "n": 262144, "dim": 322, "vocab": 259, "dy": "f16",
         "grad": "f16", "bits": 32, "dist": "uniform", "pad": 0.0},
        # the normalised points of a few queries
        {"name": "norm_queries", "op": "norm", "n": 32, "dim": 256, "x": "f32", "y": "f32", "param": "f32"},
        # a long batch through a wide model
        {"name": "norm_batch", "op": "norm", "n": 65536, "dim": 4096, "x": "bf16", "y": "bf16", "param": "bf16"},
        # an odd width and row count, float16 in, float32 points out
        {"name": "norm_odd", "op": "norm", "n": 20011, "dim": 1021, "x": "f16", "y": "f32", "param": "f32"},
        # the backward pass at the points the join takes
        {"name": "norm_grad_points", "op": "norm_grad", "n": 20000, "dim": 128, "x": "f32", "y": "f32",
         "param": "f32"},
        # the backward pass of a training batch
        {"name": "norm_grad_batch", "op": "norm_grad", "n": 32768, "dim": 2048, "x": "bf16", "y": "bf16",
         "param": "f32"},
        # the gradients of a small encoder: a table and many short tensors
        {"name": "clip_encoder", "op": "clip", "tensors": 60, "total": 3000017, "types": "f32", "clips": True},
        # the gradients of a large model, matrices in bfloat16 and vectors in float32
        {"name": "clip_model", "op": "clip", "tensors": 290, "total": 1 << 30, "types": "mixed", "clips": True},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    d = _logint(rng, lo, hi)
    # most widths in use are multiples of 8 or 16; a third are left as drawn
    k = rng.choice([1, 8, 16])
    return max(k, d - d % k)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "clip"])
    if op in ("embed", "embed_grad"):
        dim = _width(rng, 16, 4096)
        vocab = _logint(rng, 256, min(131072, (1 << 27) // dim))
        n = _logint(rng, 1, min(262144, (1 << 27) // dim))
        case = {"op": op, "n": n, "dim": dim, "vocab": vocab, "bits": rng.choice([32, 64]),
                "dist": rng.choice(["zipf", "zipf", "uniform"]), "pad": rng.choice([0.0, 0.06, 0.2])}
        a, b = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                           ("f16", "f32")])
        case.update({"table": a, "out": b} if op == "embed" else {"dy": a, "grad": b})
        return case
    if op in ("norm", "norm_grad"):
        dim = _width(rng, 16, 16384)
        n = _logint(rng, 1, min(131072, (1 << 28) // dim))
        x, y = rng.choice([("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
        return {"op": op, "n": n, "dim": dim, "x": x, "y": y, "param": rng.choice(["f32", y])}
    tensors = _logint(rng, 1, 400)
    return {"op": "clip", "tensors": tensors, "total": _logint(rng, 64 * tensors, 1 << 29),
            "types": rng.choice(["f32", "bf16", "mixed"]), "clips": rng.random() < 0.7}


# ---- inputs -----------------------------------------------------------------

def _tokens(case, gen):
    n, vocab = case["n"], case["vocab"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if case["dist"] == "zipf":  # frequency ~ 1 / (id + 1): the log of the id + 1 is uniform
        t = torch.exp(u * math.log(vocab + 1)).floor().long() - 1
    else:
        t = (u * vocab).floor().long()
    t = t.clamp_(0, vocab - 1)
    if case["pad"] > 0:
        # sequences of up to 512 positions whose tails are padding
        pos = torch.arange(n, device="cuda")
        length = min(512, n)
        cut = torch.rand((n + length - 1) // length, generator=gen, device="cuda")
        keep = length * (1 - 2 * case["pad"] * cut[pos // length])
        t = torch.where(pos % length < keep, t, torch.full_like(t, PAD))
    return t.to(torch.int64 if case["bits"] == 64 else torch.int32)


def _clip_sizes(case):
    """Sizes of the gradient tensors: a quarter are vectors, the rest share
    what is left in the proportions 1 : 2 : 3, and the last takes the remainder."""
    k, total = case["tensors"], case["total"]
    sizes, types = [], []
    weight = [0.01 if i % 4 == 3 else 1.0 + i % 3 for i in range(k)]
    s = sum(weight)
    for i in range(k):
        sizes.append(max(1, int(total * weight[i] / s)))
        types.append({"f32": "f32", "bf16": "bf16", "mixed": "f32" if i % 4 == 3 else "bf16"}[case["types"]])
    sizes[-1] = max(1, sizes[-1] + total - sum(sizes))
    return sizes, types


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(shape, dtype, scale=1.0):
        t = torch.empty(shape, device="cuda", dtype=dtype)
        t.normal_(0.0, scale, generator=gen)
        return t

    op = case["op"]
    if op in ("embed", "embed_grad"):
        v = {"tokens": _tokens(case, gen)}
        if op == "embed":
            v["table"] = normal((case["vocab"], case["dim"]), DTYPES[case["table"]], 0.02)
        else:
            v["dy"] = normal((case["n"], case["dim"]), DTYPES[case["dy"]], 0.01)
        return v
    if op in ("norm", "norm_grad"):
        n, d = case["n"], case["dim"]
        xt, yt, pt = DTYPES[case["x"]], DTYPES[case["y"]], DTYPES[case["param"]]
        x = normal((n, d), xt, 1.3)
        x += torch.randn(d, generator=gen, device="cuda").to(xt)  # activations have a mean of their own per column
        v = {"x": x, "weight": (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(pt)}
        if op == "norm":
            v["bias"] = (0.1 * torch.randn(d, generator=gen, device="cuda")).to(pt)
        else:
            v["dy"] = normal((n, d), yt, 0.1)
            v["mean"] = torch.empty(n, device="cuda")
            v["rstd"] = torch.empty(n, device="cuda")
            step = max(1, (1 << 26) // d)
            for i in range(0, n, step):  # what the forward pass saved
                xf = x[i:i + step].float()
                m = xf.sum(1) / d
                v["mean"][i:i + step] = m
                v["rstd"][i:i + step] = 1 / torch.sqrt(((xf - m[:, None]) ** 2).sum(1) / d + EPS)
        return v
    sizes, types = _clip_sizes(case)
    grads = [normal((s,), DTYPES[t], 0.003 * (1 + i % 5)) for i, (s, t) in enumerate(zip(sizes, types))]
    # the norm that such gradients are expected to have, halved or doubled
    expect = math.sqrt(sum(s * (0.003 * (1 + i % 5)) ** 2 for i, s in enumerate(sizes)))
    return {"grads": grads, "max_norm": float(np.float32(expect * (0.5 if case["clips"] else 2.0)))}


def _buckets(case, f32, rest):
    """One flat buffer per type for the clipped gradients, as buckets of an
    optimiser keep them, and each tensor's piece of its buffer: pieces start on
    16-byte boundaries and the gaps stay zero."""
    sizes, types = _clip_sizes(case)
    start, used = [], {}
    for s, t in zip(sizes, types):
        start.append(used.get(t, 0))
        used[t] = start[-1] + (s + 7) // 8 * 8
    flat = {t: torch.zeros(used[t], dtype=f32 if t == "f32" else rest, device="cuda") for t in sorted(used)}
    return list(flat.values()), [flat[t][a:a + s] for a, s, t in zip(start, sizes, types)]


def _scale(case):
    return float(np.float32(math.sqrt(case["dim"])))


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if case["op"] == "clip":
        state["flat"], state["out"] = _buckets(case, torch.float32, torch.bfloat16)
    if own:
        import exact_dimensional_distance_gb300 as edd
        state["lib"] = edd.Join()
        if case["op"] == "clip":
            state["set"] = edd.Gradients(state["grads"], state["out"])
    return state


# ---- one pass -----------------------------------------------------------------

def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(state, case, case["op"])


def _run_own(state, case, op):
    lib = state["lib"]
    if op == "embed":
        return lib.embed(state["tokens"], state["table"], scale=_scale(case), pad=PAD, dtype=DTYPES[case["out"]])
    if op == "embed_grad":
        return lib.embed_grad(state["tokens"], state["dy"], case["vocab"], scale=_scale(case), pad=PAD,
                              dtype=DTYPES[case["grad"]])
    if op == "norm":
        return lib.layer_norm(state["x"], state["weight"], state["bias"], eps=EPS, dtype=DTYPES[case["y"]])
    if op == "norm_grad":
        return lib.layer_norm_grad(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"])
    return [lib.clip_grads(state["set"], state["max_norm"])] + state["flat"]


def _run_plain(state, case, op):
    if op == "embed":
        t = state["tokens"]
        keep = t != PAD
        rows = state["table"][torch.where(keep, t, 0)].float() * _scale(case)
        return (rows * keep[:, None]).to(DTYPES[case["out"]])
    if op == "embed_grad":
        t = state["tokens"]
        keep = t != PAD
        g = torch.zeros((case["vocab"], case["dim"]), device="cuda")
        g.index_add_(0, torch.where(keep, t, 0), state["dy"].float() * keep[:, None])
        return (g * _scale(case)).to(DTYPES[case["grad"]])
    if op == "norm":
        x = state["x"].float()
        d = x.shape[1]
        mean = x.sum(1) / d
        x = x - mean[:, None]
        rstd = 1 / torch.sqrt((x * x).sum(1) / d + EPS)
        y = x * rstd[:, None] * state["weight"].float() + state["bias"].float()
        return y.to(DTYPES[case["y"]]), mean, rstd
    if op == "norm_grad":
        dy, w = state["dy"].float(), state["weight"].float()
        d = dy.shape[1]
        r = state["rstd"][:, None]
        h = (state["x"].float() - state["mean"][:, None]) * r
        g = dy * w
        dx = r * (g - g.sum(1, keepdim=True) / d - h * ((g * h).sum(1, keepdim=True) / d))
        p = state["weight"].dtype
        return dx.to(state["x"].dtype), (dy * h).sum(0).to(p), dy.sum(0).to(p)
    grads, max_norm = state["grads"], state["max_norm"]
    total = torch.stack([(g.float() * g.float()).sum() for g in grads]).sum()
    norm = torch.sqrt(total)
    c = torch.where((norm > max_norm) & torch.isfinite(norm), max_norm / norm, torch.ones_like(norm))
    for g, out in zip(grads, state["out"]):
        out.copy_((g.float() * c).to(g.dtype))
    return [norm] + state["flat"]


# ---- the definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    v = _inputs(case, seed)
    op = case["op"]
    f = torch.float64
    if op == "embed":
        t = v["tokens"].long()
        out = torch.zeros((case["n"], case["dim"]), dtype=f, device="cuda")
        at = torch.nonzero(t != PAD).flatten()
        out[at] = v["table"].index_select(0, t[at]).to(f) * _scale(case)
        return out
    if op == "embed_grad":
        t = v["tokens"].long()
        at = torch.nonzero(t != PAD).flatten()
        out = torch.zeros((case["vocab"], case["dim"]), dtype=f, device="cuda")
        step = max(1, (1 << 25) // case["dim"])
        for i in range(0, at.numel(), step):
            a = at[i:i + step]
            out.index_put_((t[a],), v["dy"][a].to(f) * _scale(case), accumulate=True)
        return out
    if op == "norm":
        n = case["n"]
        y = torch.empty((n, case["dim"]), dtype=f, device="cuda")
        mean, rstd = torch.empty(n, dtype=f, device="cuda"), torch.empty(n, dtype=f, device="cuda")
        step = max(1, (1 << 25) // case["dim"])
        for i in range(0, n, step):
            x = v["x"][i:i + step].to(f)
            var, m = torch.var_mean(x, dim=1, correction=0)
            r = (var + EPS) ** -0.5
            mean[i:i + step], rstd[i:i + step] = m, r
            y[i:i + step] = torch.addcmul(v["bias"].to(f), (x - m[:, None]) * r[:, None], v["weight"].to(f))
        return y, mean, rstd
    if op == "norm_grad":
        n, d = case["n"], case["dim"]
        dx = torch.empty((n, d), dtype=f, device="cuda")
        dw, db = torch.zeros(d, dtype=f, device="cuda"), torch.zeros(d, dtype=f, device="cuda")
        w = v["weight"].to(f)
        step = max(1, (1 << 25) // d)
        for i in range(0, n, step):
            dy, r = v["dy"][i:i + step].to(f), v["rstd"][i:i + step].to(f)
            h = v["x"][i:i + step].to(f).sub_(v["mean"][i:i + step].to(f)[:, None]).mul_(r[:, None])
            dw += torch.einsum("nd,nd->d", dy, h)
            db += dy.sum(0)
            a = torch.mv(dy, w) / d
            b = torch.einsum("nd,nd,d->n", dy, h, w) / d
            dx[i:i + step] = (dy * w - a[:, None] - h * b[:, None]) * r[:, None]
        return dx, dw, db
    if case["total"] > 1 << 30:
        return None
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g, dtype=f)) ** 2 for g in v["grads"]))
    c = v["max_norm"] / norm if norm > v["max_norm"] else 1.0
    flat, out = _buckets(case, f, f)
    for g, o in zip(v["grads"], out):
        o.copy_(g.to(f).mul_(c))
    return [torch.tensor(norm, dtype=f)] + flat


# ---- what no implementation can do without ------------------------------------------

def _distinct(case):
    """Expected number of vocabulary rows that the case's tokens touch."""
    n, vocab = case["n"] * (1 - case["pad"]), case["vocab"]
    if case["dist"] == "zipf":
        r = np.arange(1, vocab + 1, dtype=np.float64)
        p = np.log1p(1 / r) / math.log(vocab + 1)
    else:
        p = np.full(vocab, 1 / vocab)
    return float(-np.expm1(n * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        n, d, kept = case["n"], case["dim"], case["n"] * (1 - case["pad"])
        tokens = n * case["bits"] // 8
        if op == "embed":
            return {"bytes": int(tokens + _distinct(case) * d * SIZE[case["table"]] + n * d * SIZE[case["out"]]),
                    "flops": int(kept * d)}
        return {"bytes": int(tokens + kept * d * SIZE[case["dy"]] + case["vocab"] * d * SIZE[case["grad"]]),
                "flops": int(kept * d + _distinct(case) * d)}
    if op in ("norm", "norm_grad"):
        n, d, sx, sy, sp = case["n"], case["dim"], SIZE[case["x"]], SIZE[case["y"]], SIZE[case["param"]]
        if op == "norm":
            return {"bytes": n * d * (sx + sy) + 8 * n + 2 * d * sp, "flops": 8 * n * d}
        return {"bytes": n * d * (2 * sx + sy) + 8 * n + 3 * d * sp, "flops": 14 * n * d}
    sizes, types = _clip_sizes(case)
    return {"bytes": sum(2 * s * SIZE[t] for s, t in zip(sizes, types)), "flops": 3 * sum(sizes)}
