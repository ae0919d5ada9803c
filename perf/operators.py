"""Cases for timing and checking the gradient-norm and clipping operators.

Four operators over a whole list of gradient tensors:

- ``norm``: the global L2 norm of all gradients, the clipping factor that
  follows from it, and the norm of every single tensor;
- ``clip``: the same norm, and every gradient times the factor (into buffers
  of its own, or in place);
- ``adam``: the norm of the list, then the Adam step on the clipped gradients;
- ``muon``: the norm of the list, then the Muon step on the clipped gradients
  (written to an update buffer, or applied to the weights);
- ``step``: all of them as one training step: one norm over the hidden
  matrices and the other parameters together, the Muon step on the first and
  the Adam step on the second.

With ``own`` false, ``run`` computes them from elementary torch operations;
with ``own`` true, through this package's plans. The tensors are those of a
GPT-2-shaped model (``layers`` blocks of width ``d``: four d x d matrices, one
d x 4d and one 4d x d, biases and norm scales, embeddings of ``vocab`` and
``ctx`` rows). Tensors of one shape lie one after the other in one buffer, as
gradient buckets do, so odd widths put most of them off any 16-byte boundary;
``pad`` elements behind each row make the matrices strided.
"""
import math

import numpy as np
import torch

own = False

F32 = lambda x: float(np.float32(x))  # noqa: E731  (the library's scalars are float32)
COEFFS = (F32(3.4445), F32(-4.7750), F32(2.0315))
NS_STEPS = 5
MOMENTUM, NS_EPS = F32(0.95), F32(1e-7)
LR, WD = F32(0.02), F32(0.01)
ADAM = dict(lr=F32(1e-3), beta1=F32(0.9), beta2=F32(0.99), eps=F32(1e-8), wd=F32(0.1), step=100)
CLIP_EPS = F32(1e-6)
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _case(name, op, **kw):
    case = {"op": op, "layers": 1, "d": 768, "vocab": 0, "ctx": 0, "mats": True, "vecs": False, "dtype": "bf16", "vec_dtype": "fp32",
            "pad": 0, "max_norm": 1.0, "micro": 1, "inplace": False, "apply": False}
    case.update(kw)
    return dict(case, name=name) if name else case


def listed():
    return [
        # the biases and norm scales of one block: a handful of short vectors, where a call is all latency
        _case("norm vectors of a block", "norm", mats=False, vecs=True),
        # every gradient of a 124M model before its optimizer step, logged per tensor
        _case("norm 124M mixed", "norm", layers=12, vocab=50257, ctx=1024, vecs=True),
        # wide matrices (the 2048 x 8192 workload): a gradient set far larger than any cache
        _case("norm wide", "norm", layers=32, d=2048, square=False),
        # one block of odd width accumulated over three micro-batches: tensors off every boundary
        _case("clip odd block", "clip", d=765, vecs=True, vec_dtype="bf16", micro=3),
        # all gradients of a 124M model, scaled into buffers of their own
        _case("clip 124M", "clip", layers=12, vocab=50257, ctx=1024, vecs=True),
        # a 350M model's fp32 gradients in place on an ordinary step: the norm is under the limit
        _case("clip 350M in place, below", "clip", layers=24, d=1024, dtype="fp32", max_norm=1e6, inplace=True),
        # matrices that are column slices of wider rows
        _case("clip strided rows", "clip", layers=4, pad=40),
        # Adam on the short vectors of one block
        _case("adam vectors of a block", "adam", mats=False, vecs=True),
        # Adam on a 124M model's embeddings, biases and scales, bf16
        _case("adam 124M", "adam", layers=12, vocab=50257, ctx=1024, mats=False, vecs=True, vec_dtype="bf16"),
        # Muon on one block's hidden matrices
        _case("muon block", "muon"),
        # Muon on all hidden matrices of a 124M model, applied to the weights
        _case("muon 124M applied", "muon", layers=12, apply=True),
        # the whole optimizer step of a 124M model
        _case("step 124M", "step", layers=12, vocab=50257, ctx=1024, vecs=True, vec_dtype="bf16", apply=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "clip", "adam", "muon", "step"])
    heavy = op in ("muon", "step")
    kw = dict(layers=_log(rng, 1, 12), d=_log(rng, 24, 768 if heavy else 1024), max_norm=rng.choice([0.5, 1.0, 4.0, 1e6]), micro=rng.choice([1, 1, 2, 5]))
    if op == "adam":
        kw.update(mats=False, vecs=True, vec_dtype=rng.choice(["bf16", "fp32"]), vocab=_log(rng, 64, 50257), ctx=_log(rng, 16, 1024))
    elif op == "muon":
        kw.update(apply=rng.random() < 0.5)
    elif op == "step":
        kw.update(vecs=True, vec_dtype=rng.choice(["bf16", "fp32"]), vocab=_log(rng, 64, 50257), ctx=_log(rng, 16, 1024), apply=rng.random() < 0.5)
    else:
        kw.update(dtype=rng.choice(["bf16", "bf16", "fp32"]), vec_dtype=rng.choice(["bf16", "fp32"]), vecs=rng.random() < 0.7, pad=rng.choice([0, 0, 8, 3]))
        if kw["vecs"]:
            kw.update(vocab=_log(rng, 64, 50257), ctx=_log(rng, 16, 1024))
    return _case(None, op, **kw)


def _groups(case):
    """(count, rows, cols, row stride, dtype, matrix?) of the tensors that share a shape, in order."""
    n, d, pad = case["layers"], case["d"], case["pad"]
    out = []
    if case["mats"]:
        shapes = [(4 * n, d, d)] if case.get("square", True) else []
        out += [(c, r, k, k + pad, case["dtype"], True) for c, r, k in shapes + [(n, d, 4 * d), (n, 4 * d, d)]]
    if case["vecs"]:
        emb = [(1, case["vocab"], d), (1, case["ctx"], d)]
        out += [(c, r, k, k, case["vec_dtype"], False) for c, r, k in emb + [(6 * n + 2, 1, d), (n, 1, 3 * d), (n, 1, 4 * d)] if r]
    return out


def _random(g, gen, scale):
    count, rows, cols, ld, dtype, _ = g
    x = torch.zeros(count, rows, ld, dtype=DT[dtype], device="cuda")
    x[:, :, :cols].normal_(0.0, scale, generator=gen)
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    groups = _groups(case)
    s = {"case": case, "groups": groups}
    # gradients: noise of a different size for every kind of tensor, and a few strong directions in the matrices
    grads = []
    for k, g in enumerate(groups):
        x = _random(g, gen, 0.02 / (1 + k % 3))
        if g[5]:
            u = torch.randn(g[0], g[1], 4, device="cuda", generator=gen)
            v = torch.randn(g[0], 4, g[2], device="cuda", generator=gen)
            x[:, :, : g[2]] += (0.02 * torch.matmul(u, v)).to(x.dtype)
        grads.append(x)
    s["grads"] = grads
    views = [_views(x, g) for x, g in zip(grads, groups)]
    s["max_norm"], s["mul"] = F32(case["max_norm"]), F32(1.0 / case["micro"])
    if case["op"] == "clip":
        s["outs"] = grads if case["inplace"] else [torch.zeros_like(x) for x in grads]
    if case["op"] in ("muon", "step"):
        s["bufs"] = [_random(g, gen, 0.01) if g[5] else None for g in groups]
        s["new"] = [(_random(g, gen, 0.02) if case["apply"] else torch.zeros_like(x)) if g[5] else None for g, x in zip(groups, grads)]
    if case["op"] in ("adam", "step"):
        s["params"] = [None if g[5] else _random(g, gen, 0.02) for g in groups]
        s["m"] = [None if g[5] else torch.empty(x.shape, device="cuda").normal_(0.0, 1e-4, generator=gen) for g, x in zip(groups, grads)]
        s["v"] = [None if g[5] else torch.empty(x.shape, device="cuda").uniform_(1e-8, 1e-6, generator=gen) for g, x in zip(groups, grads)]
    if own:
        import muon_newton_schulz_04_amd as mu

        flat = sum(views, [])
        outs = None
        if case["op"] == "clip" and not case["inplace"]:
            outs = sum([_views(x, g) for x, g in zip(s["outs"], groups)], [])
        s["clip"] = mu.ClipPlan(flat, outs)
        s["ws"] = torch.empty(max(1, s["clip"].workspace_bytes), dtype=torch.uint8, device="cuda")
        s["norms"] = torch.empty(len(flat), device="cuda")
        some = lambda key, mat: sum([_views(x, g) for x, g in zip(s[key], groups) if g[5] == mat], [])  # noqa: E731
        if "bufs" in s:
            new = some("new", True)
            # an applied step leaves `out` unwritten: the gradient's own buffer stands in for it
            s["muon"] = mu.MuonPlan(some("grads", True), some("bufs", True), some("grads", True) if case["apply"] else new)
            if case["apply"]:
                s["muon"].set_weights(new)
            s["muon"].set_grad_scale(s["clip"].scale)
            s["mws"] = torch.empty(max(1, s["muon"].workspace_bytes), dtype=torch.uint8, device="cuda")
            s["cfg"] = mu.make_config(*COEFFS, NS_STEPS, MOMENTUM, True, NS_EPS)
        if "params" in s:
            s["adam"] = mu.AdamPlan(some("params", False), some("grads", False), some("m", False), some("v", False))
            s["adam"].set_grad_scale(s["clip"].scale)
    return s


def _views(x, g):
    """The tensors of a group, as a user's program holds them."""
    return [t[:, : g[2]] for t in x] if g[1] > 1 else [t[0] for t in x]


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    op = s["case"]["op"]
    kw = dict(max_norm=s["max_norm"], eps=CLIP_EPS, grad_mul=s["mul"], workspace=s["ws"])
    if op == "norm":
        return {"result": s["clip"].norm(norms=s["norms"], **kw), "norms": s["norms"]}
    if op == "clip":
        return {"result": s["clip"].step(**kw), "outs": s["outs"]}
    out = {"result": s["clip"].norm(**kw)}
    if "muon" in s:
        if s["case"]["apply"]:
            s["muon"].step_apply(s["cfg"], LR, WD, s["mws"])
        else:
            s["muon"].step(s["cfg"], s["mws"])
        out.update(new=s["new"], bufs=s["bufs"])
    if "adam" in s:
        s["adam"].step(**ADAM)
        out.update(params=s["params"], m=s["m"], v=s["v"])
    return out


def _run_plain(s):
    op, groups = s["case"]["op"], s["groups"]
    grads = [x[:, :, : g[2]] for x, g in zip(s["grads"], groups)]
    sums = torch.cat([x.float().square().sum((1, 2), dtype=torch.float64) for x in grads])
    norm = sums.sum().sqrt() * s["mul"]
    scale = (torch.where(norm + CLIP_EPS <= s["max_norm"], 1.0, s["max_norm"] / (norm + CLIP_EPS)) * s["mul"]).float()
    out = {"result": torch.stack([norm.float(), scale])}
    if op == "norm":
        return {**out, "norms": (sums.sqrt() * s["mul"]).float()}
    if op == "clip":
        [o[:, :, : g[2]].copy_(x.float() * scale) for o, x, g in zip(s["outs"], grads, groups)]
        return {**out, "outs": s["outs"]}
    if "bufs" in s:
        apply = s["case"]["apply"]
        [_muon_plain(x.float() * scale, b, w, apply) for x, b, w, g in zip(grads, s["bufs"], s["new"], groups) if g[5]]
        out.update(new=s["new"], bufs=s["bufs"])
    if "params" in s:
        [_adam_plain(p, x.float() * scale, m, v) for p, x, m, v, g in zip(s["params"], grads, s["m"], s["v"], groups) if not g[5]]
        out.update(params=s["params"], m=s["m"], v=s["v"])
    return out


def _adam_plain(p, g, m, v):
    h = ADAM
    m.mul_(h["beta1"]).add_((1 - h["beta1"]) * g)
    v.mul_(h["beta2"]).add_((1 - h["beta2"]) * g.square())
    mh, vh = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
    p.copy_(p.float() * (1 - h["lr"] * h["wd"]) - h["lr"] * mh / (vh.sqrt() + h["eps"]))


def _muon_plain(g, buf, new, apply):
    a, b, c = COEFFS
    buf.copy_(MOMENTUM * buf.float() + g)
    x = g + MOMENTUM * buf.float()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[1] > x.shape[2]
    x = x.mT.contiguous() if tall else x
    for _ in range(NS_STEPS):
        gram = torch.matmul(x, x.mT.contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    x = x.mT if tall else x
    new.copy_(new.float() * (1 - LR * WD) - LR * x if apply else x)


def work(case):
    """Each gradient read once for the norm and once by what uses the factor where that has to wait for the norm; states and outputs once each way."""
    flops = moved = 0
    op = case["op"]
    for count, rows, cols, _, dtype, mat in _groups(case):
        n, es = count * rows * cols, 2 if dtype == "bf16" else 4
        flops += 2 * n
        moved += n * es
        if op == "clip" and not case["inplace"]:
            moved += n * es
        if op in ("adam", "step") and not mat:
            moved += n * (2 * es + 16)
            flops += 14 * n
        if op in ("muon", "step") and mat:
            moved += n * es * (4 if case["apply"] else 3)
            m, k = min(rows, cols), max(rows, cols)
            flops += count * NS_STEPS * (m * (m + 1) * k + m * m * (m + 1) + 2 * m * m * k)
    return {"bytes": moved, "flops": flops}


def exact(case, seed):
    """The definitions in 64 bits; stored momentum keeps its type's rounding, as the next line of the definition reads it."""
    s = prepare(case, seed)
    op = case["op"]
    mats = [(s["grads"][k], g) for k, g in enumerate(s["groups"])]
    norms = [torch.linalg.vector_norm(t[..., : g[2]].double()) for x, g in mats for t in x]
    total = math.sqrt(math.fsum(float(t) ** 2 for t in norms)) * s["mul"]
    factor = s["mul"] * min(1.0, s["max_norm"] / (total + CLIP_EPS))
    out = {"result": torch.tensor([total, factor], dtype=torch.float64)}
    if op == "norm":
        out["norms"] = torch.stack(norms) * s["mul"]
    if op == "clip":
        out["outs"] = [x.double() * factor for x, _ in mats]
    if op in ("muon", "step"):
        out["new"], out["bufs"] = [None] * len(mats), [None] * len(mats)
        a, b, c = COEFFS
        for k, (x, g) in enumerate(mats):
            if not g[5]:
                continue
            new, bufs = [], []
            for i in range(g[0]):
                d = x[i].double() * factor
                bufs.append((s["bufs"][k][i].double() * MOMENTUM + d).to(x.dtype).double())
                y = d + MOMENTUM * bufs[-1]
                y = y / (torch.linalg.matrix_norm(y) + NS_EPS)
                left = g[1] <= g[2]
                for _ in range(NS_STEPS):
                    q = y @ y.T.contiguous() if left else y.T.contiguous() @ y
                    poly = b * q + c * (q @ q)
                    y = a * y + (poly @ y if left else y @ poly)
                new.append(s["new"][k][i].double() * (1.0 - LR * WD) - LR * y if case["apply"] else y)
            out["new"][k], out["bufs"][k] = torch.stack(new), torch.stack(bufs)
    if op in ("adam", "step"):
        h = ADAM
        for key in ("params", "m", "v"):
            out[key] = [None] * len(mats)
        for k, (x, g) in enumerate(mats):
            if g[5]:
                continue
            d = x.double() * factor
            out["m"][k] = torch.lerp(d, s["m"][k].double(), h["beta1"])
            out["v"][k] = torch.lerp(d * d, s["v"][k].double(), h["beta2"])
            rate = h["lr"] / (1.0 - math.pow(h["beta1"], h["step"]))
            root = torch.sqrt(out["v"][k] / (1.0 - math.pow(h["beta2"], h["step"]))) + h["eps"]
            out["params"][k] = s["params"][k].double() * (1.0 - h["lr"] * h["wd"]) - rate * out["m"][k] / root
    return out
