"""Cases for timing and checking the embedding operators and the Muon step on stacks of short matrices.

Four operators of one training step:

- ``lookup``: rows of an embedding table by token, times a scale;
- ``gradient``: the table's gradient, the sum of ``dout`` over each token's
  positions, written over the whole table or added to what it holds;
- ``rows``: the same gradient as rows (distinct tokens in ascending order,
  their sums, their number), its norm and clipping factor, and the Adam step
  of the rows on the clipped sums;
- ``stack``: the Muon step (momentum, normalisation, Newton-Schulz iteration)
  on stacks of matrices with a short side: attention heads, adapters. Written
  to an update buffer, or applied to the weights.

With ``own`` false, ``run`` computes them from elementary torch operations;
with ``own`` true, through this package's plans. Tokens follow Zipf's law over
``vocab`` (a low token is frequent, as in a byte-pair vocabulary); a share
``padded`` of them is -1: those look up zeros and carry no gradient.
``pad`` elements behind each row of a table or matrix make it strided.
"""
import math

import numpy as np
import torch

own = False

F32 = lambda x: float(np.float32(x))  # noqa: E731  (the library's scalars are float32)
QUINTIC = (F32(3.4445), F32(-4.7750), F32(2.0315))
CUBIC = (1.5, -0.5, 0.0)
MOMENTUM, NS_EPS = F32(0.95), F32(1e-7)
LR, WD = F32(0.02), F32(0.01)
ADAM = dict(lr=F32(1e-3), beta1=F32(0.9), beta2=F32(0.99), eps=F32(1e-8), wd=F32(0.1), step=100)
MAX_NORM, CLIP_EPS = 1.0, F32(1e-6)
DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "i32": torch.int32, "i64": torch.int64}


def _rows(name, op, tokens, vocab, d, **kw):
    case = {"op": op, "tokens": tokens, "vocab": vocab, "d": d, "dtype": "bf16", "act": "bf16", "index": "i64", "scale": 1.0, "padded": 0.0,
            "pad": 0, "accumulate": False}
    case.update(kw)
    return dict(case, name=name) if name else case


def _stack(name, kinds, layers, heads, side, d, **kw):
    case = {"op": "stack", "kinds": kinds, "layers": layers, "heads": heads, "side": side, "d": d, "dtype": "bf16", "cubic": False, "apply": False, "pad": 0}
    case.update(kw)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token of each of four sequences being generated: a call is all latency
        _rows("lookup 4 tokens", "lookup", 4, 50257, 768, index="i32"),
        # a micro-batch of 8 x 1024 tokens of a 124M model, a tenth of them padding, embeddings times sqrt(d)
        _rows("lookup 124M micro-batch", "lookup", 8192, 50257, 768, scale=F32(math.sqrt(768)), padded=0.1),
        # a long batch on an odd table in float32, activations in bf16
        _rows("lookup 65536 odd", "lookup", 65536, 32003, 1021, dtype="fp32"),
        # a short text on a small table: latency again, and most rows only cleared
        _rows("gradient 17 tokens", "gradient", 17, 1021, 96),
        # the embedding gradient of a 124M model over 32 x 1024 tokens, all rows written
        _rows("gradient 124M", "gradient", 32768, 50257, 768),
        # added to the gradient a tied output layer has left, float32 and odd sizes, strided rows, half of the batch padding
        _rows("gradient tied odd", "gradient", 30011, 5003, 765, dtype="fp32", pad=3, padded=0.5, accumulate=True, scale=0.5),
        # the embedding step of one micro-batch: a sixth of the table's rows or fewer change
        _rows("rows 124M micro-batch", "rows", 8192, 50257, 768, index="i32"),
        # the same for a large table in float32 and a long batch
        _rows("rows 65536 fp32", "rows", 65536, 100003, 1024, dtype="fp32", act="fp32", padded=0.05),
        # the heads of one block of a 124M model: 36 of 64 x 768 (q, k, v) and 12 of 768 x 64 (the output projection's columns)
        _stack("heads of a block", "qkvo", 1, 12, 64, 768),
        # all heads of a 124M model, applied to the weights
        _stack("heads 124M applied", "qkvo", 12, 12, 64, 768, apply=True),
        # rank-16 adapters of odd width, float32, both factors, the cubic iteration with ten steps
        _stack("adapters fp32 odd", "ab", 12, 4, 16, 765, dtype="fp32", cubic=True),
        # heads of 128 in a 2048 wide model, applied to the weights
        _stack("heads 128 x 2048 applied", "qkv", 4, 16, 128, 2048, apply=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "gradient", "gradient", "rows", "stack", "stack"])
    if op == "stack":
        kinds, side, d = rng.choice(["qkv", "qkvo", "ab"]), _log(rng, 4, 128), _log(rng, 128, 2048)
        per = {"qkv": 3, "qkvo": 4, "ab": 2}[kinds]
        cubic = rng.random() < 0.3
        count = min(_log(rng, 1, 200), max(1, (16_000_000 if cubic else 36_000_000) // (per * side * d)))
        heads = rng.choice([h for h in (1, 2, 3, 4, 8, 12) if h <= count])
        return _stack(None, kinds, max(1, count // heads), heads, side, d, dtype=rng.choice(["bf16", "bf16", "fp32"]), cubic=cubic,
                      apply=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 3]))
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    kw = dict(dtype=dtype, act=rng.choice(["bf16", dtype]), index=rng.choice(["i32", "i64"]), scale=rng.choice([1.0, 0.5, F32(math.sqrt(768))]),
              padded=rng.choice([0.0, 0.1, 0.5]), pad=rng.choice([0, 0, 8, 3]))
    if op == "gradient":
        kw["accumulate"] = rng.random() < 0.4
    return _rows(None, op, _log(rng, 1, 65536), _log(rng, 64, 65536), _log(rng, 32, 1024), **kw)


# ---------------------------------------------------------------- inputs

def _strided(rows, d, pad, dtype, gen, scale):
    x = torch.empty(rows, d + pad, dtype=DT[dtype], device="cuda")
    return x.normal_(0.0, scale, generator=gen)[:, :d]


def _tokens(case, gen):
    n, v = case["tokens"], case["vocab"]
    u = torch.rand(n, device="cuda", generator=gen, dtype=torch.float64)
    tok = (torch.exp(u * math.log(v + 1.0)).long() - 1).clamp_(0, v - 1)
    drop = torch.rand(n, device="cuda", generator=gen) < case["padded"]
    return tok.masked_fill_(drop, -1).to(DT[case["index"]])


def _groups(case):
    """(count, rows, cols, row stride, stride from matrix to matrix, tensors of that kind)."""
    h, s, d, p, n = case["heads"], case["side"], case["d"], case["pad"], case["layers"]
    out = []
    if "q" in case["kinds"]:   # heads as row blocks of [layers * 3 heads * side, d]
        out.append((3 * n * h, s, d, d + p, s * (d + p), 1))
    if "o" in case["kinds"]:   # heads as column blocks of each layer's [d, heads * side]
        out.append((h, d, s, h * s + p, s, n))
    if "a" in case["kinds"]:   # an adapter's two factors: [side, d] and [d, side]
        out += [(n * h, s, d, d + p, s * (d + p), 1), (n * h, d, s, s + p, d * (s + p), 1)]
    return out


def _stacks(case, gen, scale, strong=0.0):
    """The 3-D views [count, rows, cols] of every tensor, noise and a few strong directions."""
    out = []
    for count, rows, cols, ld, step, tensors in _groups(case):
        for _ in range(tensors):
            flat = torch.zeros((count - 1) * step + rows * ld, dtype=DT[case["dtype"]], device="cuda")
            x = flat.as_strided((count, rows, cols), (step, ld, 1))
            y = torch.randn(count, rows, cols, device="cuda", generator=gen) * scale
            if strong:
                u = torch.randn(count, rows, 3, device="cuda", generator=gen)
                v = torch.randn(count, 3, cols, device="cuda", generator=gen)
                y += strong * torch.matmul(u, v)
            out.append(x.copy_(y))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "stack":
        s["grads"] = _stacks(case, gen, 0.02, 0.02)
        s["bufs"] = _stacks(case, gen, 0.05)
        s["new"] = _stacks(case, gen, 0.02 if case["apply"] else 0.0)  # the weights, or an update buffer laid out as its gradient
        s["coeffs"], s["steps"] = (CUBIC, 10) if case["cubic"] else (QUINTIC, 5)
        if own:
            import muon_newton_schulz_04_amd as mu

            s["plan"] = mu.StackPlan(s["grads"], s["bufs"], s["grads"] if case["apply"] else s["new"])
            if case["apply"]:
                s["plan"].set_weights(s["new"])
            s["ws"] = torch.empty(max(1, s["plan"].workspace_bytes), dtype=torch.uint8, device="cuda")
            s["cfg"] = mu.make_config(*s["coeffs"], s["steps"], MOMENTUM, True, NS_EPS)
        return s
    n, v, d = case["tokens"], case["vocab"], case["d"]
    cap = min(n, v)
    s["tokens"] = _tokens(case, gen)
    s["table"] = _strided(v, d, case["pad"], case["dtype"], gen, 0.02)
    if case["op"] == "lookup":
        s["out"] = torch.zeros(n, d, dtype=DT[case["act"]], device="cuda")
    else:
        s["dout"] = _strided(n, d, 0, case["act"], gen, 1e-3)
    if case["op"] == "gradient":
        s["grad"] = _strided(v, d, case["pad"], case["dtype"], gen, 1e-3)
    if case["op"] == "rows":
        s["rows"] = torch.zeros(cap, dtype=torch.int32, device="cuda")
        s["values"] = torch.zeros(cap, d, dtype=DT[case["dtype"]], device="cuda")
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["m"] = torch.empty(v, d, device="cuda").normal_(0.0, 1e-4, generator=gen)
        s["v"] = torch.empty(v, d, device="cuda").uniform_(1e-8, 1e-6, generator=gen)
    if own:
        import muon_newton_schulz_04_amd as mu

        s["plan"] = mu.EmbeddingPlan(s["table"], n, s.get("m"), s.get("v"))
        s["ws"] = torch.empty(max(1, s["plan"].workspace_bytes), dtype=torch.uint8, device="cuda")
        if case["op"] == "rows":
            s["clip"] = mu.ClipPlan([s["values"]], [None])
            s["clip"].set_live_rows(0, s["count"], d)
            s["plan"].set_grad_scale(s["clip"].scale)
            s["cws"] = torch.empty(max(1, s["clip"].workspace_bytes), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    case = s["case"]
    op = case["op"]
    if op == "stack":
        if case["apply"]:
            s["plan"].step_apply(s["cfg"], LR, WD, s["ws"])
        else:
            s["plan"].step(s["cfg"], s["ws"])
        return {"new": s["new"], "bufs": s["bufs"]}
    if op == "lookup":
        return s["plan"].lookup(s["tokens"], s["out"], case["scale"])
    if op == "gradient":
        return s["plan"].gradient(s["tokens"], s["dout"], s["grad"], case["scale"], case["accumulate"], s["ws"])
    s["plan"].gradient_rows(s["tokens"], s["dout"], s["rows"], s["values"], s["count"], case["scale"], s["ws"])
    result = s["clip"].norm(MAX_NORM, CLIP_EPS, workspace=s["cws"])
    s["plan"].adam_rows(s["rows"], s["values"], s["count"], **ADAM)
    return {"rows": s["rows"], "values": s["values"], "count": s["count"], "result": result, "table": s["table"], "m": s["m"], "v": s["v"]}


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "stack":
        for g, b, w in zip(s["grads"], s["bufs"], s["new"]):
            _muon_plain(g.float(), b, w, s["coeffs"], s["steps"], case["apply"])
        return {"new": s["new"], "bufs": s["bufs"]}
    tok, v = s["tokens"].long(), case["vocab"]
    live = (tok >= 0) & (tok < v)
    if op == "lookup":
        x = s["table"][tok.clamp(0, v - 1)].float() * case["scale"]
        s["out"].copy_(x.masked_fill(~live.unsqueeze(1), 0.0))
        return s["out"]
    if op == "gradient":
        # padding adds zeros, spread over the table: all of it on one row would wait for one address
        acc = torch.zeros(v, case["d"], dtype=torch.float64, device="cuda")
        acc.index_add_(0, torch.where(live, tok, torch.arange(len(tok), device="cuda") % v), s["dout"].double().masked_fill_(~live.unsqueeze(1), 0.0))
        acc = acc * case["scale"]
        s["grad"].copy_(s["grad"].double() + acc if case["accumulate"] else acc)
        return s["grad"]
    ids, place = torch.unique(tok[live], return_inverse=True)
    n = len(ids)
    acc = torch.zeros(n, case["d"], dtype=torch.float64, device="cuda")
    acc.index_add_(0, place, s["dout"][live].double())
    s["rows"][:n] = ids.to(torch.int32)
    s["values"][:n] = (acc * case["scale"]).to(s["values"].dtype)
    s["count"].fill_(n)
    g = s["values"][:n].float()
    norm = g.square().sum(dtype=torch.float64).sqrt()
    scale = torch.where(norm + CLIP_EPS <= MAX_NORM, 1.0, MAX_NORM / (norm + CLIP_EPS)).float()
    g = g * scale
    h = ADAM
    m = s["m"][ids] * h["beta1"] + (1 - h["beta1"]) * g
    q = s["v"][ids] * h["beta2"] + (1 - h["beta2"]) * g.square()
    mh, vh = m / (1 - h["beta1"] ** h["step"]), q / (1 - h["beta2"] ** h["step"])
    p = s["table"][ids].float() * (1 - h["lr"] * h["wd"]) - h["lr"] * mh / (vh.sqrt() + h["eps"])
    s["m"][ids], s["v"][ids] = m, q
    s["table"][ids] = p.to(s["table"].dtype)
    return {"rows": s["rows"], "values": s["values"], "count": s["count"], "result": torch.stack([norm.float(), scale]), "table": s["table"], "m": s["m"],
            "v": s["v"]}


def _muon_plain(g, buf, new, coeffs, steps, apply):
    a, b, c = coeffs
    buf.copy_(MOMENTUM * buf.float() + g)
    x = g + MOMENTUM * buf.float()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[1] > x.shape[2]
    x = x.mT.contiguous() if tall else x
    for _ in range(steps):
        gram = torch.matmul(x, x.mT.contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    x = x.mT if tall else x
    new.copy_(new.float() * (1 - LR * WD) - LR * x if apply else x)


# ---------------------------------------------------------------- what a pass cannot do without

def _distinct(case):
    """Expected number of distinct tokens of a batch."""
    v, n = case["vocab"], case["tokens"] * (1.0 - case["padded"])
    p = np.diff(np.log(np.arange(1, v + 2))) / math.log(v + 1.0)
    return float(-np.expm1(n * np.log1p(-np.minimum(p, 1.0 - 1e-12))).sum())


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "stack":
        moved = flops = 0
        for count, rows, cols, _, _, tensors in _groups(case):
            m, k, n = min(rows, cols), max(rows, cols), count * tensors
            moved += n * rows * cols * es * (5 if case["apply"] else 4)
            flops += n * (10 if case["cubic"] else 5) * (m * (m + 1) * k + m * m * (m + 1) + 2 * m * m * k)
        return {"bytes": moved, "flops": flops}
    n, v, d = case["tokens"], case["vocab"], case["d"]
    live, index, act = n * (1.0 - case["padded"]), 4 if case["index"] == "i32" else 8, 2 if case["act"] == "bf16" else 4
    some = _distinct(case)
    moved = n * index
    if case["op"] == "lookup":
        moved += some * d * es + n * d * act
        flops = live * d
    else:
        moved += live * d * act
        flops = 2 * live * d
    if case["op"] == "gradient":
        moved += (2 * some if case["accumulate"] else v) * d * es
    if case["op"] == "rows":  # the sums are written, and the table's rows and moments read and written
        moved += some * (4 + d * (3 * es + 16))
        flops += 16 * some * d
    return {"bytes": int(moved), "flops": int(flops)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "stack":
        return _exact_stack(s)
    tok, v, scale = s["tokens"].cpu().numpy().astype(np.int64), case["vocab"], case["scale"]
    if case["op"] == "lookup":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        at = np.flatnonzero(tok >= 0)
        out[torch.from_numpy(at).cuda()] = s["table"].double()[torch.from_numpy(tok[at]).cuda()] * scale
        return out
    # positions ordered by token; each token's sum is a difference of running sums over its own stretch
    at = np.flatnonzero(tok >= 0)
    at = at[np.argsort(tok[at], kind="stable")]
    ids, first, size = np.unique(tok[at], return_index=True, return_counts=True)
    sums = torch.zeros(len(ids), case["d"], dtype=torch.float64, device="cuda")
    if len(ids):
        x = s["dout"].double()[torch.from_numpy(at).cuda()]
        sums = torch.segment_reduce(x, "sum", lengths=torch.from_numpy(size).cuda(), axis=0) * scale
    where = torch.from_numpy(ids).cuda()
    if case["op"] == "gradient":
        out = s["grad"].double() if case["accumulate"] else torch.zeros(s["grad"].shape, dtype=torch.float64, device="cuda")
        out[where] += sums
        return out
    n = len(ids)
    rows, values = torch.zeros_like(s["rows"]), torch.zeros(s["values"].shape, dtype=torch.float64, device="cuda")
    rows[:n] = where.to(torch.int32)
    values[:n] = sums
    # the step reads the sums in their stored type
    g = sums.to(s["values"].dtype).double()
    norm = float(torch.linalg.vector_norm(g))
    factor = min(1.0, MAX_NORM / (norm + CLIP_EPS))
    g = g * factor
    table, m, q = s["table"].double(), s["m"].double(), s["v"].double()
    h = ADAM
    m[where] = torch.lerp(g, m[where], h["beta1"])
    q[where] = torch.lerp(g * g, q[where], h["beta2"])
    root = torch.sqrt(q[where] / (1.0 - math.pow(h["beta2"], h["step"]))) + h["eps"]
    rate = h["lr"] / (1.0 - math.pow(h["beta1"], h["step"]))
    table[where] = table[where] * (1.0 - h["lr"] * h["wd"]) - rate * m[where] / root
    return {"rows": rows, "values": values, "count": torch.full_like(s["count"], n), "result": torch.tensor([norm, factor], dtype=torch.float64), "table": table,
            "m": m, "v": q}


def _exact_stack(s):
    a, b, c = s["coeffs"]
    out = {"new": [], "bufs": []}
    for g, buf, w in zip(s["grads"], s["bufs"], s["new"]):
        d = g.double()
        # the stored momentum keeps its type's rounding: the definition's next line reads it
        t = torch.add(d, buf.double(), alpha=MOMENTUM).to(g.dtype).double()
        y = torch.add(d, t, alpha=MOMENTUM)
        y = y / (torch.linalg.matrix_norm(y)[:, None, None] + NS_EPS)
        left = y.shape[1] <= y.shape[2]
        for _ in range(s["steps"]):
            yt = y.transpose(1, 2).contiguous()
            q = torch.bmm(y, yt) if left else torch.bmm(yt, y)
            poly = torch.baddbmm(q, q, q, beta=b, alpha=c)
            y = a * y + (torch.bmm(poly, y) if left else torch.bmm(y, poly))
        out["new"].append(w.double() * (1.0 - LR * WD) - LR * y if s["case"]["apply"] else y)
        out["bufs"].append(t)
    return out
