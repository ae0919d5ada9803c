"""The embedding table on the Adam path (include/muon_embed.h) through the C
ABI: lookup, gradient by sorted tokens, Adam on the rows of a batch, and the
norm over live rows (muon_clip_plan_set_live_rows).

Tolerances. A lookup is one float32 product rounded once: held bitwise. A sum
of k float32 terms in any order is off by at most (k - 1) 2^-24 times the sum
of their magnitudes (and terms of second order, below 2^-10 of that for k under
2^14); the product with the scale and the addition to what the gradient holds
add 2^-24 of their results each, and the last rounding half a step, eps / 2.
Adam on rows is held bitwise to AdamPlan on the same rows.
"""
import numpy as np
import pytest
import torch

import oracle
from workloads import to_f64

pytestmark = pytest.mark.gpu

mu = pytest.importorskip("muon_newton_schulz_04_amd")
DEV = "cuda"
TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ADAM = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.1, step=7)


def say(msg):
    print(msg, flush=True)


def strided(rows, cols, pad, dtype, gen, scale=1.0, offset=0):
    """(buffer, view): a matrix `offset` elements into its storage, `pad` sentinels behind each row."""
    buf = torch.full((offset + rows * (cols + pad),), 77.0, dtype=TDT[dtype])
    view = buf[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_((scale * torch.randn(rows, cols, generator=gen)).to(TDT[dtype]))
    buf = buf.to(DEV)
    return buf, buf[offset:].view(rows, cols + pad)[:, :cols]


def zipf(n, vocab, gen, padded=0.0):
    t = (torch.exp(torch.rand(n, generator=gen, dtype=torch.float64) * np.log(vocab + 1.0)).long() - 1).clamp(0, vocab - 1)
    return t.masked_fill(torch.rand(n, generator=gen) < padded, -1)


def reference(tokens, dout, vocab, scale):
    """(gradient, bound on the float32 sum's error) in float64."""
    t, x = tokens.cpu().numpy().reshape(-1).astype(np.int64), to_f64(dout).reshape(tokens.numel(), -1)
    live = (t >= 0) & (t < vocab)
    g, mag, k = np.zeros((vocab, x.shape[1])), np.zeros((vocab, x.shape[1])), np.zeros(vocab)
    np.add.at(g, t[live], x[live])
    np.add.at(mag, t[live], np.abs(x[live]))
    np.add.at(k, t[live], 1.0)
    s = float(np.float32(scale))
    err = (np.maximum(k - 1, 0)[:, None] * mag * 1.001 * abs(s) + np.abs(g * s)) * 2.0 ** -24
    return g * s, err, k > 0


def within(got, want, err, dtype):
    half = torch.finfo(TDT[dtype]).eps / 2
    return bool((np.abs(to_f64(got) - want) <= err + half * (np.abs(want) + err) + 1e-38).all())


SIZES = [(1, 1, 1), (1, 50257, 768), (3, 2, 5), (17, 1021, 96), (64, 257, 300), (1000, 5, 33), (4096, 700, 256), (5001, 3000, 765), (12345, 513, 70)]


@pytest.mark.parametrize("n,vocab,cols", SIZES)
@pytest.mark.parametrize("table,act", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
def test_lookup(n, vocab, cols, table, act):
    say(f"lookup {n} {vocab} {cols} {table} {act}")
    gen = torch.Generator().manual_seed(n + cols)
    for index, pad, offset, scale in ((torch.int64, 0, 0, 1.0), (torch.int32, 3, 1, 0.3)):
        _, e = strided(vocab, cols, pad, table, gen, offset=offset)
        obuf, out = strided(n, cols, pad, act, gen, offset=offset)
        tok = zipf(n, vocab, gen, 0.2)
        tok[n // 2] = vocab          # one past the end
        tok[0] = vocab - 1
        tok = tok.to(index).to(DEV)
        plan = mu.EmbeddingPlan(e, n)
        assert plan.lookup(tok, out, scale) is out
        t = tok.cpu().numpy()
        live = (t >= 0) & (t < vocab)
        want = np.where(live[:, None], e.float().cpu().numpy()[np.where(live, t, 0)] * np.float32(scale), np.float32(0))
        assert torch.equal(out.cpu(), torch.from_numpy(want).to(TDT[act]))
        out.fill_(77.0)
        assert bool((obuf == 77.0).all())  # nothing beside the rows was written
        plan.destroy()


@pytest.mark.parametrize("n,vocab,cols", SIZES)
@pytest.mark.parametrize("table,act", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
def test_gradient(n, vocab, cols, table, act):
    """All three forms against float64, twice (equal bits), with sentinels around what is written."""
    say(f"gradient {n} {vocab} {cols} {table} {act}")
    gen = torch.Generator().manual_seed(n * 7 + cols)
    for index, pad, offset, scale, padded in ((torch.int64, 0, 0, 1.0, 0.0), (torch.int32, 5, 1, -0.3, 0.3)):
        _, e = strided(vocab, cols, pad, table, gen, offset=offset)
        _, d = strided(n, cols, pad, act, gen, offset=offset)
        gbuf, g = strided(vocab, cols, pad, table, gen, offset=offset)
        tok = zipf(n, vocab, gen, padded).to(index).to(DEV)
        want, err, live = reference(tok, d, vocab, scale)
        plan = mu.EmbeddingPlan(e, n)
        ws = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device=DEV)  # nothing is read before it is written
        old = to_f64(g)
        first = g.clone()
        plan.gradient(tok, d, first, scale, accumulate=True, workspace=ws)
        total = old + want
        half = torch.finfo(TDT[table]).eps / 2
        bound = err + (np.abs(total) + err) * (half + 2.0 ** -24)
        assert (np.abs(to_f64(first) - total) <= bound).all()
        assert np.array_equal(to_f64(first)[~live], old[~live])  # rows without a token
        assert plan.gradient(tok, d, g, scale, workspace=ws) is g
        assert within(g, want, err, table) and not to_f64(g)[~live].any()
        again = torch.full_like(g, 5.0)
        plan.gradient(tok, d, again, scale)
        assert torch.equal(again, g)
        cap = min(n, vocab)
        rows = torch.full((cap + 1,), -9, dtype=torch.int32, device=DEV)
        values = torch.full((cap + 1, cols), 77.0, dtype=TDT[table], device=DEV)
        count = torch.full((1,), -9, dtype=torch.int32, device=DEV)
        plan.gradient_rows(tok, d, rows, values, count, scale, ws)
        ids = np.flatnonzero(live)
        assert count.item() == len(ids) and np.array_equal(rows.cpu().numpy()[:len(ids)], ids)
        assert torch.equal(values[:len(ids)], g[torch.from_numpy(ids).to(DEV)])
        assert bool((rows[len(ids):] == -9).all()) and bool((values[len(ids):] == 77.0).all())
        g.fill_(77.0)
        assert bool((gbuf == 77.0).all())
        plan.destroy()


@pytest.mark.parametrize("n,vocab", [(70000, 1), (70000, 40000), (4099, 300000)])
def test_gradient_extreme_spreads(n, vocab):
    """One token everywhere, runs that start and end at chunk borders, every token once, and a range of over 1024 entries to a sort block."""
    cols = 40
    gen = torch.Generator().manual_seed(n)
    e = torch.zeros(vocab, cols, device=DEV)
    d = torch.randn(n, cols, generator=gen).to(DEV)
    plan = mu.EmbeddingPlan(e, n)
    g = torch.empty_like(e)
    for name, tok in (("one", torch.full((n,), vocab - 1)), ("runs", torch.arange(n) // 128 % vocab), ("each", torch.randperm(n, generator=gen) % vocab),
                      ("none", torch.full((n,), -1)), ("half", torch.where(torch.arange(n) % 2 == 0, vocab // 2, -5))):
        say(f"gradient {name} n {n} vocab {vocab}")
        tok = tok.to(torch.int64).to(DEV)
        want, err, _ = reference(tok, d, vocab, 1.0)
        assert within(plan.gradient(tok, d, g), want, err, "fp32")
        r = torch.zeros(min(n, vocab), dtype=torch.int32, device=DEV)
        v = torch.zeros(min(n, vocab), cols, device=DEV)
        c = torch.zeros(1, dtype=torch.int32, device=DEV)
        plan.gradient_rows(tok, d, r, v, c)
        ids = np.unique(tok[tok >= 0].cpu().numpy())
        assert c.item() == len(ids) and np.array_equal(r[:len(ids)].cpu().numpy(), ids)
        assert torch.equal(v[:len(ids)], g[torch.from_numpy(ids).to(DEV)])
    plan.destroy()


def test_wild_tokens_touch_nothing():
    """Tokens far outside the vocabulary, in both widths."""
    e = torch.randn(10, 8, device=DEV)
    plan = mu.EmbeddingPlan(e, 8)
    for tok in (torch.tensor([2 ** 40, -2 ** 40, 2 ** 32, 2 ** 32 + 3, 10, -1, 2 ** 63 - 1, -2 ** 63]),
                torch.tensor([2 ** 31 - 1, -2 ** 31, 10, 11, -1, -2, 1 << 24, 1 << 30], dtype=torch.int32)):
        tok = tok.to(DEV)
        out = torch.full((8, 8), 3.0, device=DEV)
        plan.lookup(tok, out)
        assert not out.any()
        g = torch.ones_like(e)
        plan.gradient(tok, torch.full((8, 8), float("nan"), device=DEV), g)
        assert not g.any()
        g.fill_(2.0)
        plan.gradient(tok, torch.full((8, 8), float("nan"), device=DEV), g, accumulate=True)
        assert bool((g == 2.0).all())
    plan.destroy()


def test_no_tokens():
    e = torch.randn(300, 8, device=DEV)
    plan = mu.EmbeddingPlan(e, 0)
    for tok in (torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 5, dtype=torch.int64, device=DEV)):
        d = torch.empty(*tok.shape, 8, device=DEV)
        plan.lookup(tok, d)
        g = torch.ones_like(e)
        plan.gradient(tok, d, g, accumulate=True)
        assert bool((g == 1.0).all())
        plan.gradient(tok, d, g)
        assert not g.any()
        r, v, c = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 8, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
        plan.gradient_rows(tok, d, r, v, c)
        assert c.item() == 0
    plan.destroy()


def test_nan_and_infinity_stay_in_their_rows_and_columns():
    gen = torch.Generator().manual_seed(3)
    e, d = torch.zeros(50, 20, device=DEV), torch.randn(500, 20, generator=gen).to(DEV)
    tok = torch.randint(0, 50, (500,), generator=gen).to(DEV)
    clean = mu.EmbeddingPlan(e, 500).gradient(tok, d, torch.empty_like(e))
    d[7, 3], d[9, 4] = float("nan"), float("inf")
    g = mu.EmbeddingPlan(e, 500).gradient(tok, d, torch.empty_like(e))
    bad = torch.zeros_like(e, dtype=torch.bool)
    bad[tok[7], 3] = bad[tok[9], 4] = True
    assert torch.isnan(g[tok[7], 3]) and torch.isinf(g[tok[9], 4])
    assert torch.equal(g[~bad], clean[~bad])


def test_gradient_is_the_lookups_derivative():
    """Differences of a weighted sum of the lookup, in the table's entries (the lookup is linear: exact up to rounding)."""
    gen = torch.Generator().manual_seed(5)
    n, vocab, cols, scale = 33, 11, 7, 0.75
    e, w = torch.randn(vocab, cols, generator=gen).to(DEV), torch.randn(n, cols, generator=gen).to(DEV)
    tok = torch.randint(-1, vocab, (n,), generator=gen).to(DEV)
    plan = mu.EmbeddingPlan(e, n)
    g = plan.gradient(tok, w, torch.empty_like(e), scale)
    out = torch.empty(n, cols, device=DEV)

    def loss():
        return float((plan.lookup(tok, out, scale).double() * w.double()).sum())

    for v, c in ((0, 0), (3, 6), (10, 2), (7, 1)):
        keep = e[v, c].item()
        e[v, c] = keep + 2.0
        hi, step = loss(), e[v, c].item()
        e[v, c] = keep - 2.0
        step -= e[v, c].item()
        diff = (hi - loss()) / step
        e[v, c] = keep
        # float32 products of values under 8 with 33 weights under 5, over a step of 4
        assert abs(diff - g[v, c].item()) < 33 * 5 * 8 * 2.0 ** -24 * 2


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cols,pad", [(768, 0), (1, 0), (7, 3), (1021, 0), (2052, 8)])
def test_adam_rows_is_adam_on_those_rows(dtype, cols, pad):
    say(f"adam rows {dtype} {cols} {pad}")
    gen = torch.Generator().manual_seed(cols)
    vocab, cap = 97, 60
    buf, e = strided(vocab, cols, pad, dtype, gen, 0.02, offset=1)
    m, v = 1e-2 * torch.randn(vocab, cols, generator=gen).to(DEV), 1e-3 * torch.rand(vocab, cols, generator=gen).to(DEV)
    rows = torch.randperm(vocab, generator=gen)[:cap].to(torch.int32).to(DEV)
    values = (0.1 * torch.randn(cap, cols, generator=gen)).to(TDT[dtype]).to(DEV)
    scale = torch.full((1,), 0.37, device=DEV)
    for count, factor in ((0, None), (1, None), (41, scale), (60, None), (100, scale), (-3, None)):
        live = max(0, min(count, cap))
        at = rows[:live].long()
        p2, m2, v2 = e[at].contiguous(), m[at].contiguous(), v[at].contiguous()
        before = [x.clone() for x in (buf, m, v)]
        if live:
            dense = mu.AdamPlan([p2], [values[:live].contiguous()], [m2], [v2], [0.7], [0.5])
            dense.set_grad_scale(factor)
            dense.step(**ADAM)
        plan = mu.EmbeddingPlan(e, 8, m, v, lr_mul=0.7, wd_mul=0.5)
        plan.set_grad_scale(factor)
        plan.adam_rows(rows, values, torch.tensor([count], dtype=torch.int32, device=DEV), **ADAM)
        assert torch.equal(e[at], p2) and torch.equal(m[at], m2) and torch.equal(v[at], v2)
        rest = torch.ones(vocab, dtype=torch.bool, device=DEV)
        rest[at] = False
        old = before[0][1:].view(vocab, cols + pad)
        assert torch.equal(e[rest], old[:, :cols][rest]) and torch.equal(m[rest], before[1][rest]) and torch.equal(v[rest], before[2][rest])
        if pad:
            assert bool((buf[1:].view(vocab, cols + pad)[:, cols:] == 77.0).all())
    # rows outside the table are skipped
    before = [x.clone() for x in (buf, m, v)]
    wild = torch.tensor([-1, vocab, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    plan.adam_rows(wild, values[:4], torch.tensor([4], dtype=torch.int32, device=DEV), **ADAM)
    assert all(torch.equal(a, b) for a, b in zip(before, (buf, m, v)))
    plan.destroy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cap,cols", [(5, 3), (4000, 96), (9000, 768)])
def test_norm_and_clip_over_live_rows(dtype, cap, cols):
    """The norm of a list whose tensor has live rows is that of the list with the rest cut off; nothing behind them is written or read."""
    say(f"live rows {dtype} {cap} {cols}")
    gen = torch.Generator().manual_seed(cap)
    values = (0.1 * torch.randn(cap, cols, generator=gen)).to(TDT[dtype]).to(DEV)
    other = (0.1 * torch.randn(50, 7, generator=gen)).to(DEV)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)
    plan = mu.ClipPlan([other, values])
    plan.set_live_rows(1, count)
    norms = torch.zeros(2, device=DEV)
    for live in (0, 1, cap // 3, cap - 1, cap, cap + 5, -2):
        n = max(0, min(cap, live))
        v = values.clone()
        v[n:] = float("nan")
        values.copy_(v)
        o = other.clone()
        count.fill_(live)
        r = plan.norm(0.5, norms=norms).double().tolist()
        want, each = oracle.gradient_norms([to_f64(other), to_f64(v[:n])])
        for a, b in zip([r[0], *norms.double().tolist()], [want, *each]):
            assert abs(a - b) <= (2.0 ** -24 + 2.0 ** -36) * b
        s = plan.step(0.5)[1].item()
        assert torch.equal(values[:n], (v[:n].float() * s).to(values.dtype)) and bool(torch.isnan(values[n:]).all())
        assert torch.equal(other, o * s)
        values.copy_(torch.nan_to_num(v, 0.25))
        other.copy_(o)
    plan.set_live_rows(1, None)
    want, _ = oracle.gradient_norms([to_f64(other), to_f64(values)])
    assert abs(plan.norm()[0].item() - want) <= (2.0 ** -24 + 2.0 ** -36) * want
    plan.destroy()


def test_live_rows_refusals():
    a = torch.zeros(64, 64, device=DEV)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)
    plan = mu.ClipPlan([a, a[:, :32], a], [None] * 3)
    for i, c, cols, code in ((1, count, 32, 3), (0, count, 63, 3), (0, count, 0, 3)):
        with pytest.raises(mu.MuonError) as exc:
            plan.set_live_rows(i, c, cols)
        assert exc.value.code == code
    with pytest.raises(ValueError):
        plan.set_live_rows(0, torch.zeros(1, device=DEV))
    with pytest.raises(IndexError):
        plan.set_live_rows(3, count)
    plan.set_live_rows(-1, count)
    assert plan.norm()[0].item() == 0.0
    plan.destroy()


def test_call_refusals():
    """Arguments the library or the binding turns away, before anything is enqueued."""
    e = torch.randn(20, 8, device=DEV)
    m, v = torch.zeros_like(e), torch.zeros_like(e)
    plan = mu.EmbeddingPlan(e, 4)
    tok = torch.zeros(4, dtype=torch.int64, device=DEV)
    x, g = torch.zeros(4, 8, device=DEV), torch.zeros_like(e)
    rows, vals = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(4, 8, device=DEV)
    count = torch.ones(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    long = torch.zeros(5, dtype=torch.int64, device=DEV)

    def code(fn, *args, **kw):
        with pytest.raises(mu.MuonError) as exc:
            fn(*args, **kw)
        return exc.value.code

    assert code(plan.lookup, long, torch.zeros(5, 8, device=DEV)) == 3             # more than max_tokens
    assert code(plan.lookup, tok, x, float("nan")) == 1
    assert code(plan.lookup, tok, e[:4]) == 1                                      # into the table
    assert code(plan.gradient, tok, x, g, float("inf")) == 1
    assert code(plan.gradient, tok, x, e) == 1                                     # over the table
    assert code(plan.gradient, tok, g[:4], g) == 1                                 # dout inside grad
    assert code(plan.gradient, tok, x, g, workspace=ws[:-1]) == 5
    assert code(plan.gradient, tok, x, g, workspace=torch.empty(plan.workspace_bytes + 8, dtype=torch.uint8, device=DEV)[8:]) == 5
    assert code(plan.gradient_rows, tok, vals, rows, vals, count) == 1             # values over dout
    assert code(plan.gradient_rows, tok, x, rows, vals, rows[:1]) == 1             # count inside rows
    assert code(plan.adam_rows, rows, vals, count, **ADAM) == 1                    # no moments
    full = mu.EmbeddingPlan(e, 4, m, v)
    assert code(full.adam_rows, rows, vals, count, **{**ADAM, "step": 0}) == 1
    assert code(full.adam_rows, rows, vals, count, **{**ADAM, "beta2": 1.0}) == 1
    assert code(full.adam_rows, rows, e[:4], count, **ADAM) == 1                   # gradients inside the table
    for bad in (tok.float(), tok.cpu(), torch.zeros(8, dtype=torch.int64, device=DEV)[::2]):
        with pytest.raises((TypeError, ValueError)):
            plan.lookup(bad, x)
    for bad in (x[:3], x.half(), torch.zeros(4, 16, device=DEV)[:, ::2], x.cpu()):
        with pytest.raises((TypeError, ValueError)):
            plan.lookup(tok, bad)
    with pytest.raises(ValueError):
        plan.gradient(tok, x, g.bfloat16())
    with pytest.raises(ValueError):
        plan.gradient_rows(tok, x, rows[:3], vals[:3], count)                      # no room
    with pytest.raises(ValueError):
        plan.set_grad_scale(torch.zeros(2, device=DEV))
    assert not g.any() and not x.any()


def test_captured_gradient_and_rows_step_replay():
    """Lookup, rows, norm over live rows and the rows' Adam step in one graph, replayed on changing tokens against eager calls."""
    gen = torch.Generator().manual_seed(11)
    n, vocab, cols = 3000, 2000, 96
    tok = zipf(n, vocab, gen, 0.1).to(DEV)
    e0 = torch.randn(vocab, cols, generator=gen).bfloat16().to(DEV)
    d = (0.1 * torch.randn(n, cols, generator=gen)).bfloat16().to(DEV)

    def make():
        s = dict(e=e0.clone(), m=torch.zeros(vocab, cols, device=DEV), v=torch.zeros(vocab, cols, device=DEV),
                 out=torch.zeros(n, cols, dtype=torch.bfloat16, device=DEV), rows=torch.zeros(vocab, dtype=torch.int32, device=DEV),
                 values=torch.zeros(vocab, cols, dtype=torch.bfloat16, device=DEV), count=torch.zeros(1, dtype=torch.int32, device=DEV),
                 grad=torch.zeros(vocab, cols, dtype=torch.bfloat16, device=DEV))
        plan = mu.EmbeddingPlan(s["e"], n, s["m"], s["v"])
        clip = mu.ClipPlan([s["values"]], [None])
        clip.set_live_rows(0, s["count"])
        plan.set_grad_scale(clip.scale)
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
        cws = torch.empty(clip.workspace_bytes, dtype=torch.uint8, device=DEV)

        def step():
            plan.lookup(tok, s["out"], 1.5)
            plan.gradient(tok, d, s["grad"], workspace=ws)
            plan.gradient_rows(tok, d, s["rows"], s["values"], s["count"], workspace=ws)
            clip.norm(1.0, workspace=cws)
            plan.adam_rows(s["rows"], s["values"], s["count"], **ADAM)
        return s, step, (plan, clip)

    eager, step, keep = make()
    graphed, gstep, gkeep = make()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gstep()
    for k in range(4):
        tok.copy_(zipf(n, vocab, gen, 0.1 * k))
        d.copy_((0.1 * torch.randn(n, cols, generator=gen)).bfloat16())
        torch.cuda.synchronize()
        step()
        graph.replay()
        torch.cuda.synchronize()
        for key in eager:
            assert torch.equal(eager[key], graphed[key]), (k, key)


def test_two_streams_with_a_workspace_each():
    gen = torch.Generator().manual_seed(2)
    n, vocab, cols = 20000, 5000, 128
    e = torch.randn(vocab, cols, generator=gen).to(DEV)
    d = torch.randn(n, cols, generator=gen).to(DEV)
    toks = [zipf(n, vocab, gen, 0.1).to(DEV) for _ in range(2)]
    plan = mu.EmbeddingPlan(e, n)
    want = [plan.gradient(t, d, torch.empty_like(e)) for t in toks]
    got = [torch.empty_like(e) for _ in toks]
    streams = [torch.cuda.Stream() for _ in toks]
    torch.cuda.synchronize()
    for _ in range(5):
        for t, g, s in zip(toks, got, streams):
            plan.gradient(t, d, g, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_past_32_bits():
    """A table of over 2^31 elements: rows at its far end."""
    vocab, cols = 2_900_000, 768
    e = torch.zeros(vocab, cols, dtype=torch.bfloat16, device=DEV)
    e[-3:] = torch.randn(3, cols, device=DEV).bfloat16()
    tok = torch.tensor([vocab - 1, vocab - 3, 0, vocab - 1, vocab - 2], device=DEV)
    plan = mu.EmbeddingPlan(e, 5)
    out = torch.empty(5, cols, dtype=torch.bfloat16, device=DEV)
    assert torch.equal(plan.lookup(tok, out), e[tok])
    g = torch.ones_like(e)
    d = torch.randn(5, cols, device=DEV).bfloat16()
    plan.gradient(tok, d, g)
    assert torch.equal(g[vocab - 1], (d[0].float() + d[3].float()).bfloat16())
    assert torch.equal(g[vocab - 2], d[4]) and torch.equal(g[vocab - 3], d[1]) and torch.equal(g[0], d[2])
    g[[0, vocab - 1, vocab - 2, vocab - 3]] = 0
    assert not bool(g.any())
    plan.destroy()


def test_many_tokens():
    """More tokens than one sort pass keeps in flight, long enough for the largest chunks, against float64 on the GPU."""
    gen = torch.Generator().manual_seed(4)
    n, vocab, cols = 1_500_001, 50257, 8
    tok = zipf(n, vocab, gen, 0.02).to(torch.int32).to(DEV)
    d = torch.randn(n, cols, generator=gen).to(DEV)
    e = torch.zeros(vocab, cols, device=DEV)
    g = mu.EmbeddingPlan(e, n).gradient(tok, d, torch.empty_like(e))
    t = tok.long()
    live = t >= 0
    want = torch.zeros(vocab, cols, dtype=torch.float64, device=DEV).index_add_(0, t[live], d[live].double())
    mag = torch.zeros(vocab, cols, dtype=torch.float64, device=DEV).index_add_(0, t[live], d[live].double().abs())
    # a run of 64 terms is summed in turn, then up to 2^11 runs' sums, four lists of them: 64 + 2^9 + 4 additions deep at most
    depth = 64 + 512 + 4
    assert bool(((g.double() - want).abs() <= depth * 2.0 ** -24 * 1.001 * mag + 2.0 ** -24 * want.abs()).all())


def test_gradient_of_a_broadcast_dout():
    """Rows that share elements are refused; a copy of them gives the gradient (that of a sum over the lookup's rows)."""
    vocab, cols = 6, 40
    e = torch.zeros(vocab, cols, device=DEV)
    tok = torch.tensor([0, 3, 3, -1, 5, 3], device=DEV)
    plan = mu.EmbeddingPlan(e, 6)
    row = torch.arange(cols, dtype=torch.float32, device=DEV)
    leaf = torch.zeros(6, cols, device=DEV, requires_grad=True)
    d = torch.autograd.grad((leaf + 0).sum(0), leaf, row)[0]
    assert d.stride() == (0, 1)
    g = torch.full_like(e, 7.0)
    rows, vals = torch.zeros(6, dtype=torch.int32, device=DEV), torch.zeros(6, cols, device=DEV)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)
    for call in (lambda: plan.gradient(tok, d, g), lambda: plan.gradient_rows(tok, d, rows, vals, count), lambda: plan.lookup(tok, d),
                 lambda: plan.gradient(tok, d.contiguous(), row.expand(vocab, cols)), lambda: mu.EmbeddingPlan(row.expand(vocab, cols), 6)):
        with pytest.raises(ValueError):
            call()
    assert bool((g == 7.0).all()) and not rows.any() and not count.any()
    plan.gradient(tok, d.contiguous(), g)
    assert torch.equal(g, torch.tensor([1.0, 0, 0, 3, 0, 1], device=DEV)[:, None] * row)
    plan.destroy()


def test_live_rows_of_a_permuted_tensor_are_refused():
    x = torch.randn(6, 4, device=DEV)
    count = torch.ones(1, dtype=torch.int32, device=DEV)
    plan = mu.ClipPlan([x.t()], [None])
    with pytest.raises(mu.MuonError) as exc:
        plan.set_live_rows(0, count)
    assert exc.value.code == 3
    want = torch.linalg.vector_norm(x.double()).item()
    assert abs(plan.norm()[0].item() - want) <= 2.0 ** -23 * want  # all of it, as before
    plan.destroy()


def test_lookup_of_the_most_tokens_of_wide_rows():
    """2^24 tokens of 4097 columns, where a block for each token would be more threads than a launch holds."""
    n, cols, vocab = 1 << 24, 4097, 37
    need = n * (2 * cols + 16) + (8 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GB of free device memory")
    e = torch.randn(vocab, cols, device=DEV).bfloat16()
    tok = torch.randint(-1, vocab, (n,), device=DEV, dtype=torch.int32, generator=torch.Generator(device=DEV).manual_seed(1))
    out = torch.empty(n, cols, dtype=torch.bfloat16, device=DEV)
    plan = mu.EmbeddingPlan(e, n)
    plan.lookup(tok, out)
    rows = torch.cat([e, torch.zeros(1, cols, dtype=e.dtype, device=DEV)])  # (-1 is the last one)
    step = 1 << 18
    for i in range(0, n, step):
        assert torch.equal(out[i:i + step], rows[tok[i:i + step].long()]), i
    plan.destroy()
    del out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("form", ["dense", "added", "rows"])
@pytest.mark.parametrize("n", [1 << 16, 300_001, 1 << 22])
def test_sums_of_one_frequent_token(n, form):
    """Equal rows, whose partial sums are all rounded the same way once a float32 sum outgrows them. Runs of 64 terms leave
    63 roundings of 2^-24 of the sum of magnitudes; adding the runs' sums in float64 (under 2^19 of them) under 2^-34 of
    it; then the roundings to float32, of the product and of the addition."""
    cols = 12
    e = torch.zeros(4, cols, device=DEV)
    row = torch.linspace(0.1, 1.2, cols, device=DEV)
    d = row.repeat(n, 1)
    tok = torch.full((n,), 2, dtype=torch.int32, device=DEV)
    want = n * row.double()
    plan = mu.EmbeddingPlan(e, n)
    if form == "rows":
        rows, vals, count = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(4, cols, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        got = plan.gradient_rows(tok, d, rows, vals, count)[1][0]
        assert count.item() == 1 and rows[0].item() == 2
    else:
        got = plan.gradient(tok, d, torch.zeros_like(e), accumulate=form == "added")[2]
    off = ((got.double() - want).abs() / want).max().item()
    say(f"{n} equal rows, {form}: off by {off:.1e}")
    assert off <= (63 + 3 + 2.0 ** -10) * 2.0 ** -24
    plan.destroy()
