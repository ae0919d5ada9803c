"""The Muon step on stacks of short matrices (include/muon_stack.h) through
the C ABI, against the float64 oracle matrix by matrix.

Tolerances. Momentum buffers are the exact value rounded once: held bitwise.
For X: every product takes its operands to 2^-22 and sums in float32, so one
step leaves an error of about |a| + |b| + |c| < 12 times 2^-22, relative to X's
norm; a step multiplies an earlier error by at most |a| (along singular values
near zero). Over five quintic steps that is 12 2^-22 (3.44^0 + .. + 3.44^4) <
6e-4 in directions of singular value zero if every error lay in them: LOW for
fp32 sets, which form A anew in every step of the quintic. bf16 sets take five
steps from one A. An error of A, 2^-23 of its largest eigenvalue (half the last
place of the two fp16 numbers), grows along eigenvalues near zero by a^2 = 11.86
in each of four updates, and moves the last step's factor a + b lambda there by
|b| / |a| of what it has become: 1.39 11.86^4 2^-23 = 3.3e-3, LOW for bf16 sets
(inputs of rank one, all of whose other directions are such). Spread over all
directions, as rounding errors are on inputs of full rank, an emulation of the
same arithmetic in numpy stays below 1.1e-5 on shapes up to 128 x 2048 (4.5e-6
for fp32 sets, 6.4e-5 on square 128 x 128); TOL is ten times the first. bf16
outputs add half a step, 2^-8 of the value, per element (taken off before the
norm of what is left is compared). Weights: the same error times lr', and two
float32 roundings of the terms.
"""
import numpy as np
import pytest
import torch

import oracle
from workloads import CONFIGS, to_f64

pytestmark = pytest.mark.gpu

mu = pytest.importorskip("muon_newton_schulz_04_amd")
DEV = "cuda"
TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}
f32 = lambda x: float(np.float32(x))  # noqa: E731
QUINTIC = tuple(f32(x) for x in CONFIGS["gpt2_small_block"].coeffs)
CUBIC = (1.5, -0.5, 0.0)
MU, EPS = f32(0.95), f32(1e-7)
TOL, LOW = 1.1e-4, {"bf16": 3.3e-3, "fp32": 6e-4}


def say(msg):
    print(msg, flush=True)


def config(coeffs=QUINTIC, steps=5, momentum=MU, nesterov=True):
    return mu.make_config(*coeffs, steps, momentum, nesterov, EPS)


def view(count, rows, cols, dtype, gen, scale=0.05, side=False, pad=0, offset=0, strong=0.0):
    """(buffer, 3-D view): row blocks of one matrix, or column blocks of one; sentinels around."""
    x = scale * torch.randn(count, rows, cols, generator=gen)
    if strong:
        x += strong * torch.randn(count, rows, 3, generator=gen) @ torch.randn(count, 3, cols, generator=gen)
    ld = (count * cols if side else cols) + pad
    stride = cols if side else rows * ld
    buf = torch.full((offset + (rows if side else count * rows) * ld,), 77.0, dtype=TDT[dtype])
    buf[offset:].as_strided((count, rows, cols), (stride, ld, 1)).copy_(x)
    buf = buf.to(DEV)
    return buf, buf[offset:].as_strided((count, rows, cols), (stride, ld, 1))


def oracle_x(g, b, cfg_coeffs, steps, momentum, nesterov, dtype):
    """(X before rounding, buffer) in float64."""
    a, bb, c = cfg_coeffs
    if momentum == 0.0:
        return oracle.orthogonalize(g, a, bb, c, steps, EPS), None
    return oracle.muon_update(g, b, a=a, b=bb, c=c, steps=steps, mu=momentum, nesterov=nesterov, eps=EPS, buf_dtype=dtype)


def left_over(got, want, dtype):
    """Norm of the error beyond half a step of the output's type, relative to the norm of what is wanted."""
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    off = np.maximum(np.abs(got - want) - half * np.abs(want), 0.0)
    return np.linalg.norm(off) / max(np.linalg.norm(want), 1e-300)


def check(shape, dtype, coeffs=QUINTIC, steps=5, momentum=MU, nesterov=True, tol=TOL, seed=0, sample=None, grads=None, **kw):
    count, rows, cols = shape
    gen = torch.Generator().manual_seed(seed + rows * 31 + cols)
    gbuf, g = view(count, rows, cols, dtype, gen, strong=0.03, **kw) if grads is None else grads
    bbuf, b = view(count, rows, cols, dtype, gen, **kw)
    obuf, o = view(count, rows, cols, dtype, gen, **kw)
    g0, b0 = gbuf.clone(), to_f64(b)
    plan = mu.StackPlan([g], [b] if momentum else None, [o])
    ws = torch.full((max(1, plan.workspace_bytes),), 255, dtype=torch.uint8, device=DEV)
    plan.step(config(coeffs, steps, momentum, nesterov), ws)
    torch.cuda.synchronize()
    assert torch.equal(gbuf, g0)
    got, new, gf = to_f64(o), to_f64(b), to_f64(g)
    worst = 0.0
    for t in range(count) if sample is None else sample:
        want, buf = oracle_x(gf[t], b0[t], coeffs, steps, momentum, nesterov, dtype)
        worst = max(worst, left_over(got[t], want, dtype))
        if momentum:
            assert np.array_equal(new[t], buf), t
    say(f"{shape} {dtype} k {steps}: {worst:.2e}")
    assert worst <= tol, worst
    for buf, v in ((bbuf, b), (obuf, o)):  # nothing beside the matrices was written
        v.fill_(77.0)
        assert bool((buf == 77.0).all())
    plan.destroy()


SHAPES = [(3, 64, 768), (5, 768, 64), (2, 1, 5), (2, 5, 1), (1, 1, 1), (1, 128, 128), (4, 16, 765), (4, 765, 16), (2, 103, 141), (2, 141, 103),
          (1, 128, 2049), (3, 33, 70), (3, 70, 33), (2, 64, 64), (1, 32, 129), (1, 129, 32), (2, 65, 1000), (7, 4, 300)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_step_in_parts(shape, dtype):
    check(shape, dtype)
    check(shape, dtype, pad=3, offset=1, seed=1)
    check(shape, dtype, side=True, pad=5, offset=3, seed=2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(300, 8, 40), (260, 64, 200), (257, 200, 64), (257, 128, 130), (256, 130, 128), (256, 20, 515)], ids=str)
def test_step_a_matrix_a_workgroup(shape, dtype):
    """Enough matrices for whole ones, and runs of several, to fall to a workgroup."""
    sample = (0, 1, 7, 100, shape[0] - 1)
    check(shape, dtype, sample=sample)
    check(shape, dtype, side=True, pad=1, offset=1, seed=3, sample=sample)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(2, 64, 300), (260, 64, 65), (2, 300, 128), (2, 24, 300)], ids=str)
def test_steps_and_coefficients(shape, dtype):
    sample = (0, shape[0] - 1)
    for steps in (0, 1, 2, 3, 4, 6, 7, 13):
        check(shape, dtype, steps=steps, seed=steps, sample=sample)
    for steps in (1, 8, 10, 23):
        check(shape, dtype, CUBIC, steps, seed=steps, sample=sample)
    check(shape, dtype, (1.0, 0.0, 0.0), 3, sample=sample)  # the identity
    check(shape, dtype, momentum=0.0, sample=sample)
    check(shape, dtype, nesterov=False, sample=sample)


@pytest.mark.parametrize("shape", [(1, 128, 65536), (1, 65536, 100), (1, 3, 65536)], ids=str)
def test_longest_sides(shape):
    check(shape, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(2, 64, 256), (256, 40, 100), (2, 300, 8), (2, 128, 300)], ids=str)
def test_low_rank_and_zeros(shape, dtype):
    """Rank one, rank two, spectra over three decades, and a zero matrix among them."""
    count, rows, cols = shape
    gen = torch.Generator().manual_seed(rows)
    m = min(rows, cols)
    x = torch.randn(count, rows, 1, generator=gen) @ torch.randn(count, 1, cols, generator=gen)
    q = torch.linalg.qr(torch.randn(rows, m, generator=gen))[0], torch.linalg.qr(torch.randn(cols, m, generator=gen))[0]
    x[1] = q[0] @ torch.diag(torch.logspace(0, -3, m)) @ q[1].t()
    for zero in (False, True):
        if zero:
            x[0] = 0.0
        g = x.to(TDT[dtype]).to(DEV)
        b = torch.zeros_like(g)
        o = torch.full_like(g, 5.0)
        plan = mu.StackPlan([g], [b], [o])
        plan.step(config())
        for t in (0, 1, count - 1):
            want, buf = oracle_x(to_f64(g[t]), np.zeros((rows, cols)), QUINTIC, 5, MU, True, dtype)
            e = left_over(to_f64(o[t]), want, dtype)
            say(f"{shape} {dtype} matrix {t} zero {zero}: {e:.2e}")
            assert e <= LOW[dtype] and np.array_equal(to_f64(b[t]), buf)
        if zero:
            assert not o[0].any() and not b[0].any()
        plan.destroy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scale_of_the_gradient(dtype):
    """X does not depend on the gradient's scale, over the type's range; columns far below the rest keep their part."""
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(2, 48, 200, generator=gen)
    x[:, :, :50] *= 2.0 ** -20
    first = want = None
    for k in (0, 100, -100, 126, -80):
        g = (x * 2.0 ** (k - 3)).to(TDT[dtype]).to(DEV)
        o = torch.empty_like(g)
        plan = mu.StackPlan([g], None, [o])
        plan.step(mu.make_config(*QUINTIC, 5, 0.0, False, 0.0))
        if want is None:
            first, want = to_f64(g), o.clone()
        for t in range(2):
            assert left_over(to_f64(o[t]), oracle.orthogonalize(to_f64(g[t]), *QUINTIC, 5, 0.0), dtype) <= TOL
        # Equal bits where the gradients are the first ones times 2^k. At k = -100 some of the small columns' entries are
        # not: they lie below the smallest normal number, 2^-126, and are stored as multiples of 2^-133 (bf16) or 2^-149.
        if np.array_equal(to_f64(g), first * 2.0 ** k):
            assert torch.equal(o, want), k
        else:
            assert k == -100 and np.abs(first[to_f64(g) != first * 2.0 ** k]).max() * 2.0 ** k < 2.0 ** -126
        plan.destroy()
    # a norm below eps
    g = (x * 2.0 ** -40).to(TDT[dtype]).to(DEV)
    o = torch.empty_like(g)
    mu.StackPlan([g], None, [o]).step(config(momentum=0.0))
    for t in range(2):
        assert left_over(to_f64(o[t]), oracle.orthogonalize(to_f64(g[t]), *QUINTIC, 5, EPS), dtype) <= TOL


@pytest.mark.parametrize("count", [3, 256])
@pytest.mark.parametrize("rows,cols", [(8, 100), (64, 130), (130, 64), (128, 200)])
def test_nan_and_infinity_stay_in_their_matrix(count, rows, cols):
    gen = torch.Generator().manual_seed(1)
    g = torch.randn(count, rows, cols, generator=gen).to(DEV)
    clean, o = torch.empty_like(g), torch.empty_like(g)
    mu.StackPlan([g], None, [clean]).step(config(momentum=0.0))
    g[0, rows - 1, 2], g[2, 0, cols - 1] = float("nan"), float("inf")
    mu.StackPlan([g], None, [o]).step(config(momentum=0.0))
    torch.cuda.synchronize()
    assert bool(torch.isnan(o[0]).any()) and bool(torch.isnan(o[2]).any())
    keep = [t for t in range(count) if t not in (0, 2)]
    assert torch.equal(o[keep], clean[keep])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(3, 64, 300), (256, 64, 100), (2, 300, 128), (3, 5, 77)], ids=str)
def test_weights(shape, dtype):
    """W <- W (1 - lr' wd') - lr' X, weights in a layout of their own, on a gradient factor; `out` stays as it is."""
    count, rows, cols = shape
    lr, wd, lm, wm, factor = f32(0.02), f32(0.3), f32(0.5), f32(1.5), f32(0.37)
    gen = torch.Generator().manual_seed(cols)
    _, g = view(count, rows, cols, dtype, gen, strong=0.03)
    _, b = view(count, rows, cols, dtype, gen)
    _, o = view(count, rows, cols, dtype, gen)
    wbuf, w = view(count, rows, cols, dtype, gen, side=True, pad=3, offset=1)
    o0, b0, w0 = o.clone(), to_f64(b), to_f64(w)
    plan = mu.StackPlan([g], [b], [o])
    with pytest.raises(mu.MuonError) as exc:
        plan.step_apply(config(), lr, wd)
    assert exc.value.code == 1                             # no weights yet
    plan.set_weights([w], [lm], [wm])
    scale = torch.tensor([factor], device=DEV)
    plan.set_grad_scale(scale)
    plan.step_apply(config(), lr, wd)
    torch.cuda.synchronize()
    assert torch.equal(o, o0)
    lr1, wd1 = f32(np.float32(lr) * np.float32(lm)), f32(np.float32(wd) * np.float32(wm))
    keep = f32(1 - np.float32(lr1) * np.float32(wd1))
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for t in {0, 1, count - 1}:
        gt = np.float32(to_f64(g[t])) * np.float32(factor)
        x, buf = oracle_x(gt.astype(np.float64), b0[t], QUINTIC, 5, MU, True, dtype)
        assert np.array_equal(to_f64(b[t]), buf)
        want = w0[t] * keep - lr1 * x
        off = np.maximum(np.abs(to_f64(w[t]) - want) - half * np.abs(want) - 2.0 ** -23 * (np.abs(w0[t]) + lr1 * np.abs(x)), 0.0)
        assert np.linalg.norm(off) <= TOL * lr1 * np.linalg.norm(x)
    w.fill_(77.0)
    assert bool((wbuf == 77.0).all())
    plan.destroy()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(170, 16, 765), (171, 16, 765), (171, 765, 16), (3, 515, 4), (260, 515, 4)], ids=str)
def test_short_sides_in_small_and_large_sets(shape, dtype):
    """170 matrices of 6 tiles are a set whose workgroups solve for P themselves, 171 are not; one run of steps and several."""
    sample = (0, 1, shape[0] - 1)
    check(shape, dtype, sample=sample)
    check(shape, dtype, CUBIC, 10, sample=sample, seed=1)
    check(shape, dtype, CUBIC, 23, side=True, pad=1, offset=1, sample=sample, seed=2)
    test_weights(shape, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_aliases_steps_in_a_row_and_equal_bits(dtype):
    """out may be the gradient; two plans on equal inputs give equal bits, over three steps; a factor of one changes nothing."""
    gen = torch.Generator().manual_seed(8)
    shapes = [(5, 64, 200), (3, 200, 128), (300, 16, 40), (1, 40, 16)]
    one = torch.ones(1, device=DEV)
    runs = []
    for alias, factor in ((False, None), (True, None), (False, one)):
        gen.manual_seed(8)
        bufs = [view(*s, dtype, gen)[1] for s in shapes]
        outs = []
        for _ in range(3):
            grads = [view(*s, dtype, gen, strong=0.02)[1] for s in shapes]
            out = grads if alias else [torch.empty_strided(g.shape, g.stride(), dtype=g.dtype, device=DEV) for g in grads]
            plan = mu.StackPlan(grads, bufs, out)
            plan.set_grad_scale(factor)
            plan.step(config())
            torch.cuda.synchronize()
            outs.append([x.clone() for x in out])
            plan.destroy()
        runs.append((outs, bufs))
    for outs, bufs in runs[1:]:
        assert all(torch.equal(a, b) for x, y in zip(outs, runs[0][0]) for a, b in zip(x, y))
        assert all(torch.equal(a, b) for a, b in zip(bufs, runs[0][1]))


def test_agrees_with_the_plan_of_single_matrices():
    """The same heads through MuonPlan: within both sides' tolerances (2e-2 is that plan's)."""
    gen = torch.Generator().manual_seed(4)
    w = (0.05 * torch.randn(12 * 64, 768, generator=gen)).bfloat16().to(DEV)
    heads = w.view(12, 64, 768)
    b1, b2 = torch.zeros_like(w), torch.zeros_like(w)
    o1, o2 = torch.empty_like(w), torch.empty_like(w)
    mu.StackPlan([heads], [b1.view(12, 64, 768)], [o1.view(12, 64, 768)]).step(config())
    cut = lambda x: [x[64 * i:64 * i + 64] for i in range(12)]  # noqa: E731
    mu.MuonPlan(cut(w), cut(b2), cut(o2)).step(config())
    torch.cuda.synchronize()
    assert torch.equal(b1, b2)
    assert (o1.float() - o2.float()).norm() <= (2e-2 + 2.0 ** -8) * o2.float().norm()


def test_graph_replays_match_eager():
    gen = torch.Generator().manual_seed(6)
    shapes = [(3, 64, 300), (256, 20, 64), (2, 300, 100)]

    def make():
        gen.manual_seed(6)
        g, b, w = ([view(*s, "bf16", gen)[1] for s in shapes] for _ in range(3))
        plan = mu.StackPlan(g, b, g)
        plan.set_weights(w)
        return g, b, w, plan, torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)

    eager, graphed = make(), make()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        graphed[3].step_apply(config(), 0.02, 0.01, graphed[4])
    for k in range(4):
        for x, y in zip(eager[0], graphed[0]):
            x.copy_(0.05 * torch.randn(x.shape, generator=gen).to(DEV))
            y.copy_(x)
        torch.cuda.synchronize()
        eager[3].step_apply(config(), 0.02, 0.01, eager[4])
        graph.replay()
        torch.cuda.synchronize()
        for i in (1, 2):
            assert all(torch.equal(a, b) for a, b in zip(eager[i], graphed[i])), k


def test_two_streams_with_a_workspace_each():
    gen = torch.Generator().manual_seed(9)
    sets = [[view(40, 64, 500, "bf16", gen)[1] for _ in range(2)] for _ in range(2)]
    want = []
    for g, o in sets:
        mu.StackPlan([g], None, [o]).step(config(momentum=0.0))
        want.append(o.clone())
    plans = [mu.StackPlan([g], None, [o]) for g, o in sets]
    streams = [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(plans, streams):
            p.step(config(momentum=0.0), stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for a, (_, o) in zip(want, sets))


@pytest.mark.parametrize("shape", [(40, 16, 765), (180, 16, 765), (30, 64, 500), (5, 128, 900)], ids=str)
def test_two_graphs_of_one_plan_at_once(shape):
    """One plan, captured twice with a workspace each, replayed at once on two streams: several runs of steps (fp32), no
    state in the plan."""
    gen = torch.Generator().manual_seed(12)
    g, o = (view(*shape, "fp32", gen)[1] for _ in range(2))
    plan = mu.StackPlan([g], None, [o])
    cfg = config(CUBIC, 7, momentum=0.0)
    plan.step(cfg)
    torch.cuda.synchronize()
    want = o.clone()
    graphs, spaces = [], [torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for ws in spaces:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.step(cfg, ws)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for k in range(4):
        o.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), k  # both write the same bits


def test_call_refusals():
    g = torch.randn(2, 8, 40, device=DEV)
    b, o, w = torch.zeros_like(g), torch.full_like(g, 3.0), torch.zeros_like(g)
    plan = mu.StackPlan([g], [b], [o])
    ws = torch.empty(plan.workspace_bytes + 256, dtype=torch.uint8, device=DEV)

    def code(fn, *args, **kw):
        with pytest.raises(mu.MuonError) as exc:
            fn(*args, **kw)
        return exc.value.code

    assert code(plan.step, config(), ws[:plan.workspace_bytes - 1]) == 5
    assert code(plan.step, config(), ws[8:]) == 5
    assert code(plan.step, config(steps=-1)) == 1 and code(plan.step, config(steps=65)) == 1
    assert code(plan.step, config((4.0, 0.0, 0.0), 5)) == 1                       # leaves [-2, 2], for float32 sets too
    assert code(plan.step, mu.make_config(*QUINTIC, 5, 1.0, True, 1e-7)) == 1
    assert code(plan.step, mu.make_config(float("nan"), 0.0, 0.0, 5)) == 1
    assert code(mu.StackPlan([g], None, [o]).step, config()) == 1                  # momentum without a buffer
    assert code(plan.set_weights, [g]) == 1                                        # over the gradient
    assert code(plan.set_weights, [o]) == 1
    plan.set_weights([w])
    assert code(plan.step_apply, config(), float("nan"), 0.0) == 1
    for bad in ([w, w], [w.bfloat16()], [w[:1]]):
        with pytest.raises(ValueError):
            plan.set_weights(bad)
    torch.cuda.synchronize()
    assert bool((o == 3.0).all()) and not b.any() and not w.any()
    empty = mu.StackPlan([g[:0]], [b[:0]], [o[:0]])
    empty.step(config())
    mu.StackPlan([], [], []).step(config())


def test_one_training_step_of_heads_and_embedding():
    """Lookup, its gradient as rows, one norm over them and the heads' gradients, the stacks' Muon step and the rows'
    Adam step on the clipped gradients: every part against float64 from the same factor."""
    gen = torch.Generator().manual_seed(12)
    n, vocab, cols = 700, 300, 96
    emb = torch.randn(vocab, cols, generator=gen).bfloat16().to(DEV)
    m, v = 1e-2 * torch.randn(vocab, cols, generator=gen).to(DEV), 1e-3 * torch.rand(vocab, cols, generator=gen).to(DEV)
    tok = torch.randint(-1, vocab // 2, (n,), generator=gen).to(DEV)
    dout = (0.1 * torch.randn(n, cols, generator=gen)).bfloat16().to(DEV)
    out = torch.empty_like(dout)
    qkv, proj = (0.1 * torch.randn(3 * cols, cols, generator=gen)).bfloat16().to(DEV), (0.1 * torch.randn(cols, cols, generator=gen)).bfloat16().to(DEV)
    heads = lambda a, b: [a.view(12, 24, cols), b.view(cols, 4, 24).transpose(0, 1)]  # noqa: E731
    bufs, weights = [torch.zeros_like(qkv), torch.zeros_like(proj)], [torch.randn_like(qkv), torch.randn_like(proj)]
    rows, values = torch.zeros(vocab, dtype=torch.int32, device=DEV), torch.zeros(vocab, cols, dtype=torch.bfloat16, device=DEV)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = mu.EmbeddingPlan(emb, n, m, v)
    stacks = mu.StackPlan(heads(qkv, proj), heads(*bufs), heads(qkv, proj))
    stacks.set_weights(heads(*weights))
    clip = mu.ClipPlan([qkv, proj, values], [None] * 3)
    clip.set_live_rows(2, count)
    stacks.set_grad_scale(clip.scale)
    table.set_grad_scale(clip.scale)
    e0, m0, v0, w0 = to_f64(emb), to_f64(m), to_f64(v), [to_f64(w) for w in weights]
    table.lookup(tok, out)
    table.gradient_rows(tok, dout, rows, values, count)
    clip.norm(1.0)
    stacks.step_apply(config(), f32(0.02), f32(0.01))
    table.adam_rows(rows, values, count, f32(1e-3), f32(0.9), f32(0.99), f32(1e-8), f32(0.1), 3)
    torch.cuda.synchronize()
    k = count.item()
    ids = rows[:k].cpu().numpy()
    assert np.array_equal(ids, np.unique(tok[tok >= 0].cpu().numpy()))
    norm, _ = oracle.gradient_norms([to_f64(qkv), to_f64(proj), to_f64(values[:k])])
    s = clip.scale.item()
    assert abs(s - oracle.clip_scale(norm, max_norm=1.0, eps=f32(1e-6))) <= s * 2.0 ** -23
    # the rows: float32 arithmetic from the stored sums, then one rounding
    gr = np.float32(to_f64(values[:k])) * np.float32(s)
    p2, m2, v2 = oracle.adam_update(e0[ids], gr.astype(np.float64), m0[ids], v0[ids], lr=f32(1e-3), beta1=f32(0.9), beta2=f32(0.99), eps=f32(1e-8),
                                    wd=f32(0.1), step=3, dtype="none")
    assert np.abs(to_f64(m)[ids] - m2).max() <= 4 * 2.0 ** -24 * np.abs(m2).max() and np.abs(to_f64(v)[ids] - v2).max() <= 4 * 2.0 ** -24 * np.abs(v2).max()
    # an update is at most a few times lr here; its float32 terms are off by some 2^-22 of it
    assert (np.abs(to_f64(emb)[ids] - p2) <= 2.0 ** -8 * np.abs(p2) + 2.0 ** -20).all()
    rest = np.setdiff1d(np.arange(vocab), ids)
    assert np.array_equal(to_f64(emb)[rest], e0[rest]) and np.array_equal(to_f64(m)[rest], m0[rest])
    for g, w, w1 in zip(heads(qkv, proj), heads(*[torch.from_numpy(x) for x in w0]), heads(*weights)):
        for t in range(g.shape[0]):
            x, _ = oracle_x((np.float32(to_f64(g[t])) * np.float32(s)).astype(np.float64), np.zeros(tuple(g.shape[1:])), QUINTIC, 5, MU, True, "bf16")
            want = w[t].numpy() * f32(1 - np.float32(f32(0.02)) * np.float32(f32(0.01))) - f32(0.02) * x
            off = np.maximum(np.abs(to_f64(w1[t]) - want) - 2.0 ** -8 * np.abs(want) - 2.0 ** -23 * (np.abs(w[t].numpy()) + np.abs(x)), 0.0)
            assert np.linalg.norm(off) <= TOL * f32(0.02) * np.linalg.norm(x)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_interleaved_stacks_in_one_plan(dtype):
    """q, k and v of [layers, 3, rows, cols] buffers, and adapter factors one behind another, as stacks of one plan: the
    bits of a plan each on copies, weights among them."""
    gen = torch.Generator().manual_seed(8)
    rand = lambda *s: torch.randn(*s, generator=gen).to(TDT[dtype]).to(DEV)  # noqa: E731
    layers, rows, cols, r, d = 5, 40, 96, 8, 72
    flat = [rand(layers * (r * d + d * r)) for _ in range(4)]
    fused = [rand(layers, 3, rows, cols) for _ in range(4)]
    views = []  # per buffer (grad, momentum, out, weight): its stacks
    for x, f in zip(fused, flat):
        both = f.view(layers, 2 * r * d)
        views.append([x[:, j] for j in range(3)] + [both[:, :r * d].view(layers, r, d), both[:, r * d:].view(layers, d, r)])
    alone = [[v.clone() for v in stacks] for stacks in views]
    plan = mu.StackPlan(*views[:3])
    plan.set_weights(views[3])
    plan.step(config())
    plan.step_apply(config(), 0.02, 0.1)
    for i in range(5):
        own = mu.StackPlan(*[[a[i]] for a in alone[:3]])
        own.set_weights([alone[3][i]])
        own.step(config())
        own.step_apply(config(), 0.02, 0.1)
        for a, v in zip(alone, views):
            assert torch.equal(a[i], v[i]), i
        own.destroy()
    first = views[3][0]
    for w in (first, fused[3].view(-1)[rows * cols - 1:].as_strided(first.shape, first.stride())):
        with pytest.raises(mu.MuonError) as exc:
            plan.set_weights([first, w, *views[3][2:]])
        assert exc.value.code == 1                         # the same weights twice, one element into the neighbour
    plan.destroy()


# What a bf16 set leaves in X before its rounding. One rounding of A to its two fp16 numbers is LOW (3.3e-3) of X's norm
# where X lies in directions of singular value near zero; in the same directions and to first order the first update of A
# adds lo lo left out of A^T Q (2^-22, two roundings of 2^-23), T's rounding (0.7 3.44 / 11.86 = 0.2 of one), lo lo left out
# of T^T Q (0.4), and all that follows under 0.4, being of an A whose largest eigenvalue is a half, grown by 11.86 less per
# step: 4 in all, and float32's part of the sums of A up to 1 more. RAW is all of them at their largest and aligned. They
# are independent, so a matrix in the middle of many has less than a third of it: 3.3e-3 again.
RAW, RAW_MEDIAN = 5 * 3.3e-3, 3.3e-3


def raw_x(g, momentum):
    """(X before the output's rounding, X in float64): W <- W0 - X from W0 = bf16(X) is off by bf16's rounding of the
    difference, 2^-17 of X. A zero buffer makes u a multiple of the gradient, so both forms have the same X."""
    x = g.double()
    x = x / (torch.linalg.matrix_norm(x)[:, None, None] + EPS)
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if tall else x
    for _ in range(5):
        a = x @ x.transpose(1, 2).contiguous()
        x = QUINTIC[0] * x + (QUINTIC[1] * a + QUINTIC[2] * (a @ a)) @ x
    x = x.transpose(1, 2).contiguous() if tall else x
    w0 = x.to(g.dtype)
    w = w0.clone()
    plan = mu.StackPlan([g], [torch.zeros_like(g)] if momentum else None, [torch.empty_like(g)])
    plan.set_weights([w])
    plan.step_apply(config(momentum=MU if momentum else 0.0, nesterov=bool(momentum)), 1.0, 0.0)
    torch.cuda.synchronize()
    plan.destroy()
    return w0.double() - w.double(), x


@pytest.mark.parametrize("momentum", [False, True])
@pytest.mark.parametrize("rows,cols", [(4, 300), (8, 100), (16, 765), (40, 100), (64, 768), (768, 64), (128, 300)])
def test_x_of_bf16_sets_before_rounding(rows, cols, momentum):
    gen = torch.Generator().manual_seed(rows)
    count, m = 48, min(rows, cols)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    left, right = torch.linalg.qr(rand(count, rows, m))[0], torch.linalg.qr(rand(count, cols, m))[0].transpose(1, 2).contiguous()
    for name, tol, middle, g in (
            ("flat", TOL, TOL, 0.05 * rand(count, rows, cols)),
            ("rank one", RAW, RAW_MEDIAN, rand(count, rows, 1) @ rand(count, 1, cols)),
            ("rank two", RAW, RAW_MEDIAN, rand(count, rows, 2) @ rand(count, 2, cols)),
            ("three decades", RAW, RAW_MEDIAN, left @ torch.diag(torch.logspace(0, -3, m)) @ right),
            ("five decades", RAW, RAW_MEDIAN, left @ torch.diag(torch.logspace(0, -5, m)) @ right)):
        got, want = raw_x(g.bfloat16().to(DEV), momentum)
        off = torch.linalg.matrix_norm(got - want) / torch.linalg.matrix_norm(want)
        say(f"{rows} x {cols} {name}: at most {off.max():.1e}, median {off.median():.1e}")
        assert off.max() <= tol and off.median() <= middle
