"""Gradient norm and clipping on lists whose work items are long enough for
the kernels' unrolled loops (hundreds of MB of random values; the lists of
test_gpu_clip.py are cut into items of 4 KB, which those loops never see).

Tolerances are those of test_gpu_clip.py: squares are exact in float64, and
sums of at most 2^32 non-negative terms added in trees and runs of under 2^15
terms are off by less than 2^-37, on either side; norm and scale are rounded
once to float32 (half a step: 2^-24). Clipped gradients are held bitwise to
the exact product g * scale (48 significant bits, exact in float64) rounded
to float32 and then to the gradient's type.
"""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

mu = pytest.importorskip("muon_newton_schulz_04_amd")
DEV = "cuda"
RTOL = 2.0 ** -24 + 2.0 ** -36
BF, FP = torch.bfloat16, torch.float32
STEP = 1 << 22

# (rows, cols, elements behind each row, elements before the first, type): 418 MB, so items of 52 KB.
# Runs at several alignments; rows much shorter than an item (whole rows share one, 16-byte vectors
# and elements behind them) and longer than one (a row is cut); the tensors that a clipping call reads
# past the caches and the 256 MB that it leaves there differ with the list's order.
TENSORS = [
    (1, 24_000_007, 0, 0, BF), (200_000, 129, 7, 1, BF), (1, 20_000_003, 0, 1, FP), (30_000, 333, 5, 2, FP),
    (1, 5, 0, 3, BF), (300, 40_001, 3, 0, FP), (50_000, 700, 1, 0, BF), (0, 8, 0, 0, FP), (1, 40_000_001, 0, 3, BF),
]


def f32(x):
    return float(np.float32(x))


def close(got, want):
    return abs(got - want) <= RTOL * abs(want)


def storage(rows, cols, pad, offset, dtype):
    buf = torch.full((offset + rows * (cols + pad) + 5,), 77.0, dtype=dtype, device=DEV)
    return buf, buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def make(specs, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    made = [storage(*s) for s in specs]
    for k, (_, v) in enumerate(made):
        v.normal_(0.0, 0.01 * (1 + k % 3), generator=gen)
    return [b for b, _ in made], [v for _, v in made]


def pieces(t):
    """Blocks of whole rows or of one row's columns, of about STEP elements."""
    if t.numel() == 0:
        return
    rows, cols = t.shape
    each = max(1, STEP // cols)
    for r in range(0, rows, each):
        for c in range(0, cols, STEP):
            yield slice(r, r + each), slice(c, c + STEP)


def norms_of(grads, mul):
    sums = [math.fsum(float(t[p].double().square().sum()) for p in pieces(t)) for t in grads]
    return mul * math.sqrt(math.fsum(sums)), [mul * math.sqrt(s) for s in sums]


def check(res, norms, want, each, max_norm, eps, mul):
    n, s = res.cpu().double().tolist()
    factor = oracle.clip_scale(want, max_norm=f32(max_norm), eps=f32(eps), mul=f32(mul))
    assert close(n, want) and close(s, factor), (n, want, s, factor)
    for a, b in zip(norms.cpu().double().tolist(), each):
        assert close(a, b), (a, b)
    return res[1].double()


def check_outs(before, outs, scale):
    for k, (g, o) in enumerate(zip(before, outs)):
        for p in pieces(g):
            want = (g[p].double() * scale).float().to(g.dtype)
            assert torch.equal(o[p], want), (k, p)


@pytest.mark.parametrize("order", ["as listed", "reversed"])
def test_norm_and_clip_of_long_items(order):
    specs = TENSORS[::-1] if order == "reversed" else TENSORS
    print(f"clip: 418 MB of random values, {order}", flush=True)
    bufs, grads = make(specs, 5)
    obufs, outs = make([(r, c, p + 2, (o + 1 + 2 * k) % 7, d) if r > 1 else (r, c, p, (o + 1 + 2 * k) % 7, d)
                        for k, (r, c, p, o, d) in enumerate(specs)], 6)
    before = [b.clone() for b in bufs]
    norms = torch.full((len(grads),), -1.0, device=DEV)
    plan = mu.ClipPlan(grads, outs)
    for max_norm, eps, mul in ((1.0, 1e-6, 1.0), (1e6, 0.0, 1.0 / 3)):
        want, each = norms_of(grads, f32(mul))
        check(plan.norm(max_norm, eps, mul, norms=norms), norms, want, each, max_norm, eps, mul)
        norms.fill_(-1.0)
        scale = check(plan.step(max_norm, eps, mul, norms=norms), norms, want, each, max_norm, eps, mul)
        check_outs(grads, outs, scale)
        assert all(torch.equal(a, b) for a, b in zip(bufs, before))   # gradients are only read
    plan.destroy()
    for b, o in zip(obufs, outs):                                     # nothing beside the outs is written
        o.fill_(77.0)
        assert bool((b == 77.0).all())
    del obufs, outs
    plan = mu.ClipPlan(grads)                                         # in place
    want, each = norms_of(grads, 1.0)
    scale = check(plan.step(2.5, norms=norms), norms, want, each, 2.5, 1e-6, 1.0)
    keep = [torch.as_strided(b, g.shape, g.stride(), g.storage_offset()) for b, g in zip(before, grads)]
    check_outs(keep, grads, scale)
    for b, g in zip(bufs, grads):
        g.fill_(77.0)
        assert bool((b == 77.0).all())
    plan.destroy()


@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_one_value_anywhere_in_long_items(value):
    """A single infinity or NaN reaches the norm from any place of a run and of strided rows, wherever a
    wave's loops take it up."""
    specs = [(1, 60_000_001, 0, 1, BF), (40_000, 1001, 3, 1, FP), (100_000, 257, 4, 0, BF)]
    _, grads = make(specs, 8)
    print(f"clip: one {value} in 331 MB", flush=True)
    plan = mu.ClipPlan(grads, [None] * 3)
    norms = torch.zeros(3, device=DEV)
    finite = plan.norm(1.0, norms=norms).cpu().tolist() + norms.cpu().tolist()
    assert all(map(math.isfinite, finite))
    rng = np.random.default_rng(9)
    for k, g in enumerate(grads):
        rows, cols = g.shape
        for _ in range(24):
            at = int(rng.integers(rows)), int(rng.integers(cols))
            old = g[at].clone()
            g[at] = value
            r = plan.norm(1.0, norms=norms).cpu()
            bad = [i for i, x in enumerate(norms.cpu().tolist()) if not math.isfinite(x)]
            assert bad == [k] and not math.isfinite(r[0].item()), (k, at)
            g[at] = old
    assert plan.norm(1.0, norms=norms).cpu().tolist() + norms.cpu().tolist() == finite
    plan.destroy()


def test_norm_only_of_a_long_list():
    """More partial sums than one launch adds up: the norm after the sums' own launch, with and without
    tensor norms, and again by the clipping call."""
    n = 40000
    flat = torch.randn(n * 3, generator=torch.Generator().manual_seed(4)).to(DEV)
    grads = [t[: 1 + i % 3] for i, t in enumerate(flat.view(n, 3).unbind())]
    host, lens = flat.view(n, 3).cpu().double().numpy(), 1 + np.arange(n) % 3
    each = np.sqrt(np.sum(np.where(np.arange(3)[None, :] < lens[:, None], host, 0.0) ** 2, axis=1))
    total = math.sqrt(math.fsum(each ** 2))
    norms = torch.zeros(n, device=DEV)
    plan = mu.ClipPlan(grads)
    print("clip: norm of 40000 tensors", flush=True)
    first = plan.norm(1.0, norms=norms).clone()
    assert close(first[0].item(), total) and close(first[1].item(), 1.0 / (total + f32(1e-6)))
    assert np.all(np.abs(norms.cpu().double().numpy() - each) <= RTOL * each)
    assert torch.equal(plan.norm(1.0), first)
    assert torch.equal(plan.step(1.0), first)
    plan.destroy()
