"""The embedding table's entry points (include/muon_embed.h) without a GPU:
sizes and arguments that are refused before any device call, workspace sizes,
and how the binding checks and lays out tensors."""
import ctypes
import itertools
import os
import subprocess

import pytest
import torch

import muon_newton_schulz_04_amd as mu

OK, INVALID, DTYPE, SHAPE, ALIGN = 0, 1, 2, 3, 4
B = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return mu.load_library()


def create(lib, dtype=mu.MUON_BF16, max_tokens=64, **kw):
    f = dict(vocab=100, cols=8, ld=8, table=B, exp_avg=2 * B, exp_avg_sq=3 * B, lr_mul=1.0, wd_mul=1.0)
    f.update(kw)
    t = mu.MuonEmbedTable(*f.values())
    h = ctypes.c_void_p(7)
    code = lib.muon_embed_plan_create(ctypes.byref(t), dtype, max_tokens, ctypes.byref(h))
    if code in (INVALID, DTYPE, SHAPE, ALIGN):
        assert h.value is None  # NULL on error
    return code


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(vocab=0)), (SHAPE, dict(vocab=(1 << 24) + 1)), (SHAPE, dict(cols=0)), (SHAPE, dict(cols=65537, ld=65537)),
    (SHAPE, dict(ld=7)), (SHAPE, dict(ld=(1 << 40) + 1)), (SHAPE, dict(max_tokens=-1)), (SHAPE, dict(max_tokens=(1 << 24) + 1)),
    (SHAPE, dict(max_tokens=1 << 24, cols=8193, ld=8193)),
    (DTYPE, dict(dtype=2)), (INVALID, dict(table=None)), (INVALID, dict(exp_avg=None)), (INVALID, dict(exp_avg_sq=None)),
    (INVALID, dict(lr_mul=float("nan"))), (INVALID, dict(wd_mul=float("inf"))),
    (ALIGN, dict(table=B + 1)), (ALIGN, dict(dtype=mu.MUON_F32, table=B + 2)), (ALIGN, dict(exp_avg=2 * B + 2)),
    (INVALID, dict(exp_avg=B + 100 * 8 * 2 - 4)),                    # moments inside the table
    (INVALID, dict(exp_avg=2 * B, exp_avg_sq=2 * B + 100 * 8 * 4 - 4)),
    (INVALID, dict(table=(1 << 64) - 16)),                           # past the end of the address space
])
def test_plan_refusals(lib, want, kw):
    assert create(lib, **kw) == want


def test_plan_accepts_what_only_a_device_can_refuse(lib):
    if torch.cuda.is_available():
        pytest.skip("checks the order of the tests where there is no device")
    for kw in ({}, dict(exp_avg=None, exp_avg_sq=None), dict(ld=11), dict(vocab=1, cols=1, ld=1), dict(max_tokens=0),
               dict(table=B + 2), dict(exp_avg=B + 100 * 8 * 2)):
        assert create(lib, **kw) == 6  # MUON_E_DEVICE: everything else was fine


def test_null_arguments(lib):
    n = ctypes.c_void_p(None)
    t = mu.MuonEmbedTokens(None, 0, 0, 0)
    a = mu.MuonEmbedActs(None, 8, 0, 0)
    assert lib.muon_embed_plan_create(None, 0, 1, ctypes.byref(ctypes.c_void_p())) == INVALID
    assert lib.muon_embed_plan_create(ctypes.byref(mu.MuonEmbedTable()), 0, 1, None) == INVALID
    assert lib.muon_embed_plan_lookup(n, ctypes.byref(t), 1.0, ctypes.byref(a), None) == INVALID
    assert lib.muon_embed_plan_gradient(n, ctypes.byref(t), ctypes.byref(a), 1.0, None, 8, 0, None, 0, None) == INVALID
    assert lib.muon_embed_plan_gradient_rows(n, ctypes.byref(t), ctypes.byref(a), 1.0, None, None, None, None, 0, None) == INVALID
    assert lib.muon_embed_plan_adam_rows(n, None, None, None, None, 0, None) == INVALID
    assert lib.muon_embed_plan_set_grad_scale(n, None) == INVALID
    assert lib.muon_embed_workspace_bytes(1, 1, 1, None) == INVALID
    assert lib.muon_clip_plan_set_live_rows(n, 0, None, 1) == INVALID
    lib.muon_embed_plan_destroy(n)


def test_workspace_grows_with_the_batch(lib):
    """A plan's workspace serves every smaller batch: sizes never fall as the batch grows."""
    for vocab, cols in ((1, 1), (50257, 768), (100, 65536), (1 << 24, 8)):
        last = 0
        for n in sorted({0, 1, 2, 3, 4, 5, 63, 64, 65, 1000, 4096, 5461, 5462, 16383, 16384, 16385, 65536, 100000}):
            size = mu.muon_embed_workspace_bytes(vocab, cols, n)
            assert size >= last and size > 0
            last = size
    # the records (16 bytes a token), the partial sums (two rows a chunk) and a byte for every table row
    n = mu.muon_embed_workspace_bytes(50257, 768, 32768)
    assert 32768 * 16 <= n <= 32768 * 16 + 2 * 1366 * 768 * 4 + 50257 + 8192
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, -1), ((1 << 24) + 1, 1, 1), (1, 65537, 1), (1, 1, (1 << 24) + 1)):
        with pytest.raises(mu.MuonError):
            mu.muon_embed_workspace_bytes(*bad)


def test_binding_refuses_host_tensors_and_wrong_types():
    with pytest.raises(ValueError):
        mu.EmbeddingPlan(torch.zeros(4, 4), 8)  # host memory


def host_plan(vocab, cols):
    """A plan of the binding without the library's: what the binding checks comes before any call."""
    plan = object.__new__(mu.EmbeddingPlan)
    plan.handle, plan.device, plan.dtype = ctypes.c_void_p(None), torch.device("cpu"), mu.MUON_F32
    plan.vocab, plan.cols, plan.max_tokens, plan.workspace_bytes = vocab, cols, 64, 64
    plan._keep = (torch.zeros(vocab, cols), None, None)
    return plan


def shared_rows(n, cols):
    """Views of n rows of cols elements whose rows share elements: broadcast ones, overlapping ones, and the gradient that
    autograd hands to what a sum over the rows was taken of."""
    leaf = torch.zeros(n, cols, requires_grad=True)
    views = [torch.ones(cols).expand(n, cols), torch.ones(1, cols).expand(n, cols),
             torch.autograd.grad((leaf + 0).sum(0), leaf, torch.ones(cols))[0]]
    if cols > 1:
        views.append(torch.ones(n + cols).as_strided((n, cols), (1, 1)))
        views.append(torch.ones(n * cols).as_strided((n, cols), (cols - 1, 1)))
    assert all(v.stride(0) < cols and v.shape == (n, cols) for v in views)
    return views


@pytest.mark.parametrize("cols", [1, 2, 8])
def test_rows_that_share_elements_are_refused(cols):
    plan, tok = host_plan(6, cols), torch.zeros(5, dtype=torch.int64)
    good = torch.zeros(5, cols)
    for x in shared_rows(5, cols):
        for call in (lambda: plan.lookup(tok, x), lambda: plan.gradient(tok, x, torch.zeros(6, cols)),
                     lambda: plan.gradient_rows(tok, x, torch.zeros(5, dtype=torch.int32), good.clone(), torch.zeros(1, dtype=torch.int32))):
            with pytest.raises(ValueError, match="share"):
                call()
    for x in shared_rows(6, cols):
        with pytest.raises(ValueError, match="share"):
            mu.EmbeddingPlan(x, 4)
        with pytest.raises(ValueError, match="share"):
            plan.gradient(tok, good, x)
    # tokens of two dimensions: a broadcast of all rows
    tok2, x = torch.zeros(2, 5, dtype=torch.int64), torch.ones(cols).expand(2, 5, cols)
    with pytest.raises(ValueError, match="share"):
        plan.lookup(tok2, x)
    with pytest.raises(ValueError):
        plan.lookup(tok2, torch.ones(5, cols).expand(2, 5, cols))
    # one row, or none, shares nothing
    for n in (0, 1):
        assert plan._acts(torch.ones(cols).expand(n, cols), torch.zeros(n, dtype=torch.int64)).ld == cols
    assert plan._acts(torch.zeros(5, cols + 3)[:, :cols], tok).ld == cols + 3


def test_lookup_grid_fits_a_launch(tmp_path):
    """A launch holds under 2^32 threads, 2^24 - 1 blocks of 256. Every size that a plan accepts: all tokens have a block,
    none is empty, and a block's vectors count within 32 bits."""
    csrc = os.path.join(os.path.dirname(mu.__file__), "csrc")
    src = tmp_path / "grid.cpp"
    src.write_text("""#include <cstdio>
#include "embed_grid.hpp"
int main() {
  long long cols, n;
  while (std::scanf("%lld %lld", &cols, &n) == 2) {
    const muon_embed::LookGrid g = muon_embed::lookup_grid(cols, n);
    std::printf("%lld %lld %lld\\n", (long long)g.vpr, (long long)g.per, (long long)g.blocks);
  }
}
""")
    exe = str(tmp_path / "grid")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", f"-I{csrc}", str(src), "-o", exe], check=True)
    slabs = lambda cols: (cols + 255) // 256  # noqa: E731
    sizes = [(c, n) for c, n in itertools.product(
        (1, 7, 8, 9, 768, 4095, 4096, 4097, 4104, 8191, 8192, 8193, 65535, 65536),
        (1, 2, 255, 256, 1 << 20, (1 << 21) - 1, 1 << 21, (1 << 23) + 1, (1 << 24) - 2, (1 << 24) - 1, 1 << 24))
        if (n + 63) // 64 * slabs(c) <= 1 << 23]
    assert (4097, 1 << 24) in sizes and (8192, 1 << 24) in sizes
    for c, n in sizes:
        mu.muon_embed_workspace_bytes(1, c, n)  # accepted
    out = subprocess.run([exe], input="\n".join(f"{c} {n}" for c, n in sizes), check=True, stdout=subprocess.PIPE, text=True).stdout
    for (c, n), line in zip(sizes, out.splitlines(), strict=True):
        vpr, per, blocks = map(int, line.split())
        assert vpr == -(-c // 8) and blocks * 256 < 1 << 32, (c, n)
        assert (blocks - 1) * per < n <= blocks * per and vpr * per < 1 << 31, (c, n)
