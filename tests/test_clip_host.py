"""Global gradient norm and clipping (include/muon_clip.h) without a GPU: the
oracle's functions against closed forms (and planted mistakes in them), the
list validation, workspace sizes, and how the binding lays tensors out."""
import ctypes
import math

import numpy as np
import pytest
import torch

import muon_newton_schulz_04_amd as mu
import oracle
from tests.test_oracle_mutations import load_mutant

B = 1 << 40
F32, BF16 = mu.MUON_F32, mu.MUON_BF16


# ------------------------------------------------------------------- oracle

def pin_norms(impl):
    n, each = impl.gradient_norms([np.array([3.0, 0.0]), np.array([[-4.0]]), np.zeros(0)])
    assert n == 5.0 and each == [3.0, 4.0, 0.0]
    n, each = impl.gradient_norms([np.array([3.0]), np.array([4.0])], 0.5)
    assert n == 2.5 and each == [1.5, 2.0]
    n, _ = impl.gradient_norms([np.full(4, 3.0e38), np.full(4, 1e-45)])     # squares leave float32's range
    assert n == 6.0e38


def pin_scale(impl):
    assert impl.clip_scale(5.0, max_norm=1.0, eps=0.0) == 0.2
    assert impl.clip_scale(3.0, max_norm=1.0, eps=1.0, mul=0.5) == 0.125
    assert impl.clip_scale(0.75, max_norm=1.0, eps=0.25, mul=0.5) == 0.5    # at the limit: not clipped
    assert impl.clip_scale(0.0, max_norm=0.0, eps=0.0) == 1.0
    assert impl.clip_scale(2.0, max_norm=0.0, eps=0.0) == 0.0
    assert impl.clip_scale(math.inf, max_norm=1.0, eps=0.0) == 0.0
    assert impl.clip_scale(math.inf, max_norm=math.inf, eps=0.0) == 1.0
    assert math.isnan(impl.clip_scale(math.nan, max_norm=1.0, eps=0.0))


def pin_product(impl):
    # 1.0078125 * 0.75 = 193.5 * 2^-8 lies half way between two bf16 values: to even
    assert impl.clip_gradient([1.0078125], 0.75)[0] == 194 * 2.0 ** -8
    assert impl.clip_gradient([3.0], np.float64(np.float32(1 / 3)), "fp32")[0] == 1.0
    assert impl.clip_gradient([-2.0], 0.25)[0] == -0.5
    x = impl.clip_gradient([1.0 + 2.0 ** -7], float(np.float32(0.1)))[0]
    assert x == oracle.bf16_round(x) and abs(x - 0.10078125) <= 0.10078125 * 2.0 ** -8


PINS = [pin_norms, pin_scale, pin_product]
MISTAKES = {
    "no_square": ("np.sum(np.square(np.asarray(g, dtype=np.float64)))", "np.sum(np.asarray(g, dtype=np.float64))"),
    "sum_of_norms": ("mul * float(np.sqrt(np.sum(sums)))", "mul * float(np.sum(np.sqrt(sums)))"),
    "norm_without_mul": ("return mul * float(np.sqrt(np.sum(sums)))", "return float(np.sqrt(np.sum(sums)))"),
    "tensor_norms_without_mul": ("[mul * float(np.sqrt(s)) for s in sums]", "[float(np.sqrt(s)) for s in sums]"),
    "float32_squares": ("np.square(np.asarray(g, dtype=np.float64))", "np.square(np.asarray(g, dtype=np.float32))"),
    "eps_dropped": ("(float(max_norm) / (float(norm) + float(eps)))", "(float(max_norm) / float(norm))"),
    "always_clipped": ("    if norm + eps <= max_norm:\n        return float(mul)\n", ""),
    "limit_excluded": ("if norm + eps <= max_norm:", "if norm + eps < max_norm:"),
    "mul_dropped_when_clipped": ("return float(mul) * (float(max_norm)", "return (float(max_norm)"),
    "mul_dropped_when_not": ("        return float(mul)\n", "        return 1.0\n"),
    "product_not_rounded": ("return bf16_round(x) if dtype == \"bf16\" else x", "return x"),
}


@pytest.mark.parametrize("pin", PINS, ids=lambda p: p.__name__)
def test_clip_oracle_pin(pin):
    pin(oracle)


@pytest.mark.parametrize("name", sorted(MISTAKES))
def test_clip_oracle_mistake_is_caught(name):
    mutant = load_mutant(name, *MISTAKES[name])
    failed = []
    for pin in PINS:
        try:
            pin(mutant)
        except Exception:  # an AssertionError, or a division by zero
            failed.append(pin.__name__)
    assert failed


# --------------------------------------------------------------- validation

def status(recs, n=None):
    arr = (mu.MuonClipTensor * max(1, len(recs)))()
    for i, r in enumerate(recs):
        arr[i] = mu.MuonClipTensor(*r)
    out = ctypes.c_size_t(0)
    lib = mu.load_library()
    code = lib.muon_clip_workspace_bytes(arr, len(recs) if n is None else n, ctypes.byref(out))
    plan = ctypes.c_void_p(1)
    made = lib.muon_clip_plan_create(arr, len(recs) if n is None else n, ctypes.byref(plan))
    if code != 0:                                   # refused before any device call, and no plan
        assert made == code and not plan.value
    elif plan.value:
        lib.muon_clip_plan_destroy(plan)
    return code, out.value


OK = (4, 8, 8, 8, B, B, BF16, 0)


@pytest.mark.parametrize("recs,want", [
    ([(4, 8, 8, 8, B, B, 7, 0)], 2),                                       # unknown dtype
    ([(4, 8, 8, 8, B, B, BF16, 1)], 1),                                    # reserved field
    ([(-1, 8, 8, 8, B, B, BF16, 0)], 3),                                   # negative rows
    ([(4, -8, 8, 8, B, B, BF16, 0)], 3),                                   # negative cols
    ([(4, 8, 7, 8, B, B + 4096, BF16, 0)], 3),                             # ld < cols
    ([(4, 8, 8, 7, B, B + 4096, BF16, 0)], 3),                             # out_ld < cols
    ([((1 << 40) + 1, 1, 1, 1, B, 0, BF16, 0)], 3),                        # too many rows
    ([(1 << 21, 1 << 20, 1 << 20, 1 << 20, B, 0, BF16, 0)], 3),            # too many elements
    ([(1 << 20, 1, 1 << 30, 1, B, 0, BF16, 0)], 3),                        # too long a stride
    ([(1, 1 << 40, 1 << 40, 0, B, 0, BF16, 0), (1, 1, 1, 0, B, 0, BF16, 0)], 3),  # too many together
    ([(4, 8, 8, 8, 0, B, BF16, 0)], 1),                                    # NULL grad
    ([(4, 8, 8, 8, B + 1, B + 4096, BF16, 0)], 4),                         # misaligned grad
    ([(4, 8, 8, 8, B + 2, B + 4096, F32, 0)], 4),
    ([(4, 8, 8, 8, B, B + 4097, BF16, 0)], 4),                             # misaligned out
    ([(4, 8, 8, 9, B, B, BF16, 0)], 1),                                    # in place with another stride
    ([(4, 8, 8, 8, B, B + 2, BF16, 0)], 1),                                # out overlaps its grad
    ([OK, OK], 1),                                                         # the same tensor twice, written
    ([OK, (1, 1, 1, 0, B + 62, 0, BF16, 0)], 1),                           # a read inside a written range
    ([(1, 8, 8, 8, (1 << 64) - 8, 0, F32, 0)], 3),                         # past the address space
])
def test_clip_list_validation(recs, want):
    assert status(recs)[0] == want


def test_clip_list_accepts():
    assert status([OK])[0] == 0
    assert status([(4, 8, 8, 99, B, 0, BF16, 0)] * 3)[0] == 0              # only read: repeats are fine
    assert status([(4, 8, 8, 16, B, B + 4096, BF16, 0), (1, 5, 5, 5, B + 64, B + 8192, F32, 0)])[0] == 0
    assert status([(0, 8, 0, 0, 0, 0, F32, 0), (8, 0, 0, 0, 0, 0, BF16, 0)])[0] == 0
    code, nb = status([], n=0)
    assert code == 0 and nb > 0
    assert status([OK], n=-1)[0] == 3
    lib = mu.load_library()
    assert lib.muon_clip_workspace_bytes(None, 1, ctypes.byref(ctypes.c_size_t(0))) == 1
    assert lib.muon_clip_workspace_bytes(None, 0, None) == 1
    assert lib.muon_clip_plan_create(None, 0, None) == 1
    for entry in (lib.muon_clip_plan_norm, lib.muon_clip_plan_step):
        assert entry(None, ctypes.byref(mu.MuonClipConfig(1.0, 0.0, 1.0)), B, None, B, 1 << 20, None) == 1
    assert lib.muon_plan_set_grad_scale(None, B) == 1
    assert lib.muon_adam_plan_set_grad_scale(None, B) == 1
    lib.muon_clip_plan_destroy(None)


def test_clip_workspace_grows_with_the_list_but_not_with_sizes():
    """A few sums per work item; items are bounded by the list length and a
    constant, whatever the sizes."""
    small = status([(1, 10, 10, 10, B, B, F32, 0)])[1]
    huge = status([(1, 1 << 39, 1 << 39, 0, B, 0, F32, 0)])[1]
    assert small <= huge <= 1 << 20
    many = [(1, 1, 1, 0, B, 0, F32, 0)] * 5000
    assert status(many)[1] >= 8 * 5000
    tall = status([(1 << 22, 3, 5, 0, B, 0, BF16, 0)])[1]                  # short rows share an item
    assert tall <= 1 << 18


# ------------------------------------------------------------------- layout

def layout(t):
    return mu._row_layout(t)[:3]


def test_row_layout():
    x = torch.zeros(6, 10)
    assert layout(x) == (1, 60, 60)
    assert layout(x.t()) == (1, 60, 60)                     # dense in any order
    assert layout(x[:, :7]) == (6, 7, 10)
    assert layout(x[:, :7].t()) == (6, 7, 10)
    assert layout(x[::2]) == (3, 10, 20)
    assert layout(x[:, 3]) == (6, 1, 10)
    assert layout(x[2]) == (1, 10, 10)
    assert layout(torch.zeros(())) == (1, 1, 1)
    assert layout(torch.zeros(2, 3, 4, 5).permute(2, 0, 3, 1)) == (1, 120, 120)
    assert layout(torch.zeros(2, 3, 4)[:, :, :2]) == (6, 2, 4)
    assert layout(torch.zeros(2, 1, 4)[:, :, :1]) == (2, 1, 4)
    assert layout(torch.zeros(4, 6, 8)[:, ::2, :3]) == (12, 3, 16)
    assert layout(torch.zeros(4, 6)[:, ::2]) == (12, 1, 2)
    for bad in (torch.zeros(3).expand(4, 3), torch.zeros(4, 5, 8)[:, ::2, :3],
                torch.zeros(9).as_strided((3, 3), (2, 1))):
        with pytest.raises(ValueError):
            layout(bad)


def test_binding_refuses_mismatched_lists():
    g = [torch.zeros(4, 6), torch.zeros(5, dtype=torch.bfloat16)]
    assert mu.muon_clip_workspace_bytes(g) > 0
    assert mu.muon_clip_workspace_bytes(g, [None, None]) > 0
    assert mu.muon_clip_workspace_bytes([torch.zeros(4, 6)[:, :5]], [torch.zeros(4, 5)]) > 0
    assert mu.muon_clip_workspace_bytes([torch.zeros(4, 5)], [torch.zeros(4, 6)[:, :5]]) > 0
    for grads, outs in [(g, g[:1]), (g, [g[0].bfloat16(), g[1]]), (g, [g[0].t(), g[1]]),
                        ([torch.zeros(4, 6)], [torch.zeros(6, 4).t()]),
                        ([torch.zeros(4, 6)[:, :5]], [torch.zeros(5, 6)[:, :4].t()])]:
        with pytest.raises(ValueError):
            mu.muon_clip_workspace_bytes(grads, outs)
    with pytest.raises(TypeError):
        mu.muon_clip_workspace_bytes([torch.zeros(3, dtype=torch.float64)])
    with pytest.raises(ValueError):
        mu.ClipPlan(g)                                     # not in device memory


def test_adam_plan_refuses_a_list_beyond_one_launch():
    """16 tensors of 2^31 elements need 2^24 blocks, one more than a launch holds: refused before any device call."""
    arr = (mu.MuonAdamTensor * 16)()
    for i in range(16):
        at = (1 << 44) + i * (1 << 40)
        arr[i] = mu.MuonAdamTensor(1 << 31, at, at + (1 << 36), at + (1 << 37), at + (1 << 38), 1.0, 0.0)
    plan = ctypes.c_void_p(1)
    lib = mu.load_library()
    assert lib.muon_adam_plan_create(arr, 16, BF16, ctypes.byref(plan)) == 3 and not plan.value
    items = ctypes.c_int64(0)
    assert lib.muon_adam_work_items(arr, 16, BF16, ctypes.byref(items)) == 0 and items.value == 16 << 17


# ------------------------------------------------------- column slices

def rect(base, ld, r0, rows, c0, cols, write, dtype=BF16):
    es = 4 if dtype == F32 else 2
    at = base + (r0 * ld + c0) * es
    return (rows, cols, ld, ld if write else 0, at, at if write else 0, dtype, 0)


def test_column_slices_of_one_matrix_are_accepted():
    """q, k and v of a fused gradient, clipped in place: their ranges run into each other, their columns do not."""
    for dtype in (BF16, F32):
        d, rows = 48, 64
        qkv = [rect(B, 3 * d, 0, rows, k * d, d, True, dtype) for k in range(3)]
        assert status(qkv)[0] == 0 and status(qkv[::-1])[0] == 0
        assert status(qkv + [rect(B + (1 << 20), 7, 0, 5, 0, 7, True)])[0] == 0
        assert status(qkv[:2] + [rect(B, 3 * d, 0, rows, 2 * d, d, False, dtype)])[0] == 0      # one of them only read
        assert status(qkv[1:] + [rect(B, 3 * d, 0, 5, 0, d, True, dtype), rect(B, 3 * d, 5, rows - 5, 0, d, True, dtype)])[0] == 0
        assert status(qkv[:2] + [rect(B, 3 * d, 9, 1, 2 * d, d, True, dtype)])[0] == 0          # one row of the last
        for bad in (rect(B, 3 * d, 0, rows, 2 * d - 1, d, True, dtype),                         # a column too far left
                    rect(B, 3 * d, 0, rows, 2 * d - 1, d, False, dtype),
                    rect(B, 3 * d, 1, rows, 2 * d + 1, d, True, dtype),                         # into the next row's first column
                    rect(B, 3 * d, 9, 1, 2 * d, d + 1, True, dtype),
                    rect(B, 3 * d + 1, 0, rows, 2 * d, d, True, dtype),                         # another stride
                    rect(B, 3 * d, 3, 2, 0, 3 * d, True, dtype),                                # whole rows
                    rect(B, 3 * d, 0, rows, d, d, True, dtype)):                                # the same slice twice
            assert status(qkv[:2] + [bad])[0] == 1 and status([bad] + qkv[:2])[0] == 1
    x = torch.zeros(20, 30)
    assert mu.muon_clip_workspace_bytes([x[:, :10], x[:, 10:20], x[:, 20:]]) > 0                # in place
    assert mu.muon_clip_workspace_bytes([x[:, :10]], [x[:, 20:]]) > 0
    with pytest.raises(mu.MuonError):
        mu.muon_clip_workspace_bytes([x[:, :11], x[:, 10:20]])


def cells(t):
    rows, cols, ld, _, at, _, dtype, _ = t
    es = 4 if dtype == F32 else 2
    return {at + (r * ld + c) * es + b for r in range(rows) for c in range(cols) for b in range(es)}


def meets(ts):
    made = [(cells(t), t[5] != 0) for t in ts]
    return any(a[0] & b[0] for i, a in enumerate(made) for b in made[:i] if a[1] or b[1])


def test_overlaps_against_every_byte():
    """Random lists in a small buffer: a list with a shared written byte is never accepted, and a matrix cut
    into columns (each possibly into rows, all shuffled) always is."""
    rng = np.random.default_rng(12)
    kept = refused = 0
    for _ in range(3000):
        ld = int(rng.integers(2, 9))
        ts = []
        for _ in range(int(rng.integers(2, 5))):
            cols, stride = int(rng.integers(1, ld + 1)), ld if rng.random() < 0.9 else ld + 1
            ts.append(rect(B, stride, int(rng.integers(0, 6)), int(rng.integers(1, 5)), int(rng.integers(0, ld)), cols,
                           rng.random() < 0.6, F32 if rng.random() < 0.1 else BF16))
        code = status(ts)[0]
        assert code in (0, 1)
        if meets(ts):
            refused += 1
            assert code == 1
        kept += code == 0
    assert kept > 300 and refused > 300
    for _ in range(500):
        ld, rows = int(rng.integers(3, 12)), int(rng.integers(1, 9))
        cuts = [0, *sorted(rng.choice(np.arange(1, ld), size=int(rng.integers(1, ld)), replace=False).tolist()), ld]
        ts = []
        for a, b in zip(cuts, cuts[1:]):
            at = 0 if rng.random() < 0.7 else int(rng.integers(0, rows))
            mid = int(rng.integers(at, rows + 1))
            ts += [rect(B, ld, r0, n, a, b - a, rng.random() < 0.7) for r0, n in ((at, mid - at), (mid, rows - mid)) if n]
        order = rng.permutation(len(ts))
        assert not meets(ts) and status([ts[i] for i in order])[0] == 0
