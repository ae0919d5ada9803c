"""Python binding of the MI355X Muon Newton-Schulz library.

Argument marshalling only: every step of the update runs in the HIP kernels
of ``lib/libmuon_mi355x.so`` (built by ``build.py``); torch supplies device
memory and streams. The names mirror the C ABI in ``include/muon.h``.
There is no CPU fallback: if the library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence

import numpy as np

__all__ = [
    "LIB_PATH", "MuonError", "MuonMatrix", "MuonConfig", "MuonBufferInfo",
    "KERNEL_NAMES", "load_library", "muon_abi_version", "muon_status_str",
    "muon_workspace_bytes", "muon_plan_create", "muon_plan_step", "muon_plan_destroy",
    "muon_step", "muon_orthogonalize", "muon_schedule_query", "muon_plan_set_timing",
    "muon_plan_kernel_times", "muon_plan_buffer_info", "MuonPlan", "make_config",
    "muon_plan_set_chained", "muon_plan_set_chain_timeout", "muon_plan_chain_state",
    "muon_plan_chain_times",
    "MuonWeight", "MuonApply", "muon_plan_set_weights", "muon_plan_step_apply",
    "muon_plan_step_noalloc", "MUON_SCRATCH_BYTES",
    "MuonAdamTensor", "MuonAdamConfig", "AdamPlan", "muon_adam_plan_create",
    "muon_adam_plan_step", "muon_adam_plan_destroy", "muon_adam_work_items",
    "muon_plan_set_grad_scale", "muon_adam_plan_set_grad_scale",
    "MuonClipTensor", "MuonClipConfig", "ClipPlan", "muon_clip_plan_create",
    "muon_clip_plan_norm", "muon_clip_plan_step", "muon_clip_plan_destroy",
    "muon_clip_workspace_bytes", "muon_clip_plan_set_live_rows",
    "MuonEmbedTable", "MuonEmbedTokens", "MuonEmbedActs", "EmbeddingPlan",
    "muon_embed_workspace_bytes", "muon_embed_plan_create", "muon_embed_plan_lookup",
    "muon_embed_plan_gradient", "muon_embed_plan_gradient_rows", "muon_embed_plan_adam_rows",
    "muon_embed_plan_set_grad_scale", "muon_embed_plan_destroy",
    "MuonStack", "MuonStackWeight", "StackPlan", "muon_stack_workspace_bytes",
    "muon_stack_plan_create", "muon_stack_plan_step", "muon_stack_plan_set_weights",
    "muon_stack_plan_step_apply", "muon_stack_plan_set_grad_scale", "muon_stack_plan_destroy",
    "MUON_F32", "MUON_BF16", "MUON_PRECISION_DEFAULT",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libmuon_mi355x.so")
MUON_F32, MUON_BF16 = 0, 1
KERNEL_NAMES = ["momentum", "normalize", "gram", "poly", "update"]
STATUS = ["MUON_OK", "MUON_E_INVALID", "MUON_E_DTYPE", "MUON_E_SHAPE", "MUON_E_ALIGN",
          "MUON_E_WORKSPACE", "MUON_E_DEVICE", "MUON_E_LAUNCH", "MUON_E_ALLOC", "MUON_E_SCRATCH"]
MUON_SCRATCH_BYTES = 128 << 20


class MuonError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS[code] if 0 <= code < len(STATUS) else code} "
                         f"({muon_status_str(code)})")


class MuonMatrix(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("grad", ctypes.c_void_p), ("momentum", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class MuonConfig(ctypes.Structure):
    _fields_ = [("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("steps", ctypes.c_int32), ("momentum", ctypes.c_float),
                ("nesterov", ctypes.c_int32), ("eps", ctypes.c_float),
                ("precision", ctypes.c_int32)]


class MuonWeight(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("lr_mul", ctypes.c_float), ("wd_mul", ctypes.c_float)]


class MuonApply(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("wd", ctypes.c_float)]


class MuonAdamTensor(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("lr_mul", ctypes.c_float), ("wd_mul", ctypes.c_float)]


class MuonAdamConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("wd", ctypes.c_float), ("step", ctypes.c_int32)]


class MuonClipTensor(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("out_ld", ctypes.c_int64), ("grad", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MuonClipConfig(ctypes.Structure):
    _fields_ = [("max_norm", ctypes.c_float), ("eps", ctypes.c_float), ("grad_mul", ctypes.c_float)]


class MuonEmbedTable(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("lr_mul", ctypes.c_float), ("wd_mul", ctypes.c_float)]


class MuonEmbedTokens(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("wide", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MuonEmbedActs(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MuonStack(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("stride", ctypes.c_int64), ("grad", ctypes.c_void_p),
                ("momentum", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class MuonStackWeight(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("ld", ctypes.c_int64), ("stride", ctypes.c_int64),
                ("lr_mul", ctypes.c_float), ("wd_mul", ctypes.c_float)]


class MuonBufferInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("m", "n", "mp", "np", "x_lo", "x_op0", "x_op1", "gram", "poly", "x0_scale")]


_lib = None


def load_library(path: str = LIB_PATH):
    """Loads the HIP library (once). Raises ImportError if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"Muon HIP library not built: {path} missing "
                          "(run python -m muon_newton_schulz_04_amd.build)")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "muon_abi_version": (i32, []),
        "muon_status_str": (ctypes.c_char_p, [i32]),
        "muon_workspace_bytes": (i32, [P(MuonMatrix), i32, i32, P(sz)]),
        "muon_plan_create": (i32, [P(MuonMatrix), i32, i32, P(vp)]),
        "muon_plan_step": (i32, [vp, P(MuonConfig), vp, sz, vp]),
        "muon_plan_step_noalloc": (i32, [vp, P(MuonConfig), vp]),
        "muon_plan_destroy": (None, [vp]),
        "muon_step": (i32, [P(MuonMatrix), i32, i32, P(MuonConfig), vp, sz, vp]),
        "muon_orthogonalize": (i32, [P(MuonMatrix), i32, i32, P(MuonConfig), vp, sz, vp]),
        "muon_schedule_query": (i32, [P(MuonMatrix), i32, i32, i32, P(i32), i64, P(i64)]),
        "muon_plan_set_timing": (i32, [vp, i32]),
        "muon_plan_kernel_times": (i32, [vp, P(ctypes.c_double), P(i64)]),
        "muon_plan_chain_times": (i32, [vp, P(ctypes.c_double), P(i64)]),
        "muon_plan_buffer_info": (i32, [vp, i32, P(MuonBufferInfo)]),
        "muon_plan_set_chained": (i32, [vp, i32]),
        "muon_plan_set_chain_timeout": (i32, [vp, i64]),
        "muon_plan_chain_state": (i32, [vp, P(i32), P(i32)]),
        "muon_plan_set_weights": (i32, [vp, P(MuonWeight), i32]),
        "muon_plan_step_apply": (i32, [vp, P(MuonConfig), P(MuonApply), vp, sz, vp]),
        "muon_adam_plan_create": (i32, [P(MuonAdamTensor), i32, i32, P(vp)]),
        "muon_adam_plan_step": (i32, [vp, P(MuonAdamConfig), vp]),
        "muon_adam_plan_destroy": (None, [vp]),
        "muon_plan_set_grad_scale": (i32, [vp, vp]),
        "muon_adam_plan_set_grad_scale": (i32, [vp, vp]),
        "muon_clip_workspace_bytes": (i32, [P(MuonClipTensor), i32, P(sz)]),
        "muon_clip_plan_create": (i32, [P(MuonClipTensor), i32, P(vp)]),
        "muon_clip_plan_norm": (i32, [vp, P(MuonClipConfig), vp, vp, vp, sz, vp]),
        "muon_clip_plan_step": (i32, [vp, P(MuonClipConfig), vp, vp, vp, sz, vp]),
        "muon_clip_plan_destroy": (None, [vp]),
        "muon_clip_plan_set_live_rows": (i32, [vp, i32, vp, i64]),
        "muon_embed_workspace_bytes": (i32, [i64, i64, i64, P(sz)]),
        "muon_embed_plan_create": (i32, [P(MuonEmbedTable), i32, i64, P(vp)]),
        "muon_embed_plan_lookup": (i32, [vp, P(MuonEmbedTokens), ctypes.c_float, P(MuonEmbedActs), vp]),
        "muon_embed_plan_gradient": (i32, [vp, P(MuonEmbedTokens), P(MuonEmbedActs), ctypes.c_float, vp, i64, i32,
                                           vp, sz, vp]),
        "muon_embed_plan_gradient_rows": (i32, [vp, P(MuonEmbedTokens), P(MuonEmbedActs), ctypes.c_float, vp, vp, vp,
                                                vp, sz, vp]),
        "muon_embed_plan_adam_rows": (i32, [vp, P(MuonAdamConfig), vp, vp, vp, i64, vp]),
        "muon_embed_plan_set_grad_scale": (i32, [vp, vp]),
        "muon_embed_plan_destroy": (None, [vp]),
        "muon_stack_workspace_bytes": (i32, [P(MuonStack), i32, i32, P(sz)]),
        "muon_stack_plan_create": (i32, [P(MuonStack), i32, i32, P(vp)]),
        "muon_stack_plan_step": (i32, [vp, P(MuonConfig), vp, sz, vp]),
        "muon_stack_plan_set_weights": (i32, [vp, P(MuonStackWeight), i32]),
        "muon_stack_plan_step_apply": (i32, [vp, P(MuonConfig), P(MuonApply), vp, sz, vp]),
        "muon_stack_plan_set_grad_scale": (i32, [vp, vp]),
        "muon_stack_plan_destroy": (None, [vp]),
        "muon_adam_work_items": (i32, [P(MuonAdamTensor), i32, i32, P(i64)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(code: int, where: str):
    if code != 0:
        raise MuonError(code, where)


def muon_abi_version() -> int:
    return load_library().muon_abi_version()


def muon_status_str(code: int) -> str:
    return load_library().muon_status_str(int(code)).decode()


# ------------------------------------------------------------ marshalling

def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    if t.dtype == torch.float32:
        return MUON_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _ld(t) -> int:
    if t.dim() != 2:
        raise ValueError("matrices must be 2-D")
    rows, cols = t.shape
    if rows and cols > 1 and t.stride(1) != 1:
        raise ValueError("matrices must be row-major with unit column stride")
    return t.stride(0) if rows > 1 else cols


def _row_stride(t) -> int:
    """_ld of a matrix whose rows must not share elements (as those of an expanded view do)."""
    ld = _ld(t)
    if ld < t.shape[1]:
        raise ValueError("rows must not share elements: give a contiguous copy of a broadcast or overlapping view")
    return ld


def _matrices(grads, momenta, outs):
    """muon_matrix array (and dtype code) from lists of torch tensors."""
    n = len(grads)
    if len(outs) != n or (momenta is not None and len(momenta) != n):
        raise ValueError("grads, momenta and outs must have the same length")
    arr = (MuonMatrix * max(n, 1))()
    dt = None
    for i in range(n):
        g, o = grads[i], outs[i]
        m = None if momenta is None else momenta[i]
        for t in (g, o) + (() if m is None else (m,)):
            d = _dtype_code(t)
            if dt is None:
                dt = d
            elif d != dt:
                raise TypeError("all tensors of a call must share one dtype")
            if t.shape != g.shape:
                raise ValueError("grad, momentum and out must have the same shape")
        ld = _ld(g)
        if _ld(o) != ld or (m is not None and _ld(m) != ld):
            raise ValueError("grad, momentum and out must share one row stride")
        arr[i] = MuonMatrix(g.shape[0], g.shape[1], ld, _ptr(g), _ptr(m), _ptr(o))
    return arr, n, (MUON_BF16 if dt is None else dt)


def _shape_matrices(shapes: Sequence, dtype: int):
    """muon_matrix array for shape-only host queries: distinct, aligned,
    never dereferenced placeholder addresses."""
    n = len(shapes)
    arr = (MuonMatrix * max(n, 1))()
    es = 4 if dtype == MUON_F32 else 2
    base = 1 << 44
    for i, (r, c) in enumerate(shapes):
        span = ((r * c * es) + 4095) // 4096 * 4096 + 4096
        arr[i] = MuonMatrix(r, c, c, base, base + span, base + 2 * span)
        base += 3 * span
    return arr, n


MUON_PRECISION_DEFAULT = 0


def make_config(a: float, b: float, c: float, steps: int, momentum: float = 0.0,
                nesterov: bool = False, eps: float = 1e-7,
                precision: int = MUON_PRECISION_DEFAULT) -> MuonConfig:
    return MuonConfig(a, b, c, int(steps), momentum, 1 if nesterov else 0, eps, int(precision))


def _current_stream(index: int) -> int:
    # the handle alone: building the Stream object around it takes about 2 us
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _stream_handle(stream) -> Optional[int]:
    import torch
    if stream is None:
        return _current_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _workspace(nbytes: int, device, workspace):
    import torch
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if workspace.data_ptr() % 256:
        raise ValueError("workspace must be 256-byte aligned")
    return workspace


def _scale_ptr(t, device) -> Optional[int]:
    import torch
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() != 1 or not t.is_cuda or device not in (None, t.device):
        raise ValueError("the gradient scale is one float32 element on the plan's device")
    return t.data_ptr()


# ---------------------------------------------------------------- entry points

def muon_workspace_bytes(mats, dtype: Optional[int] = None) -> int:
    """Workspace bytes for a list of gradient tensors, or of (rows, cols)
    shapes with ``dtype`` (MUON_BF16 / MUON_F32)."""
    lib = load_library()
    if len(mats) and isinstance(mats[0], (tuple, list)):
        arr, n = _shape_matrices(mats, dtype if dtype is not None else MUON_BF16)
        dt = dtype if dtype is not None else MUON_BF16
    else:
        arr, n, dt = _matrices(mats, None, mats)
    out = ctypes.c_size_t(0)
    _check(lib.muon_workspace_bytes(arr, n, dt, ctypes.byref(out)), "muon_workspace_bytes")
    return out.value


def muon_schedule_query(shapes: Sequence, dtype: int, kind: int) -> np.ndarray:
    """Host-only: the (items, 4) int32 schedule of kernel ``kind``."""
    lib = load_library()
    arr, n = _shape_matrices(shapes, dtype)
    cnt = ctypes.c_int64(0)
    _check(lib.muon_schedule_query(arr, n, dtype, kind, None, 0, ctypes.byref(cnt)),
           "muon_schedule_query")
    buf = np.zeros((max(cnt.value, 1), 4), dtype=np.int32)
    _check(lib.muon_schedule_query(arr, n, dtype, kind,
                                   buf.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                   cnt.value, ctypes.byref(cnt)), "muon_schedule_query")
    return buf[: cnt.value]


class MuonPlan:
    """A plan over fixed tensors (their pointers are baked into the plan)."""

    def __init__(self, grads, momenta, outs):
        lib = load_library()
        self._keep = (list(grads), None if momenta is None else list(momenta), list(outs))
        arr, n, dt = _matrices(grads, momenta, outs)
        self.dtype = dt
        self.n = n
        self.device = grads[0].device if n else None
        h = ctypes.c_void_p(None)
        _check(lib.muon_plan_create(arr, n, dt, ctypes.byref(h)), "muon_plan_create")
        self.handle = h
        ws = ctypes.c_size_t(0)
        _check(lib.muon_workspace_bytes(arr, n, dt, ctypes.byref(ws)), "muon_workspace_bytes")
        self.workspace_bytes = ws.value

    def step(self, cfg: MuonConfig, workspace=None, stream=None):
        ws = _workspace(self.workspace_bytes, self.device, workspace)
        _check(load_library().muon_plan_step(self.handle, ctypes.byref(cfg), ws.data_ptr(),
                                             ws.numel(), _stream_handle(stream)),
               "muon_plan_step")
        return ws

    def step_noalloc(self, cfg: MuonConfig, stream=None):
        """muon_plan_step_noalloc: the same step with the library's fixed
        device scratch array as workspace (no allocation)."""
        _check(load_library().muon_plan_step_noalloc(self.handle, ctypes.byref(cfg),
                                                     _stream_handle(stream)),
               "muon_plan_step_noalloc")

    def set_weights(self, weights, lr_mul=None, wd_mul=None):
        """Attaches one weight tensor per matrix (same shape and dtype as its
        grad, row-major); lr_mul / wd_mul: per-matrix multipliers (default 1)."""
        n = self.n
        if len(weights) != n:
            raise ValueError("one weight per matrix")
        lr_mul = [1.0] * n if lr_mul is None else list(lr_mul)
        wd_mul = [1.0] * n if wd_mul is None else list(wd_mul)
        arr = (MuonWeight * max(n, 1))()
        grads = self._keep[0]
        for i, w in enumerate(weights):
            if w is None:
                arr[i] = MuonWeight(None, 0, lr_mul[i], wd_mul[i])
                continue
            if w.shape != grads[i].shape or _dtype_code(w) != self.dtype:
                raise ValueError("weight must match its grad's shape and dtype")
            arr[i] = MuonWeight(_ptr(w), _ld(w), float(lr_mul[i]), float(wd_mul[i]))
        _check(load_library().muon_plan_set_weights(self.handle, arr, n), "muon_plan_set_weights")
        self._weights = list(weights)

    def step_apply(self, cfg: MuonConfig, lr: float, wd: float, workspace=None, stream=None):
        """One Muon update whose last step writes W <- W (1 - lr wd wd_mul) - lr lr_mul X
        into the attached weights (``out`` is not written)."""
        ws = _workspace(self.workspace_bytes, self.device, workspace)
        ap = MuonApply(float(lr), float(wd))
        _check(load_library().muon_plan_step_apply(self.handle, ctypes.byref(cfg), ctypes.byref(ap),
                                                   ws.data_ptr(), ws.numel(),
                                                   _stream_handle(stream)),
               "muon_plan_step_apply")
        return ws

    def set_grad_scale(self, scale):
        """Later steps use grad * scale, ``scale`` a one-element float32 tensor on the
        plan's device that is read when the step runs (e.g. ``ClipPlan.scale``) and may not
        change until it has ended; None detaches it."""
        p = _scale_ptr(scale, self.device)
        _check(load_library().muon_plan_set_grad_scale(self.handle, p), "muon_plan_set_grad_scale")
        self._grad_scale = scale

    def set_timing(self, mode):
        """0 / False: off; 1 / True: each kernel over the whole set in its own
        timed launch; 2: the step's own launches timed as they run."""
        _check(load_library().muon_plan_set_timing(self.handle, int(mode)), "muon_plan_set_timing")

    def chain_times(self):
        """(total ms, launches) of the chained launches timed with mode 2
        since the last read."""
        ms, n = ctypes.c_double(0.0), ctypes.c_int64(0)
        _check(load_library().muon_plan_chain_times(self.handle, ctypes.byref(ms), ctypes.byref(n)),
               "muon_plan_chain_times")
        return ms.value, n.value

    def kernel_times(self):
        """{kernel name: (total ms, launches)} since timing was enabled / last read."""
        ms = (ctypes.c_double * 5)()
        n = (ctypes.c_int64 * 5)()
        _check(load_library().muon_plan_kernel_times(self.handle, ms, n), "muon_plan_kernel_times")
        return {KERNEL_NAMES[k]: (ms[k], n[k]) for k in range(5)}

    def set_chained(self, on: bool):
        """Use the chained launch where the plan has one (default) or the separate launches."""
        _check(load_library().muon_plan_set_chained(self.handle, 1 if on else 0),
               "muon_plan_set_chained")

    def set_chain_timeout(self, microseconds: int):
        """Bound of one wait of the chained launch (default 2 s)."""
        _check(load_library().muon_plan_set_chain_timeout(self.handle, int(microseconds)),
               "muon_plan_set_chain_timeout")

    def chain_state(self):
        """(chained, error): whether steps use the chained launch, and the plan's error
        word since the last query (0: none; waits for the device, clears the word)."""
        c, e = ctypes.c_int32(0), ctypes.c_int32(0)
        _check(load_library().muon_plan_chain_state(self.handle, ctypes.byref(c), ctypes.byref(e)),
               "muon_plan_chain_state")
        return int(c.value), int(e.value)

    def buffer_info(self, idx: int) -> dict:
        info = MuonBufferInfo()
        _check(load_library().muon_plan_buffer_info(self.handle, idx, ctypes.byref(info)),
               "muon_plan_buffer_info")
        return {f: getattr(info, f) for f, _ in MuonBufferInfo._fields_}

    def destroy(self):
        if self.handle:
            load_library().muon_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def muon_plan_create(grads, momenta, outs) -> MuonPlan:
    return MuonPlan(grads, momenta, outs)


def muon_plan_step(plan: MuonPlan, cfg: MuonConfig, workspace=None, stream=None):
    return plan.step(cfg, workspace, stream)


def muon_plan_destroy(plan: MuonPlan):
    plan.destroy()


def muon_plan_set_weights(plan: MuonPlan, weights, lr_mul=None, wd_mul=None):
    plan.set_weights(weights, lr_mul, wd_mul)


def muon_plan_step_apply(plan: MuonPlan, cfg: MuonConfig, lr: float, wd: float, workspace=None,
                         stream=None):
    return plan.step_apply(cfg, lr, wd, workspace, stream)


def muon_plan_step_noalloc(plan: MuonPlan, cfg: MuonConfig, stream=None):
    return plan.step_noalloc(cfg, stream)


def muon_plan_set_grad_scale(plan: MuonPlan, scale):
    plan.set_grad_scale(scale)


def muon_plan_set_timing(plan: MuonPlan, mode):
    plan.set_timing(mode)


def muon_plan_chain_times(plan: MuonPlan):
    return plan.chain_times()


def muon_plan_kernel_times(plan: MuonPlan):
    return plan.kernel_times()


def muon_plan_set_chained(plan: MuonPlan, on: bool):
    plan.set_chained(on)


def muon_plan_set_chain_timeout(plan: MuonPlan, microseconds: int):
    plan.set_chain_timeout(microseconds)


def muon_plan_chain_state(plan: MuonPlan):
    return plan.chain_state()


def muon_plan_buffer_info(plan: MuonPlan, idx: int) -> dict:
    return plan.buffer_info(idx)


def muon_step(grads: List, momenta: Optional[List], outs: List, cfg: MuonConfig,
              workspace=None, stream=None):
    """One Muon update of every matrix (plan cached by the library)."""
    lib = load_library()
    arr, n, dt = _matrices(grads, momenta, outs)
    ws_bytes = ctypes.c_size_t(0)
    _check(lib.muon_workspace_bytes(arr, n, dt, ctypes.byref(ws_bytes)), "muon_workspace_bytes")
    ws = _workspace(ws_bytes.value, grads[0].device if n else "cuda", workspace)
    _check(lib.muon_step(arr, n, dt, ctypes.byref(cfg), ws.data_ptr(), ws.numel(),
                         _stream_handle(stream)), "muon_step")
    return ws


def muon_orthogonalize(grads: List, outs: List, cfg: MuonConfig, workspace=None, stream=None):
    """Normalise + Newton-Schulz only (no momentum state)."""
    lib = load_library()
    arr, n, dt = _matrices(grads, None, outs)
    ws_bytes = ctypes.c_size_t(0)
    _check(lib.muon_workspace_bytes(arr, n, dt, ctypes.byref(ws_bytes)), "muon_workspace_bytes")
    ws = _workspace(ws_bytes.value, grads[0].device if n else "cuda", workspace)
    _check(lib.muon_orthogonalize(arr, n, dt, ctypes.byref(cfg), ws.data_ptr(), ws.numel(),
                                  _stream_handle(stream)), "muon_orthogonalize")
    return ws


# ------------------------------------------------------------------ Adam branch

def _adam_tensors(params, grads, exp_avgs, exp_avg_sqs, lr_mul=None, wd_mul=None):
    """muon_adam_tensor array (and dtype code) from lists of torch tensors
    (each contiguous; moments float32)."""
    import torch
    n = len(params)
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == n):
        raise ValueError("params, grads and the two moment lists must have the same length")
    lr_mul = [1.0] * n if lr_mul is None else list(lr_mul)
    wd_mul = [1.0] * n if wd_mul is None else list(wd_mul)
    arr = (MuonAdamTensor * max(n, 1))()
    dt = None
    for i in range(n):
        p, g, m, v = params[i], grads[i], exp_avgs[i], exp_avg_sqs[i]
        for t in (p, g, m, v):
            if not t.is_contiguous():
                raise ValueError("Adam tensors must be contiguous")
            if t.numel() != p.numel():
                raise ValueError("param, grad and moments must have the same element count")
        if m.dtype != torch.float32 or v.dtype != torch.float32:
            raise TypeError("Adam moments are float32")
        d = _dtype_code(p)
        if _dtype_code(g) != d:
            raise TypeError("param and grad must share one dtype")
        if dt is None:
            dt = d
        elif d != dt:
            raise TypeError("all parameters of a call must share one dtype")
        arr[i] = MuonAdamTensor(p.numel(), _ptr(p), _ptr(g), _ptr(m), _ptr(v),
                                float(lr_mul[i]), float(wd_mul[i]))
    return arr, n, (MUON_BF16 if dt is None else dt)


def muon_adam_work_items(params, grads, exp_avgs, exp_avg_sqs) -> int:
    arr, n, dt = _adam_tensors(params, grads, exp_avgs, exp_avg_sqs)
    out = ctypes.c_int64(0)
    _check(load_library().muon_adam_work_items(arr, n, dt, ctypes.byref(out)), "muon_adam_work_items")
    return out.value


class AdamPlan:
    """Adam over a fixed list of tensors (pointers baked into the plan)."""

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, lr_mul=None, wd_mul=None):
        lib = load_library()
        self._keep = (list(params), list(grads), list(exp_avgs), list(exp_avg_sqs))
        arr, n, dt = _adam_tensors(params, grads, exp_avgs, exp_avg_sqs, lr_mul, wd_mul)
        self.dtype = dt
        h = ctypes.c_void_p(None)
        _check(lib.muon_adam_plan_create(arr, n, dt, ctypes.byref(h)), "muon_adam_plan_create")
        self.handle = h

    def set_grad_scale(self, scale):
        """Later steps use grad * scale (see ``MuonPlan.set_grad_scale``)."""
        p = _scale_ptr(scale, self._keep[0][0].device if self._keep[0] else None)
        _check(load_library().muon_adam_plan_set_grad_scale(self.handle, p),
               "muon_adam_plan_set_grad_scale")
        self._grad_scale = scale

    def step(self, lr: float, beta1: float, beta2: float, eps: float, wd: float, step: int,
             stream=None):
        cfg = MuonAdamConfig(float(lr), float(beta1), float(beta2), float(eps), float(wd), int(step))
        _check(load_library().muon_adam_plan_step(self.handle, ctypes.byref(cfg),
                                                  _stream_handle(stream)), "muon_adam_plan_step")

    def destroy(self):
        if self.handle:
            load_library().muon_adam_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def muon_adam_plan_create(params, grads, exp_avgs, exp_avg_sqs, lr_mul=None, wd_mul=None):
    return AdamPlan(params, grads, exp_avgs, exp_avg_sqs, lr_mul, wd_mul)


def muon_adam_plan_step(plan: AdamPlan, lr, beta1, beta2, eps, wd, step, stream=None):
    plan.step(lr, beta1, beta2, eps, wd, step, stream)


def muon_adam_plan_destroy(plan: AdamPlan):
    plan.destroy()


def muon_adam_plan_set_grad_scale(plan: AdamPlan, scale):
    plan.set_grad_scale(scale)


# ------------------------------------------- global gradient norm and clipping

def _row_layout(t):
    """(rows, cols, ld, order of the dimensions) of a tensor whose elements lie in
    rows of consecutive elements at one stride: any dense tensor (also a permuted
    one) is one row, a 2-D view with a unit stride has its own rows."""
    dims = sorted((d for d in range(t.dim()) if t.shape[d] != 1), key=lambda d: t.stride(d))
    cols, ld, rows = 1, None, 1
    for d in dims:
        n, st = t.shape[d], t.stride(d)
        if ld is None and st == cols:
            cols *= n
        elif ld is None and st > cols:
            ld, rows = st, n
        elif ld is not None and st == ld * rows:
            rows *= n
        else:
            raise ValueError("a gradient must be rows of consecutive elements at one row stride")
    return rows, cols, cols if ld is None else ld, dims


def _clip_tensors(grads, outs):
    """muon_clip_tensor array from lists of torch tensors (``outs`` None: in place;
    an entry None: the norm only)."""
    n = len(grads)
    outs = list(grads) if outs is None else list(outs)
    if len(outs) != n:
        raise ValueError("grads and outs must have the same length")
    arr = (MuonClipTensor * max(n, 1))()
    device = grads[0].device if n else None
    for i, (g, o) in enumerate(zip(grads, outs)):
        dt = _dtype_code(g)
        if g.device != device or (o is not None and o is not g and o.device != device):
            raise ValueError("all tensors of a list must be on one device")
        if o is not None and o is not g and (o.dtype != g.dtype or o.shape != g.shape):
            raise ValueError("an out must match its grad's shape and dtype")
        numel = g.numel()
        if numel == 0:
            arr[i] = MuonClipTensor(0, 0, 0, 0, None, None, dt, 0)
            continue
        if g.is_contiguous() and (o is None or o is g or o.is_contiguous()):
            arr[i] = MuonClipTensor(1, numel, numel, numel, g.data_ptr(), _ptr(o), dt, 0)
            continue
        rows, cols, ld, dims = _row_layout(g)
        old = ld
        if o is not None:
            # the two are walked side by side: rows of the same length, the dimensions in the same order
            r2, c2, old, dims2 = _row_layout(o)
            if dims2 != dims:
                raise ValueError("an out must order its dimensions as its grad does")
            if (r2, c2) != (rows, cols):
                if c2 == rows * cols:       # out is dense, grad has rows
                    old = cols
                elif cols == r2 * c2:       # grad is dense, out has rows
                    rows, cols, ld = r2, c2, c2
                else:
                    raise ValueError("grad and out must split into the same rows")
        arr[i] = MuonClipTensor(rows, cols, ld, old, _ptr(g), _ptr(o), dt, 0)
    return arr, n


def muon_clip_workspace_bytes(grads, outs=None) -> int:
    arr, n = _clip_tensors(grads, outs)
    out = ctypes.c_size_t(0)
    _check(load_library().muon_clip_workspace_bytes(arr, n, ctypes.byref(out)),
           "muon_clip_workspace_bytes")
    return out.value


class ClipPlan:
    """Global norm of a fixed list of gradients (bf16 and float32 may be mixed) and
    clipping by it. ``outs`` None clips in place; a list of tensors receives the
    clipped gradients. With a None among them the plan computes norms only and
    refuses ``step``; ``[None] * n`` also takes lists with a gradient twice or with
    overlapping views, which cannot be clipped in place (column slices of one
    matrix can, if their columns are disjoint).

    ``result`` holds {norm, scale} of the last call on the device, ``scale`` is a view of
    its second element (what ``set_grad_scale`` of the optimizer plans takes; 1 before the
    first call). Calls that
    overlap in time, graphs replayed at once among them, need a ``workspace``, a ``result``
    and ``norms`` each (a workspace is allocated per call unless one is given)."""

    def __init__(self, grads, outs=None):
        import torch
        lib = load_library()
        grads = list(grads)
        self._keep = (grads, None if outs is None else list(outs))
        arr, n = _clip_tensors(grads, outs)
        self.n = n
        self.device = grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
        if self.device.type != "cuda":
            raise ValueError("gradients must be in device memory")
        self.handle = ctypes.c_void_p(None)
        ws = ctypes.c_size_t(0)
        _check(lib.muon_clip_workspace_bytes(arr, n, ctypes.byref(ws)), "muon_clip_workspace_bytes")
        self.workspace_bytes = ws.value
        h = ctypes.c_void_p(None)
        with torch.cuda.device(self.device):
            _check(lib.muon_clip_plan_create(arr, n, ctypes.byref(h)), "muon_clip_plan_create")
        self.handle = h
        # a factor of one until the first call; complete before any stream's call can write it
        self.result = torch.tensor([0.0, 1.0], dtype=torch.float32, device=self.device)
        torch.cuda.current_stream(self.device).synchronize()
        self.scale = self.result[1:2]

    def _run(self, entry, max_norm, eps, grad_mul, norms, result, workspace, stream):
        import torch
        result = self.result if result is None else result
        for t, k in ((result, 2), (norms, self.n)):
            if t is not None and (t.dtype != torch.float32 or t.numel() != k or not t.is_contiguous()
                                  or t.device != self.device):
                raise ValueError(f"result and norms are contiguous float32 tensors of 2 and {self.n} "
                                 f"elements on {self.device}")
        if workspace is None and stream is None:
            workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
        elif workspace is None:
            # allocated and, once dropped, reused in the order of the stream that uses it
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), self.device)
            with torch.cuda.stream(s):
                workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
        elif workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {self.device}")
        cfg = MuonClipConfig(float(max_norm), float(eps), float(grad_mul))
        index = self.device.index
        handle = _current_stream(index) if stream is None else _stream_handle(stream)
        args = (self.handle, ctypes.byref(cfg), result.data_ptr(), _ptr(norms), workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), handle)
        fn = getattr(load_library(), entry)
        if torch.cuda.current_device() == index:
            _check(fn(*args), entry)
        else:
            with torch.cuda.device(index):
                _check(fn(*args), entry)
        return result

    def norm(self, max_norm: float = float("inf"), eps: float = 1e-6, grad_mul: float = 1.0, norms=None,
             result=None, workspace=None, stream=None):
        """Writes {norm, scale} into ``result`` (the plan's own unless given) and each
        tensor's norm into ``norms`` (float32, one per tensor); gradients are only read.
        Returns ``result``; nothing waits for the device."""
        return self._run("muon_clip_plan_norm", max_norm, eps, grad_mul, norms, result, workspace, stream)

    def step(self, max_norm: float, eps: float = 1e-6, grad_mul: float = 1.0, norms=None, result=None,
             workspace=None, stream=None):
        """``norm``, then every gradient times the scale into its out (in place without outs).
        An optimizer plan that takes these gradients must not have the scale attached too."""
        return self._run("muon_clip_plan_step", max_norm, eps, grad_mul, norms, result, workspace, stream)

    def set_live_rows(self, index: int, count, cols: Optional[int] = None):
        """Tensor ``index`` holds rows of ``cols`` elements (its last dimension unless given), of
        which later calls take the first ``count``, a one-element int32 tensor on the plan's device
        that is read when they run; the rows behind it are neither read nor written. The tensor must
        be contiguous. None: all rows."""
        import torch
        g = self._keep[0][index]
        if count is not None and (count.dtype != torch.int32 or count.numel() != 1 or count.device != self.device):
            raise ValueError("the number of live rows is one int32 element on the plan's device")
        if count is not None and not g.is_contiguous():
            raise MuonError(3, "muon_clip_plan_set_live_rows")  # (a permuted dense tensor is one row to the library)
        cols = (g.shape[-1] if g.dim() else 1) if cols is None else int(cols)
        index = index % self.n
        with torch.cuda.device(self.device):
            _check(load_library().muon_clip_plan_set_live_rows(self.handle, index, _ptr(count), cols),
                   "muon_clip_plan_set_live_rows")
        self._live = {**getattr(self, "_live", {}), index: count}

    def destroy(self):
        if self.handle:
            load_library().muon_clip_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def muon_clip_plan_create(grads, outs=None) -> ClipPlan:
    return ClipPlan(grads, outs)


def muon_clip_plan_norm(plan: ClipPlan, max_norm=float("inf"), eps=1e-6, grad_mul=1.0, norms=None, result=None,
                        workspace=None, stream=None):
    return plan.norm(max_norm, eps, grad_mul, norms, result, workspace, stream)


def muon_clip_plan_step(plan: ClipPlan, max_norm, eps=1e-6, grad_mul=1.0, norms=None, result=None, workspace=None,
                        stream=None):
    return plan.step(max_norm, eps, grad_mul, norms, result, workspace, stream)


def muon_clip_plan_destroy(plan: ClipPlan):
    plan.destroy()


def muon_clip_plan_set_live_rows(plan: ClipPlan, index: int, count, cols: Optional[int] = None):
    plan.set_live_rows(index, count, cols)


# ------------------------------------------------------------ embedding table

def muon_embed_workspace_bytes(vocab: int, cols: int, max_tokens: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().muon_embed_workspace_bytes(vocab, cols, max_tokens, ctypes.byref(out)),
           "muon_embed_workspace_bytes")
    return out.value


class EmbeddingPlan:
    """One embedding table (vocab x cols, bf16 or float32, rows at any stride) and its
    float32 moments, for batches of at most ``max_tokens`` tokens.

    Tokens are int32 or int64 tensors of any contiguous shape; one outside [0, vocab) looks
    up zeros and carries no gradient. Activations (``out``, ``dout``) have the tokens' shape
    and ``cols`` behind it, in bf16 or float32 whatever the table's type, and rows at one
    stride that share no elements (a broadcast ``dout`` is refused: pass a contiguous copy).
    A gradient needs a ``workspace``, allocated per call unless one is given; calls that
    overlap in time need one each. Nothing waits for the device."""

    def __init__(self, table, max_tokens: int, exp_avg=None, exp_avg_sq=None, lr_mul: float = 1.0,
                 wd_mul: float = 1.0):
        import torch
        lib = load_library()
        self.handle = ctypes.c_void_p(None)
        ld = _row_stride(table)
        if not table.is_cuda:
            raise ValueError("the table must be in device memory")
        self.dtype, self.device = _dtype_code(table), table.device
        for t in (exp_avg, exp_avg_sq):
            if t is None:
                continue
            if t.dtype != torch.float32:
                raise TypeError("Adam moments are float32")
            if t.shape != table.shape or not t.is_contiguous() or t.device != self.device:
                raise ValueError("moments must be contiguous, of the table's shape and on its device")
        self.vocab, self.cols = table.shape
        self.max_tokens = int(max_tokens)
        self._keep = (table, exp_avg, exp_avg_sq)
        self.workspace_bytes = muon_embed_workspace_bytes(self.vocab, self.cols, self.max_tokens)
        t = MuonEmbedTable(self.vocab, self.cols, ld, _ptr(table), _ptr(exp_avg), _ptr(exp_avg_sq),
                           float(lr_mul), float(wd_mul))
        h = ctypes.c_void_p(None)
        with torch.cuda.device(self.device):
            _check(lib.muon_embed_plan_create(ctypes.byref(t), self.dtype, self.max_tokens, ctypes.byref(h)),
                   "muon_embed_plan_create")
        self.handle = h

    def _tokens(self, tokens):
        import torch
        if tokens.dtype not in (torch.int32, torch.int64):
            raise TypeError("tokens are int32 or int64")
        if tokens.device != self.device or not tokens.is_contiguous():
            raise ValueError(f"tokens must be contiguous and on {self.device}")
        return MuonEmbedTokens(tokens.data_ptr(), tokens.numel(), 1 if tokens.dtype == torch.int64 else 0, 0)

    def _acts(self, x, tokens):
        dt = _dtype_code(x)
        if x.device != self.device or x.shape != (*tokens.shape, self.cols):
            raise ValueError(f"activations have the tokens' shape and {self.cols} columns, on {self.device}")
        if x.is_contiguous():
            ld = self.cols
        else:
            y = x.flatten(0, -2) if x.dim() > 2 else x
            if y.dim() != 2 or y.data_ptr() != x.data_ptr():
                raise ValueError("activations must be rows of consecutive elements at one row stride")
            ld = _row_stride(y)
        return MuonEmbedActs(x.data_ptr(), ld, dt, 0)

    def _rows(self, rows, values, count, need):
        import torch
        for t, dt in ((rows, torch.int32), (count, torch.int32)):
            if t.dtype != dt or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"rows and count are contiguous int32 tensors on {self.device}")
        if _dtype_code(values) != self.dtype or not values.is_contiguous() or values.device != self.device:
            raise ValueError(f"values must be contiguous, of the table's type and on {self.device}")
        if values.dim() != 2 or values.shape[1] != self.cols or rows.shape != values.shape[:1] or count.numel() != 1:
            raise ValueError("rows, values and count have shapes (r,), (r, cols) and one element")
        if rows.numel() < need:
            raise ValueError(f"rows and values need room for {need} rows")

    def _call(self, entry, *args, stream=None):
        import torch
        index = self.device.index
        handle = _current_stream(index) if stream is None else _stream_handle(stream)
        fn = getattr(load_library(), entry)
        if torch.cuda.current_device() == index:
            _check(fn(self.handle, *args, handle), entry)
        else:
            with torch.cuda.device(index):
                _check(fn(self.handle, *args, handle), entry)

    def _ws(self, workspace, stream):
        import torch
        if workspace is None:
            if stream is None:
                return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
            # allocated and, once dropped, reused in the order of the stream that uses it
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), self.device)
            with torch.cuda.stream(s):
                return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
        if workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {self.device}")
        return workspace

    def lookup(self, tokens, out, scale: float = 1.0, stream=None):
        """out[i] = scale * table[tokens[i]]; returns ``out``."""
        t, o = self._tokens(tokens), self._acts(out, tokens)
        self._call("muon_embed_plan_lookup", ctypes.byref(t), float(scale), ctypes.byref(o), stream=stream)
        return out

    def gradient(self, tokens, dout, grad, scale: float = 1.0, accumulate: bool = False, workspace=None, stream=None):
        """The lookup's gradient into ``grad`` (the table's shape and type): every row is written,
        or with ``accumulate`` the rows that have tokens are added to. Returns ``grad``."""
        t, d = self._tokens(tokens), self._acts(dout, tokens)
        if _dtype_code(grad) != self.dtype or grad.shape != self._keep[0].shape or grad.device != self.device:
            raise ValueError("grad must match the table's shape, type and device")
        ld = _row_stride(grad)
        ws = self._ws(workspace, stream)
        self._call("muon_embed_plan_gradient", ctypes.byref(t), ctypes.byref(d), float(scale), grad.data_ptr(),
                   ld, 1 if accumulate else 0, ws.data_ptr(), ws.numel() * ws.element_size(), stream=stream)
        return grad

    def gradient_rows(self, tokens, dout, rows, values, count, scale: float = 1.0, workspace=None, stream=None):
        """The gradient as rows: the distinct tokens ascending into ``rows`` (int32), their sums into
        ``values`` (the table's type) and their number into ``count`` (one int32). ``rows`` and
        ``values`` have room for min(number of tokens, vocab) rows; those behind ``count`` stay as they are."""
        t, d = self._tokens(tokens), self._acts(dout, tokens)
        self._rows(rows, values, count, min(tokens.numel(), self.vocab))
        ws = self._ws(workspace, stream)
        self._call("muon_embed_plan_gradient_rows", ctypes.byref(t), ctypes.byref(d), float(scale), rows.data_ptr(),
                   values.data_ptr(), count.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), stream=stream)
        return rows, values, count

    def set_grad_scale(self, scale):
        """Later ``adam_rows`` use values * scale (see ``MuonPlan.set_grad_scale``)."""
        p = _scale_ptr(scale, self.device)
        _check(load_library().muon_embed_plan_set_grad_scale(self.handle, p), "muon_embed_plan_set_grad_scale")
        self._grad_scale = scale

    def adam_rows(self, rows, values, count, lr: float, beta1: float, beta2: float, eps: float, wd: float, step: int,
                  stream=None):
        """The Adam step (``AdamPlan.step``) of the table's rows ``rows[:count]`` with gradients
        ``values[:count]``; the other rows and their moments stay as they are."""
        self._rows(rows, values, count, 0)
        cfg = MuonAdamConfig(float(lr), float(beta1), float(beta2), float(eps), float(wd), int(step))
        self._call("muon_embed_plan_adam_rows", ctypes.byref(cfg), rows.data_ptr(), values.data_ptr(),
                   count.data_ptr(), min(rows.numel(), self.vocab), stream=stream)

    def destroy(self):
        if self.handle:
            load_library().muon_embed_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def muon_embed_plan_create(table, max_tokens, exp_avg=None, exp_avg_sq=None, lr_mul=1.0, wd_mul=1.0) -> EmbeddingPlan:
    return EmbeddingPlan(table, max_tokens, exp_avg, exp_avg_sq, lr_mul, wd_mul)


def muon_embed_plan_lookup(plan: EmbeddingPlan, tokens, out, scale=1.0, stream=None):
    return plan.lookup(tokens, out, scale, stream)


def muon_embed_plan_gradient(plan: EmbeddingPlan, tokens, dout, grad, scale=1.0, accumulate=False, workspace=None,
                             stream=None):
    return plan.gradient(tokens, dout, grad, scale, accumulate, workspace, stream)


def muon_embed_plan_gradient_rows(plan: EmbeddingPlan, tokens, dout, rows, values, count, scale=1.0, workspace=None,
                                  stream=None):
    return plan.gradient_rows(tokens, dout, rows, values, count, scale, workspace, stream)


def muon_embed_plan_adam_rows(plan: EmbeddingPlan, rows, values, count, lr, beta1, beta2, eps, wd, step, stream=None):
    plan.adam_rows(rows, values, count, lr, beta1, beta2, eps, wd, step, stream)


def muon_embed_plan_set_grad_scale(plan: EmbeddingPlan, scale):
    plan.set_grad_scale(scale)


def muon_embed_plan_destroy(plan: EmbeddingPlan):
    plan.destroy()


# ------------------------------------------------ stacks of short matrices

def _stack_layout(t):
    """(count, rows, cols, ld, stride) of a 3-D view with a unit column stride (2-D: one matrix)."""
    if t.dim() == 2:
        t = t.unsqueeze(0)
    if t.dim() != 3:
        raise ValueError("a stack is a 3-D tensor (count, rows, cols), or one matrix")
    count, rows, cols = t.shape
    if t.numel() and cols > 1 and t.stride(2) != 1:
        raise ValueError("stacks must be row-major with unit column stride")
    return count, rows, cols, t.stride(1) if rows > 1 else cols, t.stride(0) if count > 1 else 0


def _stacks(grads, momenta, outs):
    """muon_stack array (and dtype code) from lists of torch tensors."""
    n = len(grads)
    if len(outs) != n or (momenta is not None and len(momenta) != n):
        raise ValueError("grads, momenta and outs must have the same length")
    arr = (MuonStack * max(n, 1))()
    dt = None
    for i in range(n):
        g, m, o = grads[i], None if momenta is None else momenta[i], outs[i]
        layout = _stack_layout(g)
        for t in (g, o) + (() if m is None else (m,)):
            d = _dtype_code(t)
            dt = d if dt is None else dt
            if d != dt:
                raise TypeError("all tensors of a call must share one dtype")
            if t.shape != g.shape or t.device != grads[0].device:
                raise ValueError("grad, momentum and out must have the same shape and device")
            if g.numel() and _stack_layout(t) != layout:
                raise ValueError("grad, momentum and out must share their strides")
        arr[i] = MuonStack(*layout, _ptr(g), _ptr(m), _ptr(o))
    return arr, n, (MUON_BF16 if dt is None else dt)


def muon_stack_workspace_bytes(grads, momenta=None, outs=None) -> int:
    arr, n, dt = _stacks(grads, momenta, grads if outs is None else outs)
    out = ctypes.c_size_t(0)
    _check(load_library().muon_stack_workspace_bytes(arr, n, dt, ctypes.byref(out)), "muon_stack_workspace_bytes")
    return out.value


class StackPlan:
    """The Muon step on stacks of matrices with a short side (at most 128): 3-D views
    (count, rows, cols) over bf16 or float32 tensors, every matrix orthogonalised by itself.
    The heads of a fused projection are ``w.view(heads, head_dim, d)``, those of an output
    projection ``w.view(d, heads, head_dim).transpose(0, 1)``: no copy is made. grad, momentum
    and out of a stack share their strides; ``out`` may be the grad itself, and is written by
    ``step`` only (``step_apply`` writes the weights). A step needs a ``workspace``, allocated per
    call unless one is given; calls that overlap in time need one each."""

    def __init__(self, grads, momenta, outs):
        import torch
        lib = load_library()
        self.handle = ctypes.c_void_p(None)
        self._keep = (list(grads), None if momenta is None else list(momenta), list(outs))
        arr, n, dt = _stacks(*self._keep)
        self.dtype, self.n = dt, n
        self.device = grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
        if self.device.type != "cuda":
            raise ValueError("stacks must be in device memory")
        ws = ctypes.c_size_t(0)
        _check(lib.muon_stack_workspace_bytes(arr, n, dt, ctypes.byref(ws)), "muon_stack_workspace_bytes")
        self.workspace_bytes = ws.value
        h = ctypes.c_void_p(None)
        with torch.cuda.device(self.device):
            _check(lib.muon_stack_plan_create(arr, n, dt, ctypes.byref(h)), "muon_stack_plan_create")
        self.handle = h

    def set_weights(self, weights, lr_mul=None, wd_mul=None):
        """Attaches one weight tensor per stack (the grad's shape and dtype, its own strides);
        lr_mul / wd_mul: per-stack multipliers (default 1)."""
        import torch
        n = self.n
        if len(weights) != n:
            raise ValueError("one weight per stack")
        lr_mul = [1.0] * n if lr_mul is None else list(lr_mul)
        wd_mul = [1.0] * n if wd_mul is None else list(wd_mul)
        arr = (MuonStackWeight * max(n, 1))()
        for i, w in enumerate(weights):
            g = self._keep[0][i]
            if w is None:
                arr[i] = MuonStackWeight(None, 0, 0, float(lr_mul[i]), float(wd_mul[i]))
                continue
            if w.shape != g.shape or _dtype_code(w) != self.dtype or w.device != self.device:
                raise ValueError("weight must match its grad's shape, dtype and device")
            ld, stride = _stack_layout(w)[3:]
            arr[i] = MuonStackWeight(_ptr(w), ld, stride, float(lr_mul[i]), float(wd_mul[i]))
        with torch.cuda.device(self.device):
            _check(load_library().muon_stack_plan_set_weights(self.handle, arr, n), "muon_stack_plan_set_weights")
        self._weights = list(weights)

    def set_grad_scale(self, scale):
        """Later steps use grad * scale (see ``MuonPlan.set_grad_scale``)."""
        p = _scale_ptr(scale, self.device)
        _check(load_library().muon_stack_plan_set_grad_scale(self.handle, p), "muon_stack_plan_set_grad_scale")
        self._grad_scale = scale

    def _run(self, entry, args, workspace, stream):
        import torch
        if workspace is None and stream is None:
            workspace = torch.empty(max(1, self.workspace_bytes), dtype=torch.uint8, device=self.device)
        elif workspace is None:
            # allocated and, once dropped, reused in the order of the stream that uses it
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), self.device)
            with torch.cuda.stream(s):
                workspace = torch.empty(max(1, self.workspace_bytes), dtype=torch.uint8, device=self.device)
        elif workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {self.device}")
        index = self.device.index
        handle = _current_stream(index) if stream is None else _stream_handle(stream)
        args = (self.handle, *args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), handle)
        fn = getattr(load_library(), entry)
        if torch.cuda.current_device() == index:
            _check(fn(*args), entry)
        else:
            with torch.cuda.device(index):
                _check(fn(*args), entry)
        return workspace

    def step(self, cfg: MuonConfig, workspace=None, stream=None):
        """One Muon update of every matrix into its out and momentum; returns the workspace."""
        return self._run("muon_stack_plan_step", (ctypes.byref(cfg),), workspace, stream)

    def step_apply(self, cfg: MuonConfig, lr: float, wd: float, workspace=None, stream=None):
        """The same with W <- W (1 - lr' wd') - lr' X into the attached weights, lr' = lr lr_mul, wd' = wd wd_mul
        (``out`` is not written)."""
        ap = MuonApply(float(lr), float(wd))
        return self._run("muon_stack_plan_step_apply", (ctypes.byref(cfg), ctypes.byref(ap)), workspace, stream)

    def destroy(self):
        if self.handle:
            load_library().muon_stack_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def muon_stack_plan_create(grads, momenta, outs) -> StackPlan:
    return StackPlan(grads, momenta, outs)


def muon_stack_plan_step(plan: StackPlan, cfg: MuonConfig, workspace=None, stream=None):
    return plan.step(cfg, workspace, stream)


def muon_stack_plan_set_weights(plan: StackPlan, weights, lr_mul=None, wd_mul=None):
    plan.set_weights(weights, lr_mul, wd_mul)


def muon_stack_plan_step_apply(plan: StackPlan, cfg: MuonConfig, lr: float, wd: float, workspace=None, stream=None):
    return plan.step_apply(cfg, lr, wd, workspace, stream)


def muon_stack_plan_set_grad_scale(plan: StackPlan, scale):
    plan.set_grad_scale(scale)


def muon_stack_plan_destroy(plan: StackPlan):
    plan.destroy()
