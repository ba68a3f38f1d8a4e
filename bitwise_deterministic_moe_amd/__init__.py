"""Python binding of libmoedet: the bitwise-deterministic MoE expert layer
for MI355X (gfx950).

Argument marshalling only.  Every step of the layer runs in the HIP kernels
of ``libmoedet.so``; PyTorch supplies device memory and the current stream.
The functions carry the names of the C ABI (include/moedet.h).  There is no
fallback: a missing library raises ``MoeLibraryMissing``.
"""
import ctypes
import functools
import math
import os
from dataclasses import dataclass, replace
from typing import Optional

import torch

__all__ = [
    "DETERMINISTIC", "ATOMIC", "Problem", "Routing", "MoeError", "MoeLibraryMissing",
    "load_library", "library_path", "moe_workspace_size", "moe_rows_cap", "moe_stage_names",
    "moe_fwd", "moe_bwd_dgrad_dprob", "moe_bwd_wgrad", "moe_fingerprint", "moe_sched_elems", "moe_mfma_rate",
    "moe_router_bwd", "moe_router_fwd", "moe_sgd_step", "moe_mx_quantize", "moe_mx_dgrad_fc1",
    "moe_bwd_dgrad_dprob_noalloc", "moe_mx_quantize_t", "moe_mx_fwd_fc1", "moe_mx_fwd_fc2", "EXPORTED_SYMBOLS",
    "moe_mx_wgrad_rows", "moe_mx_quantize_wgrad", "moe_mx_wgrad", "MXW_TOKEN", "MXW_ROW", "MXW_ACT_P",
    "moe_route", "moe_layernorm_fwd", "moe_layernorm_bwd", "moe_linear_fwd", "moe_linear_bwd", "moe_glu_fwd",
    "moe_glu_bwd", "moe_layernorm_workspace_size", "moe_linear_workspace_size", "moe_glu_workspace_size", "ACTIVATIONS",
    "moe_linear_stage_names", "moe_glu_stage_names",
]

DETERMINISTIC = 0
ATOMIC = 1
DTYPE_CODE = {"f32": 0, "bf16": 1, "i32": 2, "u8": 3, "i64": 4, "f64": 5}
TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_TORCH_TO_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.int32: 2, torch.uint8: 3,
                  torch.int64: 4, torch.float64: 5}
EXPORTED_SYMBOLS = ("moe_abi_version", "moe_status_string", "moe_rows_cap", "moe_sched_elems",
                    "moe_workspace_size", "moe_stage_names", "moe_fwd", "moe_bwd_dgrad_dprob", "moe_bwd_wgrad",
                    "moe_fingerprint", "moe_mfma_rate", "moe_router_bwd", "moe_router_fwd", "moe_sgd_step",
                    "moe_mx_quantize", "moe_mx_dgrad_fc1", "moe_mx_dgrad_fc2",
                    "moe_nvfp4_quantize", "moe_bwd_dgrad_dprob_noalloc", "moe_mx_quantize_t", "moe_mx_fwd_fc1",
                    "moe_mx_fwd_fc2", "moe_mx_wgrad_rows", "moe_mx_quantize_wgrad", "moe_mx_wgrad", "moe_route",
                    "moe_source_hash", "moe_layernorm_workspace_size", "moe_layernorm_fwd", "moe_layernorm_bwd",
                    "moe_linear_workspace_size", "moe_linear_fwd", "moe_linear_bwd", "moe_glu_workspace_size",
                    "moe_glu_fwd", "moe_glu_bwd", "moe_linear_stage_names", "moe_glu_stage_names")
# activations of the dense operators (moe_act)
ACTIVATIONS = {"none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4}
# matrices of a dense call that may start at any element (moe_any)
_ANY = {"x": 0x100, "w": 0x200, "y": 0x400, "rest": 0x800}
# rows read by moe_mx_quantize_wgrad (moe_mxw_src)
MXW_TOKEN, MXW_ROW, MXW_ACT_P = 0, 1, 2

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


class MoeError(RuntimeError):
    pass


class MoeLibraryMissing(MoeError):
    pass


class MoeLibraryStale(MoeError):
    """The in-tree libmoedet.so was built from other sources than the tree's."""


class _CProblem(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("d_model", ctypes.c_int32), ("d_ffn", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("expert_begin", ctypes.c_int32), ("num_local", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("combine", ctypes.c_int32),
                ("debug_shuffle_seed", ctypes.c_uint64), ("stage_events", ctypes.c_void_p),
                ("n_stage_events", ctypes.c_int32)]


class _CRouting(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_idx", "topk_prob", "counts", "offsets",
                                                "row_src", "row_tok", "row_prob", "slot_row", "sched")]


class _CDense(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("z_dtype", ctypes.c_int32),
                ("act", ctypes.c_int32),
                ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldy", ctypes.c_int64), ("ldz", ctypes.c_int64),
                ("ldr", ctypes.c_int64), ("debug_shuffle_seed", ctypes.c_uint64)]


def library_path() -> str:
    return os.environ.get("MOEDET_LIB", os.path.join(_HERE, "libmoedet.so"))


def load_library() -> ctypes.CDLL:
    """Load libmoedet.so (build it with ``python -m bitwise_deterministic_moe_amd.build``)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise MoeLibraryMissing(f"{path} not found; build it with python -m bitwise_deterministic_moe_amd.build")
    lib = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER(_CProblem)
    R = ctypes.POINTER(_CRouting)
    lib.moe_abi_version.restype = ctypes.c_int
    lib.moe_source_hash.restype = ctypes.c_char_p
    lib.moe_source_hash.argtypes = []
    if "MOEDET_LIB" not in os.environ and os.path.isdir(os.path.join(_HERE, "csrc")):
        # the in-tree library must have been built from the tree's sources
        from .build import source_hash
        built, tree = lib.moe_source_hash().decode(), source_hash()
        if built != tree:
            raise MoeLibraryStale(f"{path} was built from sources {built}, the tree holds {tree}; rebuild it with "
                                  "python -m bitwise_deterministic_moe_amd.build")
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_rows_cap.argtypes = [P, ctypes.POINTER(ctypes.c_int64)]
    lib.moe_sched_elems.argtypes = [P, ctypes.POINTER(ctypes.c_int64)]
    lib.moe_workspace_size.argtypes = [P, ctypes.c_int, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]
    lib.moe_stage_names.restype = ctypes.c_char_p
    lib.moe_stage_names.argtypes = [P, ctypes.c_int, ctypes.c_int]
    lib.moe_fwd.argtypes = [P, vp, vp, vp, vp, R, vp, vp, vp, sz, ctypes.c_int, vp]
    lib.moe_bwd_dgrad_dprob.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_int, vp]
    lib.moe_bwd_wgrad.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_int, vp]
    lib.moe_bwd_dgrad_dprob_noalloc.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int, vp]
    lib.moe_fingerprint.argtypes = [vp, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int64), ctypes.c_int64,
                                    vp, vp, vp]
    lib.moe_mfma_rate.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_float, vp, vp]
    lib.moe_router_bwd.argtypes = [P, R, vp, vp, vp, vp, vp, vp, ctypes.c_int, vp]
    lib.moe_router_fwd.argtypes = [P, vp, vp, vp, vp]
    lib.moe_sgd_step.argtypes = [vp, vp, ctypes.c_int64, ctypes.c_float, vp, ctypes.c_int, vp]
    lib.moe_mx_quantize.argtypes = [vp, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, vp, vp, ctypes.c_uint64, vp]
    lib.moe_mx_dgrad_fc1.argtypes = [P, R, vp, vp, vp, vp, vp, vp]
    lib.moe_nvfp4_quantize.argtypes = [vp, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, vp, vp, vp, ctypes.c_uint64,
                                       vp]
    lib.moe_mx_dgrad_fc2.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_int, vp]
    lib.moe_mx_quantize_t.argtypes = [vp, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vp, vp,
                                      ctypes.c_uint64, vp]
    lib.moe_mx_fwd_fc1.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_mx_fwd_fc2.argtypes = [P, R, vp, vp, vp, vp, vp, vp, sz, ctypes.c_int, vp]
    lib.moe_mx_wgrad_rows.argtypes = [P, ctypes.POINTER(ctypes.c_int64)]
    lib.moe_route.argtypes = [P, vp, R, vp, sz, ctypes.c_int, vp]
    lib.moe_mx_quantize_wgrad.argtypes = [P, R, vp, ctypes.c_int, vp, vp, vp]
    lib.moe_mx_wgrad.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    i64, u64, N = ctypes.c_int64, ctypes.c_uint64, ctypes.POINTER(_CDense)
    lib.moe_layernorm_fwd.argtypes = [vp, vp, vp, ctypes.c_int, i64, i64, i64, ctypes.c_float, vp, vp, vp, u64, vp]
    lib.moe_layernorm_workspace_size.argtypes = [i64, i64, ctypes.POINTER(sz)]
    lib.moe_layernorm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i64, i64, vp, vp, vp, vp, sz,
                                      u64, vp]
    for f in ("moe_linear_workspace_size", "moe_glu_workspace_size"):
        getattr(lib, f).argtypes = [N, ctypes.POINTER(sz), ctypes.POINTER(sz)]
        getattr(lib, f).restype = ctypes.c_int
    for f in ("moe_linear_stage_names", "moe_glu_stage_names"):
        getattr(lib, f).argtypes = [N, ctypes.c_int, ctypes.c_char_p, sz]
        getattr(lib, f).restype = ctypes.c_int
    lib.moe_linear_fwd.argtypes = [N] + [vp] * 7 + [sz, vp]
    lib.moe_linear_bwd.argtypes = [N] + [vp] * 9 + [sz, vp]
    lib.moe_glu_fwd.argtypes = [N] + [vp] * 7 + [sz, vp]
    lib.moe_glu_bwd.argtypes = [N] + [vp] * 11 + [sz, vp]
    for f in ("moe_layernorm_fwd", "moe_layernorm_workspace_size", "moe_layernorm_bwd", "moe_linear_fwd",
              "moe_linear_bwd", "moe_glu_fwd", "moe_glu_bwd"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("moe_route", "moe_mx_wgrad_rows", "moe_mx_quantize_wgrad", "moe_mx_wgrad", "moe_rows_cap",
              "moe_sched_elems", "moe_workspace_size", "moe_fwd", "moe_bwd_dgrad_dprob",
              "moe_bwd_dgrad_dprob_noalloc", "moe_mx_quantize_t", "moe_mx_fwd_fc1", "moe_mx_fwd_fc2",
              "moe_bwd_wgrad", "moe_fingerprint", "moe_mfma_rate", "moe_router_bwd", "moe_router_fwd",
              "moe_sgd_step", "moe_mx_quantize", "moe_mx_dgrad_fc1", "moe_mx_dgrad_fc2", "moe_nvfp4_quantize"):
        getattr(lib, f).restype = ctypes.c_int
    _LIB = lib
    return lib


def moe_source_hash() -> str:
    """Hash of the sources the loaded library was built from."""
    return load_library().moe_source_hash().decode()


def _check(status: int, what: str):
    if status != 0:
        msg = load_library().moe_status_string(status).decode()
        raise MoeError(f"{what}: status {status} ({msg})")


@dataclass(frozen=True)
class Problem:
    """Mirror of ``moe_problem``."""
    tokens: int
    d_model: int
    d_ffn: int
    num_experts: int
    top_k: int
    expert_begin: int = 0
    num_local: Optional[int] = None
    dtype: str = "bf16"
    combine: int = 1
    shuffle_seed: int = 0

    @property
    def local(self) -> int:
        return self.num_experts if self.num_local is None else self.num_local

    @property
    def rows_cap(self) -> int:
        return self.tokens * min(self.top_k, self.local)

    def with_seed(self, seed: int) -> "Problem":
        return replace(self, shuffle_seed=seed)

    def c(self, events=None) -> _CProblem:
        p = _CProblem(self.tokens, self.d_model, self.d_ffn, self.num_experts, self.top_k,
                      self.expert_begin, self.local, DTYPE_CODE[self.dtype], self.combine,
                      self.shuffle_seed & 0xFFFFFFFFFFFFFFFF, None, 0)
        if events:
            arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
            p.stage_events = ctypes.cast(arr, ctypes.c_void_p)
            p.n_stage_events = len(events)
            p._keep = arr
        return p

    @classmethod
    def from_config(cls, cfg, shuffle_seed: int = 0) -> "Problem":
        return cls(cfg.tokens, cfg.d_model, cfg.d_ffn, cfg.num_experts, cfg.top_k, cfg.expert_begin,
                   cfg.num_local, cfg.dtype, cfg.combine, shuffle_seed)


@dataclass
class Routing:
    """Device routing state (mirror of ``moe_routing``)."""
    topk_idx: torch.Tensor
    topk_prob: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    row_src: torch.Tensor
    row_tok: torch.Tensor
    row_prob: torch.Tensor
    slot_row: torch.Tensor
    sched: torch.Tensor

    @classmethod
    def empty(cls, prob: Problem, device="cuda") -> "Routing":
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        T, k, el, rc = prob.tokens, prob.top_k, prob.local, prob.rows_cap
        return cls(torch.empty((T, k), **i32), torch.empty((T, k), **f32), torch.empty(el, **i32),
                   torch.empty(el + 1, **i32), torch.empty(rc, **i32), torch.empty(rc, **i32),
                   torch.empty(rc, **f32), torch.empty(T * k, **i32), torch.empty(moe_sched_elems(prob), **i32))

    def c(self) -> _CRouting:
        return _CRouting(*[_ptr(getattr(self, n)) for n, _ in _CRouting._fields_])

    @property
    def rows(self) -> int:
        """R (synchronises: reads offsets[-1] to the host)."""
        return int(self.offsets[-1].item())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return t.data_ptr() or None


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _ws(nbytes: int, ws: Optional[torch.Tensor], device) -> torch.Tensor:
    if ws is not None:
        return ws
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def moe_rows_cap(prob: Problem) -> int:
    v = ctypes.c_int64()
    _check(load_library().moe_rows_cap(ctypes.byref(prob.c()), ctypes.byref(v)), "moe_rows_cap")
    return v.value


def moe_sched_elems(prob: Problem) -> int:
    """int32 elements of Routing.sched."""
    v = ctypes.c_int64()
    _check(load_library().moe_sched_elems(ctypes.byref(prob.c()), ctypes.byref(v)), "moe_sched_elems")
    return v.value


def moe_workspace_size(prob: Problem, mode: int = DETERMINISTIC):
    """Bytes of workspace for (moe_fwd, moe_bwd_dgrad_dprob, moe_bwd_wgrad)."""
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().moe_workspace_size(ctypes.byref(prob.c()), mode, ctypes.byref(a), ctypes.byref(b),
                                             ctypes.byref(c)), "moe_workspace_size")
    return a.value, b.value, c.value


def moe_stage_names(prob: Problem, mode: int, call: int):
    s = load_library().moe_stage_names(ctypes.byref(prob.c()), mode, call)
    return s.decode().split(",") if s else None


def moe_fwd(prob: Problem, logits, x, w1, w2, mode: int = DETERMINISTIC, routing: Routing = None,
            h=None, y=None, ws=None, events=None):
    """Routing + expert MLP + combine.  Returns (routing, h, y_or_rows)."""
    lib = load_library()
    dev = x.device
    dt = TORCH_DTYPE[prob.dtype]
    routing = routing or Routing.empty(prob, dev)
    if h is None:
        h = torch.empty((prob.rows_cap, prob.d_ffn), dtype=dt, device=dev)
    if y is None:
        y = torch.empty((prob.tokens if prob.combine else prob.rows_cap, prob.d_model), dtype=dt, device=dev)
    need = moe_workspace_size(prob, mode)[0]
    ws = _ws(need, ws, dev)
    T, E, D, F, el, rc = prob.tokens, prob.num_experts, prob.d_model, prob.d_ffn, prob.local, prob.rows_cap
    _need(logits, T * E, torch.float32, "moe_fwd logits")
    _need(x, T * D, dt, "moe_fwd x")
    _need(w1, el * D * F, dt, "moe_fwd w1")
    _need(w2, el * F * D, dt, "moe_fwd w2")
    _need(h, rc * F, dt, "moe_fwd h")
    _need(y, (T if prob.combine else rc) * D, dt, "moe_fwd y")
    cp, cr = prob.c(events), routing.c()
    _check(lib.moe_fwd(ctypes.byref(cp), _ptr(logits), _ptr(x), _ptr(w1), _ptr(w2), ctypes.byref(cr), _ptr(h),
                       _ptr(y), _ptr(ws), ws.numel(), mode, _stream()), "moe_fwd")
    return routing, h, y


def moe_route(prob: Problem, logits, mode: int = DETERMINISTIC, routing: Routing = None, ws=None, events=None):
    """The routing stage of moe_fwd alone (top-k, permutation, work list).
    Returns the routing."""
    lib = load_library()
    dev = logits.device
    routing = routing or Routing.empty(prob, dev)
    ws = _ws(moe_workspace_size(prob, mode)[0], ws, dev)
    _need(logits, prob.tokens * prob.num_experts, torch.float32, "moe_route logits")
    cp, cr = prob.c(events), routing.c()
    _check(lib.moe_route(ctypes.byref(cp), _ptr(logits), ctypes.byref(cr), _ptr(ws), ws.numel(), mode, _stream()),
           "moe_route")
    return routing


def moe_bwd_dgrad_dprob(prob: Problem, routing: Routing, dy, w1, w2, h, mode: int = DETERMINISTIC,
                        dx=None, dprob=None, dh=None, ws=None, events=None):
    """fc2 dgrad with dprob + fc1 dgrad + dx combine.
    Returns (dx_or_rows, dprob, dh)."""
    lib = load_library()
    dev = h.device
    dt = TORCH_DTYPE[prob.dtype]
    if dx is None:
        dx = torch.empty((prob.tokens if prob.combine else prob.rows_cap, prob.d_model), dtype=dt, device=dev)
    if dprob is None:
        dprob = torch.empty((prob.tokens, prob.top_k), dtype=torch.float32, device=dev)
    if dh is None:
        dh = torch.empty((prob.rows_cap, prob.d_ffn), dtype=dt, device=dev)
    need = moe_workspace_size(prob, mode)[1]
    ws = _ws(need, ws, dev)
    T, k, D, F, el, rc = prob.tokens, prob.top_k, prob.d_model, prob.d_ffn, prob.local, prob.rows_cap
    _need(dy, T * D, dt, "moe_bwd_dgrad_dprob dy")
    _need(w1, el * D * F, dt, "moe_bwd_dgrad_dprob w1")
    _need(w2, el * F * D, dt, "moe_bwd_dgrad_dprob w2")
    _need(h, rc * F, dt, "moe_bwd_dgrad_dprob h")
    _need(dx, (T if prob.combine else rc) * D, dt, "moe_bwd_dgrad_dprob dx")
    _need(dprob, T * k, torch.float32, "moe_bwd_dgrad_dprob dprob")
    _need(dh, rc * F, dt, "moe_bwd_dgrad_dprob dh")
    cp, cr = prob.c(events), routing.c()
    _check(lib.moe_bwd_dgrad_dprob(ctypes.byref(cp), ctypes.byref(cr), _ptr(dy), _ptr(w1), _ptr(w2), _ptr(h),
                                   _ptr(dx), _ptr(dprob), _ptr(dh), _ptr(ws), ws.numel(), mode, _stream()),
           "moe_bwd_dgrad_dprob")
    return dx, dprob, dh


NOALLOC_SCRATCH_BYTES = 64 << 20   # MOE_NOALLOC_SCRATCH_BYTES of moedet.h


def moe_bwd_dgrad_dprob_noalloc(prob: Problem, routing: Routing, dy, w1, w2, h, dx, dprob, dh,
                                mode: int = DETERMINISTIC, events=None):
    """moe_bwd_dgrad_dprob with the library's static per-GPU workspace: the
    caller passes inputs and preallocated outputs, nothing is allocated.
    Returns (dx_or_rows, dprob, dh)."""
    lib = load_library()
    dt = TORCH_DTYPE[prob.dtype]
    T, k, D, F, el, rc = prob.tokens, prob.top_k, prob.d_model, prob.d_ffn, prob.local, prob.rows_cap
    _need(dy, T * D, dt, "moe_bwd_dgrad_dprob_noalloc dy")
    _need(w1, el * D * F, dt, "moe_bwd_dgrad_dprob_noalloc w1")
    _need(w2, el * F * D, dt, "moe_bwd_dgrad_dprob_noalloc w2")
    _need(h, rc * F, dt, "moe_bwd_dgrad_dprob_noalloc h")
    _need(dx, (T if prob.combine else rc) * D, dt, "moe_bwd_dgrad_dprob_noalloc dx")
    _need(dprob, T * k, torch.float32, "moe_bwd_dgrad_dprob_noalloc dprob")
    _need(dh, rc * F, dt, "moe_bwd_dgrad_dprob_noalloc dh")
    cp, cr = prob.c(events), routing.c()
    _check(lib.moe_bwd_dgrad_dprob_noalloc(ctypes.byref(cp), ctypes.byref(cr), _ptr(dy), _ptr(w1), _ptr(w2), _ptr(h),
                                           _ptr(dx), _ptr(dprob), _ptr(dh), mode, _stream()),
           "moe_bwd_dgrad_dprob_noalloc")
    return dx, dprob, dh


def moe_bwd_wgrad(prob: Problem, routing: Routing, x, dy, h, dh, mode: int = DETERMINISTIC, dw1=None,
                  dw2=None, ws=None, events=None):
    """Expert weight gradients (float32) from the layer input x, the upstream
    gradient dy, the saved h and dh.  Returns (dw1, dw2)."""
    lib = load_library()
    dev = dh.device
    el, D, F = prob.local, prob.d_model, prob.d_ffn
    if dw1 is None:
        dw1 = torch.empty((el, D, F), dtype=torch.float32, device=dev)
    if dw2 is None:
        dw2 = torch.empty((el, F, D), dtype=torch.float32, device=dev)
    need = moe_workspace_size(prob, mode)[2]
    ws = _ws(need, ws, dev)
    dt = TORCH_DTYPE[prob.dtype]
    T, rc = prob.tokens, prob.rows_cap
    _need(x, T * D, dt, "moe_bwd_wgrad x")
    _need(dy, T * D, dt, "moe_bwd_wgrad dy")
    _need(h, rc * F, dt, "moe_bwd_wgrad h")
    _need(dh, rc * F, dt, "moe_bwd_wgrad dh")
    _need(dw1, el * D * F, torch.float32, "moe_bwd_wgrad dw1")
    _need(dw2, el * F * D, torch.float32, "moe_bwd_wgrad dw2")
    cp, cr = prob.c(events), routing.c()
    _check(lib.moe_bwd_wgrad(ctypes.byref(cp), ctypes.byref(cr), _ptr(x), _ptr(dy), _ptr(h), _ptr(dh), _ptr(dw1),
                             _ptr(dw2), _ptr(ws), ws.numel(), mode, _stream()), "moe_bwd_wgrad")
    return dw1, dw2


def moe_router_bwd(prob: Problem, routing: Routing, dprob, x, w_router, mode: int = DETERMINISTIC, dlogits=None,
                   dw_router=None, dx_router=None):
    """Router backward (full layer only).  Returns (dlogits float32 [T,E],
    dw_router float32 [E,D], dx_router [T,D] in the storage dtype)."""
    lib = load_library()
    dev = w_router.device
    T, E, D = prob.tokens, prob.num_experts, prob.d_model
    if dlogits is None:
        dlogits = torch.empty((T, E), dtype=torch.float32, device=dev)
    if dw_router is None:
        dw_router = torch.empty((E, D), dtype=torch.float32, device=dev)
    if dx_router is None:
        dx_router = torch.empty((T, D), dtype=TORCH_DTYPE[prob.dtype], device=dev)
    dt = TORCH_DTYPE[prob.dtype]
    _need(dprob, T * prob.top_k, torch.float32, "moe_router_bwd dprob")
    _need(x, T * D, dt, "moe_router_bwd x")
    _need(w_router, E * D, dt, "moe_router_bwd w_router")
    _need(dlogits, T * E, torch.float32, "moe_router_bwd dlogits")
    _need(dw_router, E * D, torch.float32, "moe_router_bwd dw_router")
    _need(dx_router, T * D, dt, "moe_router_bwd dx_router")
    cp, cr = prob.c(), routing.c()
    _check(lib.moe_router_bwd(ctypes.byref(cp), ctypes.byref(cr), _ptr(dprob), _ptr(x), _ptr(w_router), _ptr(dlogits),
                              _ptr(dw_router), _ptr(dx_router), mode, _stream()), "moe_router_bwd")
    return dlogits, dw_router, dx_router


def moe_router_fwd(prob: Problem, x, w_router, logits=None):
    """Router logits float32 [T,E] = x w_router^T (d ascending, fp32 FMA)."""
    lib = load_library()
    if logits is None:
        logits = torch.empty((prob.tokens, prob.num_experts), dtype=torch.float32, device=w_router.device)
    dt = TORCH_DTYPE[prob.dtype]
    _need(x, prob.tokens * prob.d_model, dt, "moe_router_fwd x")
    _need(w_router, prob.num_experts * prob.d_model, dt, "moe_router_fwd w_router")
    _need(logits, prob.tokens * prob.num_experts, torch.float32, "moe_router_fwd logits")
    cp = prob.c()
    _check(lib.moe_router_fwd(ctypes.byref(cp), _ptr(x), _ptr(w_router), _ptr(logits), _stream()), "moe_router_fwd")
    return logits


def moe_sgd_step(master: torch.Tensor, grad: torch.Tensor, lr: float, runtime: torch.Tensor):
    """master -= lr * grad (float32, in place); runtime = master rounded to
    runtime's dtype.  All three tensors contiguous with the same element count."""
    lib = load_library()
    if not (master.is_contiguous() and grad.is_contiguous() and runtime.is_contiguous()):
        raise MoeError("moe_sgd_step needs contiguous tensors")
    n = master.numel()
    if grad.numel() != n or runtime.numel() != n or master.dtype != torch.float32 or grad.dtype != torch.float32:
        raise MoeError("moe_sgd_step: master and grad float32 with runtime's element count")
    code = _TORCH_TO_CODE[runtime.dtype]
    _check(lib.moe_sgd_step(_ptr(master), _ptr(grad), n, lr, _ptr(runtime), code, _stream()), "moe_sgd_step")
    return master, runtime


def _need(t: torch.Tensor, numel: int, dtype, what: str):
    """Argument check before a raw pointer crosses the boundary: the kernels
    behind it take sizes from the problem, not from the tensor."""
    if t.dtype != dtype or not t.is_contiguous() or t.numel() != numel:
        raise MoeError(f"{what}: need a contiguous {dtype} tensor of {numel} elements, "
                       f"got {t.dtype} {tuple(t.shape)} (contiguous={t.is_contiguous()})")


def moe_mx_quantize(t: torch.Tensor, codes=None, scales=None, shuffle_seed: int = 0):
    """MXFP8 (E4M3 codes, E8M0 scales per 32 elements of the last dimension)
    of a contiguous float32 or bf16 tensor.  Returns (codes uint8 with t's
    shape, scales uint8 [..., cols/32])."""
    lib = load_library()
    if not t.is_contiguous() or t.dim() < 1:
        raise MoeError("moe_mx_quantize needs a contiguous tensor")
    cols = t.shape[-1]
    rows = t.numel() // cols if cols else 0
    if codes is None:
        codes = torch.empty(t.shape, dtype=torch.uint8, device=t.device)
    if scales is None:
        scales = torch.empty(tuple(t.shape[:-1]) + (cols // 32,), dtype=torch.uint8, device=t.device)
    _need(codes, t.numel(), torch.uint8, "moe_mx_quantize codes")
    _need(scales, rows * (cols // 32), torch.uint8, "moe_mx_quantize scales")
    _check(lib.moe_mx_quantize(_ptr(t), _TORCH_TO_CODE[t.dtype], rows, cols, _ptr(codes), _ptr(scales),
                               shuffle_seed & 0xFFFFFFFFFFFFFFFF, _stream()), "moe_mx_quantize")
    return codes, scales


def moe_nvfp4_quantize(t: torch.Tensor, shuffle_seed: int = 0):
    """NVFP4 of a contiguous float32 or bf16 tensor (blocks of 16 along the
    last dimension).  Returns (packed codes uint8 [..., cols/2], block scales
    uint8 [..., cols/16], tensor scale float32 [1])."""
    lib = load_library()
    if not t.is_contiguous() or t.dim() < 1:
        raise MoeError("moe_nvfp4_quantize needs a contiguous tensor")
    cols = t.shape[-1]
    rows = t.numel() // cols if cols else 0
    codes = torch.empty(tuple(t.shape[:-1]) + (cols // 2,), dtype=torch.uint8, device=t.device)
    scales = torch.empty(tuple(t.shape[:-1]) + (cols // 16,), dtype=torch.uint8, device=t.device)
    g = torch.empty(1, dtype=torch.float32, device=t.device)
    _check(lib.moe_nvfp4_quantize(_ptr(t), _TORCH_TO_CODE[t.dtype], rows, cols, _ptr(codes), _ptr(scales), _ptr(g),
                                  shuffle_seed & 0xFFFFFFFFFFFFFFFF, _stream()), "moe_nvfp4_quantize")
    return codes, scales, g


def moe_mx_dgrad_fc1(prob: Problem, routing: Routing, dh_mx, w1_mx, dx_rows=None):
    """MXFP8 fc1 data gradient: dx_rows [rows_cap, D] bf16 from (codes, scales)
    of dh [rows_cap, F] and of W1 [num_local, D, F] (moe_mx_quantize outputs)."""
    lib = load_library()
    (dc, ds), (wc, wsc) = dh_mx, w1_mx
    if dx_rows is None:
        dx_rows = torch.empty((prob.rows_cap, prob.d_model), dtype=torch.bfloat16, device=dc.device)
    rc, D, F, el = prob.rows_cap, prob.d_model, prob.d_ffn, prob.local
    _need(dc, rc * F, torch.uint8, "moe_mx_dgrad_fc1 dh codes")
    _need(ds, rc * (F // 32), torch.uint8, "moe_mx_dgrad_fc1 dh scales")
    _need(wc, el * D * F, torch.uint8, "moe_mx_dgrad_fc1 W1 codes")
    _need(wsc, el * D * (F // 32), torch.uint8, "moe_mx_dgrad_fc1 W1 scales")
    _need(dx_rows, rc * D, torch.bfloat16, "moe_mx_dgrad_fc1 dx_rows")
    cp, cr = prob.c(), routing.c()
    _check(lib.moe_mx_dgrad_fc1(ctypes.byref(cp), ctypes.byref(cr), _ptr(dc), _ptr(ds), _ptr(wc), _ptr(wsc),
                                _ptr(dx_rows), _stream()), "moe_mx_dgrad_fc1")
    return dx_rows


def moe_mx_dgrad_fc2(prob: Problem, routing: Routing, dy_mx, w2_mx, h, mode: int = DETERMINISTIC, dprob=None,
                     dh=None, ws=None):
    """MXFP8 fc2 data gradient with the fused dprob / dh epilogue, from
    (codes, scales) of dy [T, D] and of W2 [num_local, F, D] (moe_mx_quantize
    outputs) and the saved h.  Returns (dprob float32 [T, k], dh bf16
    [rows_cap, F]).  The workspace is the dgrad one (moe_workspace_size)."""
    lib = load_library()
    (dc, ds), (wc, wsc) = dy_mx, w2_mx
    dev = h.device
    if dprob is None:
        dprob = torch.empty((prob.tokens, prob.top_k), dtype=torch.float32, device=dev)
    if dh is None:
        dh = torch.empty((prob.rows_cap, prob.d_ffn), dtype=torch.bfloat16, device=dev)
    ws = _ws(moe_workspace_size(prob, mode)[1], ws, dev)
    T, k, rc, D, F, el = prob.tokens, prob.top_k, prob.rows_cap, prob.d_model, prob.d_ffn, prob.local
    _need(dc, T * D, torch.uint8, "moe_mx_dgrad_fc2 dy codes")
    _need(ds, T * (D // 32), torch.uint8, "moe_mx_dgrad_fc2 dy scales")
    _need(wc, el * F * D, torch.uint8, "moe_mx_dgrad_fc2 W2 codes")
    _need(wsc, el * F * (D // 32), torch.uint8, "moe_mx_dgrad_fc2 W2 scales")
    _need(h, rc * F, torch.bfloat16, "moe_mx_dgrad_fc2 h")
    _need(dprob, T * k, torch.float32, "moe_mx_dgrad_fc2 dprob")
    _need(dh, rc * F, torch.bfloat16, "moe_mx_dgrad_fc2 dh")
    cp, cr = prob.c(), routing.c()
    _check(lib.moe_mx_dgrad_fc2(ctypes.byref(cp), ctypes.byref(cr), _ptr(dc), _ptr(ds), _ptr(wc), _ptr(wsc), _ptr(h),
                                _ptr(dprob), _ptr(dh), _ptr(ws), ws.numel(), mode, _stream()),
           "moe_mx_dgrad_fc2")
    return dprob, dh


def moe_mx_quantize_t(t: torch.Tensor, codes=None, scales=None, shuffle_seed: int = 0):
    """MXFP8 of the transpose of each [rows, cols] matrix of a contiguous
    [groups, rows, cols] (or [rows, cols]) float32 / bf16 tensor: blocks of 32
    consecutive rows of a column.  Returns (codes uint8 [groups, cols, rows],
    scales uint8 [groups, cols, rows/32]) (without the group axis for 2-D input)."""
    lib = load_library()
    if not t.is_contiguous() or t.dim() not in (2, 3):
        raise MoeError("moe_mx_quantize_t needs a contiguous [groups,] rows, cols tensor")
    g, rows, cols = (1,) + tuple(t.shape) if t.dim() == 2 else tuple(t.shape)
    shp = (cols, rows) if t.dim() == 2 else (g, cols, rows)
    if codes is None:
        codes = torch.empty(shp, dtype=torch.uint8, device=t.device)
    if scales is None:
        scales = torch.empty(shp[:-1] + (rows // 32,), dtype=torch.uint8, device=t.device)
    _need(codes, g * rows * cols, torch.uint8, "moe_mx_quantize_t codes")
    _need(scales, g * cols * (rows // 32), torch.uint8, "moe_mx_quantize_t scales")
    _check(lib.moe_mx_quantize_t(_ptr(t), _TORCH_TO_CODE[t.dtype], g, rows, cols, _ptr(codes), _ptr(scales),
                                 shuffle_seed & 0xFFFFFFFFFFFFFFFF, _stream()), "moe_mx_quantize_t")
    return codes, scales


def moe_mx_fwd_fc1(prob: Problem, routing: Routing, x_mx, w1t_mx, h=None, act=None):
    """MXFP8 forward fc1: h and act = relu(h)^2 (bf16 [rows_cap, F]) from the
    (codes, scales) of x [T, D] (moe_mx_quantize) and of W1 transposed
    [num_local, F, D] (moe_mx_quantize_t of W1).  Returns (h, act)."""
    lib = load_library()
    (xc, xs), (wc, wsc) = x_mx, w1t_mx
    rc, T, D, F, el = prob.rows_cap, prob.tokens, prob.d_model, prob.d_ffn, prob.local
    if h is None:
        h = torch.empty((rc, F), dtype=torch.bfloat16, device=xc.device)
    if act is None:
        act = torch.empty((rc, F), dtype=torch.bfloat16, device=xc.device)
    _need(xc, T * D, torch.uint8, "moe_mx_fwd_fc1 x codes")
    _need(xs, T * (D // 32), torch.uint8, "moe_mx_fwd_fc1 x scales")
    _need(wc, el * F * D, torch.uint8, "moe_mx_fwd_fc1 W1^T codes")
    _need(wsc, el * F * (D // 32), torch.uint8, "moe_mx_fwd_fc1 W1^T scales")
    _need(h, rc * F, torch.bfloat16, "moe_mx_fwd_fc1 h")
    _need(act, rc * F, torch.bfloat16, "moe_mx_fwd_fc1 act")
    cp, cr = prob.c(), routing.c()
    _check(lib.moe_mx_fwd_fc1(ctypes.byref(cp), ctypes.byref(cr), _ptr(xc), _ptr(xs), _ptr(wc), _ptr(wsc), _ptr(h),
                              _ptr(act), _stream()), "moe_mx_fwd_fc1")
    return h, act


def moe_mx_fwd_fc2(prob: Problem, routing: Routing, act_mx, w2t_mx, mode: int = DETERMINISTIC, y=None, ws=None):
    """MXFP8 forward fc2 and the combine: y [T, D] (combine=1) or the o rows
    [rows_cap, D] (bf16) from the (codes, scales) of act [rows_cap, F]
    (moe_mx_quantize) and of W2 transposed [num_local, D, F] (moe_mx_quantize_t
    of W2).  The workspace is the forward one (moe_workspace_size)."""
    lib = load_library()
    (ac, asc), (wc, wsc) = act_mx, w2t_mx
    rc, T, D, F, el = prob.rows_cap, prob.tokens, prob.d_model, prob.d_ffn, prob.local
    out_rows = T if prob.combine else rc
    if y is None:
        y = torch.empty((out_rows, D), dtype=torch.bfloat16, device=ac.device)
    ws = _ws(moe_workspace_size(prob, mode)[0], ws, ac.device)
    _need(ac, rc * F, torch.uint8, "moe_mx_fwd_fc2 act codes")
    _need(asc, rc * (F // 32), torch.uint8, "moe_mx_fwd_fc2 act scales")
    _need(wc, el * D * F, torch.uint8, "moe_mx_fwd_fc2 W2^T codes")
    _need(wsc, el * D * (F // 32), torch.uint8, "moe_mx_fwd_fc2 W2^T scales")
    _need(y, out_rows * D, torch.bfloat16, "moe_mx_fwd_fc2 y")
    cp, cr = prob.c(), routing.c()
    _check(lib.moe_mx_fwd_fc2(ctypes.byref(cp), ctypes.byref(cr), _ptr(ac), _ptr(asc), _ptr(wc), _ptr(wsc), _ptr(y),
                              _ptr(ws), ws.numel(), mode, _stream()), "moe_mx_fwd_fc2")
    return y


def moe_mx_wgrad_rows(prob: Problem) -> int:
    """rpad_cap: padded rows of the MXFP8 weight-gradient operands (each
    expert's routed rows padded to a multiple of 64)."""
    v = ctypes.c_int64()
    _check(load_library().moe_mx_wgrad_rows(ctypes.byref(prob.c()), ctypes.byref(v)), "moe_mx_wgrad_rows")
    return v.value


def moe_mx_quantize_wgrad(prob: Problem, routing: Routing, src: torch.Tensor, kind: int, codes=None, scales=None):
    """MXFP8 of a weight-gradient operand along each expert's routed rows.
    kind MXW_TOKEN: src [T, D] gathered by token (x, dY); MXW_ROW: src
    [rows_cap, F] (dH); MXW_ACT_P: src = h [rows_cap, F], encodes
    p relu(h)^2.  Returns (codes uint8 [rpad_cap / 64, cols, 64], scales
    uint8 [rpad_cap / 64, cols, 2]), slice-major; slices past the padded
    total are not written."""
    lib = load_library()
    rp = moe_mx_wgrad_rows(prob)
    cols = prob.d_model if kind == MXW_TOKEN else prob.d_ffn
    rows = prob.tokens if kind == MXW_TOKEN else prob.rows_cap
    _need(src, rows * cols, torch.bfloat16, "moe_mx_quantize_wgrad src")
    if codes is None:
        codes = torch.empty((rp // 64, cols, 64), dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = torch.empty((rp // 64, cols, 2), dtype=torch.uint8, device=src.device)
    _need(codes, cols * rp, torch.uint8, "moe_mx_quantize_wgrad codes")
    _need(scales, cols * (rp // 32), torch.uint8, "moe_mx_quantize_wgrad scales")
    cp, cr = prob.c(), routing.c()
    _check(lib.moe_mx_quantize_wgrad(ctypes.byref(cp), ctypes.byref(cr), _ptr(src), kind, _ptr(codes), _ptr(scales),
                                     _stream()), "moe_mx_quantize_wgrad")
    return codes, scales


def moe_mx_wgrad(prob: Problem, routing: Routing, x_mx, dh_mx, act_mx, dy_mx, dw1=None, dw2=None):
    """MXFP8 weight gradients dW1 [num_local, D, F] and dW2 [num_local, F, D]
    (float32) from the moe_mx_quantize_wgrad encodings of x (MXW_TOKEN), dH
    (MXW_ROW), h (MXW_ACT_P) and dY (MXW_TOKEN)."""
    lib = load_library()
    rp = moe_mx_wgrad_rows(prob)
    D, F, el = prob.d_model, prob.d_ffn, prob.local
    ops = []
    for (c, s), n, name in ((x_mx, D, "x"), (dh_mx, F, "dh"), (act_mx, F, "act"), (dy_mx, D, "dy")):
        _need(c, n * rp, torch.uint8, f"moe_mx_wgrad {name} codes")
        _need(s, n * (rp // 32), torch.uint8, f"moe_mx_wgrad {name} scales")
        ops += [_ptr(c), _ptr(s)]
    dev = x_mx[0].device
    if dw1 is None:
        dw1 = torch.empty((el, D, F), dtype=torch.float32, device=dev)
    if dw2 is None:
        dw2 = torch.empty((el, F, D), dtype=torch.float32, device=dev)
    _need(dw1, el * D * F, torch.float32, "moe_mx_wgrad dw1")
    _need(dw2, el * F * D, torch.float32, "moe_mx_wgrad dw2")
    cp, cr = prob.c(), routing.c()
    _check(lib.moe_mx_wgrad(ctypes.byref(cp), ctypes.byref(cr), *ops, _ptr(dw1), _ptr(dw2), _stream()),
           "moe_mx_wgrad")
    return dw1, dw2


def moe_fingerprint(t: torch.Tensor, dtype: Optional[str] = None, chunk_elems: int = 65536,
                    shape=None, sync: bool = True):
    """Chunk hashes (device uint64 as int64 tensor) and the total.

    ``dtype`` names the element type ("f32", "bf16", "i32", ...); by default
    it follows the tensor.  With ``sync`` the 8-byte total is copied to the
    host and returned as a Python int; otherwise the device tensor."""
    lib = load_library()
    if not t.is_contiguous():
        raise MoeError("fingerprint needs a contiguous tensor")
    code = DTYPE_CODE[dtype] if dtype else _TORCH_TO_CODE[t.dtype]
    shape = tuple(t.shape) if shape is None else tuple(shape)
    n = 1
    for s in shape:
        n *= s
    m = (n + chunk_elems - 1) // chunk_elems
    hashes = torch.empty(max(m, 1), dtype=torch.int64, device=t.device)
    total = torch.empty(1, dtype=torch.int64, device=t.device)
    arr = (ctypes.c_int64 * max(len(shape), 1))(*shape)
    _check(lib.moe_fingerprint(_ptr(t), code, len(shape), arr, chunk_elems, _ptr(hashes), _ptr(total), _stream()),
           "moe_fingerprint")
    if not sync:
        return hashes[:m], total
    return hashes[:m], int(total.item()) & 0xFFFFFFFFFFFFFFFF


def moe_mfma_rate(blocks: int, iters: int, value: float = 0.125, sink: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Enqueue the MFMA-rate loop on the current stream; returns the sink
    (float32 [256 * blocks] on the current device)."""
    lib = load_library()
    if sink is None:
        sink = torch.empty(256 * blocks, dtype=torch.float32, device="cuda")
    _check(lib.moe_mfma_rate(blocks, iters, value, _ptr(sink), _stream()), "moe_mfma_rate")
    return sink


# ---------------------------------------------------------------- dense operators
def _mat(t: torch.Tensor, cols: int, dtype, what: str, rows: Optional[int] = None):
    """(rows, row distance) of a matrix [..., cols] of unit stride along its
    rows: two-dimensional with any row distance, or contiguous."""
    shape = t.shape
    if t.dtype is dtype and len(shape) == 2 and shape[1] == cols and t.is_contiguous() and rows in (None, shape[0]):
        return shape[0], cols
    if t.dtype != dtype or len(shape) == 0 or shape[-1] != cols:
        raise MoeError(f"{what}: need a {dtype} tensor [..., {cols}], got {t.dtype} {tuple(shape)}")
    if len(shape) == 2:
        n, ld = shape[0], t.stride(0)
        if n and ((cols > 1 and t.stride(1) != 1) or (n > 1 and ld < cols)):
            raise MoeError(f"{what}: rows of unit stride at least their length apart are needed, got strides {t.stride()}")
        if n <= 1:
            ld = cols
    else:
        if not t.is_contiguous():
            raise MoeError(f"{what}: a tensor of {len(shape)} dimensions must be contiguous")
        n, ld = t.numel() // cols if cols else 0, cols
    if rows is not None and n != rows:
        raise MoeError(f"{what}: need {rows} rows, got {n}")
    return n, ld


def _storage(t: torch.Tensor, what: str) -> int:
    if t.dtype is torch.bfloat16:
        return 1
    if t.dtype is torch.float32:
        return 0
    raise MoeError(f"{what}: float32 or bfloat16 is needed, got {t.dtype}")


def _grad_code(dtype, storage, what: str) -> int:
    if dtype is not torch.float32 and dtype is not storage:
        raise MoeError(f"{what}: grad_dtype must be torch.float32 or the storage type, got {dtype}")
    return _TORCH_TO_CODE[dtype]


def _z_mat(t, cols: int, storage, what: str, rows: int):
    """(type code, row distance) of a saved pre-activation, float32 or of the
    storage type."""
    if t.dtype is not torch.float32 and t.dtype is not storage:
        raise MoeError(f"{what}: need float32 or {storage}, got {t.dtype}")
    return _TORCH_TO_CODE[t.dtype], _mat(t, cols, t.dtype, what, rows)[1]


def _act_code(act: str, what: str) -> int:
    try:
        return ACTIVATIONS[act]
    except (KeyError, TypeError):
        raise MoeError(f"{what}: act must be one of {', '.join(ACTIVATIONS)}, got {act!r}") from None


def _any_code(x: int, w: int, y: int, rest: int) -> int:
    """The moe_any bits of a call: which addresses (of several matrices, their
    or) are no multiples of 16 bytes."""
    return (x & 15 and _ANY["x"]) | (w & 15 and _ANY["w"]) | (y & 15 and _ANY["y"]) | (rest & 15 and _ANY["rest"])


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the handle without building a Stream object, where torch has the call
# (1.9 us less on every call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(what: str, fn, args, first, *tensors):
    """fn(*args, stream) on the GPU of the call's tensors, in its current
    stream."""
    dev = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise MoeError(f"{what}: tensors on {first.device} and {t.device}")
    if dev < 0:
        raise MoeError(f"{what}: tensors must be on a GPU, got {first.device}")
    if dev == _current_device():
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status, what)


def _like(x: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of x's shape and type."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _flat(x: torch.Tensor, shape, strides, dtype) -> torch.Tensor:
    """A tensor beside x.  empty_strided is the fastest of torch's ways to one (with
    plain tuples, 1 us less than new_empty with a slice of x.shape)."""
    return torch.empty_strided(shape, strides, dtype=dtype, device=x.device)


def _new(x: torch.Tensor, cols: int, dtype) -> torch.Tensor:
    """A contiguous tensor of x's shape with `cols` columns."""
    if x.dim() == 2:
        return _flat(x, (x.shape[0], cols), (cols, 1), dtype)
    return x.new_empty(x.shape[:-1] + (cols,), dtype=dtype)


def moe_layernorm_workspace_size(rows: int, cols: int) -> int:
    """Workspace bytes of moe_layernorm_bwd."""
    n = ctypes.c_size_t()
    _check(load_library().moe_layernorm_workspace_size(rows, cols, ctypes.byref(n)), "moe_layernorm_workspace_size")
    return n.value


def moe_layernorm_fwd(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5, y=None, mean=None, rstd=None,
                      shuffle_seed: int = 0):
    """Layer norm of the rows of x [..., D] (float32 or bf16):
    y = (x - mean) rstd weight + bias.  Returns (y, mean, rstd), the last two
    float32 per row, as the backward reads them."""
    lib, what = load_library(), "moe_layernorm_fwd"
    code = _storage(x, what)
    if x.dim() == 0:
        raise MoeError(f"{what}: x needs a dimension to normalise")
    cols = x.shape[-1]
    rows, ldx = _mat(x, cols, x.dtype, what + " x")
    if not (0.0 <= eps < math.inf):
        raise MoeError(f"{what}: eps must be finite and not negative, got {eps}")
    if weight is not None:
        _need(weight, cols, x.dtype, what + " weight")
    if bias is not None:
        _need(bias, cols, x.dtype, what + " bias")
    if y is None:
        y = _like(x)
    else:
        _need(y, rows * cols, x.dtype, what + " y")
    if mean is None and rstd is None:
        mean = _flat(x, (rows,), (1,), torch.float32) if x.dim() == 2 else x.new_empty(x.shape[:-1], dtype=torch.float32)
        rstd = torch.empty_like(mean)
    elif mean is None or rstd is None:
        raise MoeError(f"{what}: mean and rstd are given together")
    else:
        _need(mean, rows, torch.float32, what + " mean")
        _need(rstd, rows, torch.float32, what + " rstd")
    _run(what, lib.moe_layernorm_fwd,
         (x.data_ptr(), _ptr(weight), _ptr(bias), code, rows, cols, ldx, eps, y.data_ptr(), mean.data_ptr(),
          rstd.data_ptr(), shuffle_seed), x, weight, bias, y, mean, rstd)
    return y, mean, rstd


def moe_layernorm_bwd(dy: torch.Tensor, x: torch.Tensor, weight, mean, rstd, dx_add=None, dx=None, dweight=None,
                      dbias=None, ws=None, shuffle_seed: int = 0):
    """Layer norm backward from the forward's x, weight, mean and rstd;
    dx_add [..., D] (another branch's gradient) is added to dx.  Returns
    (dx, dweight float32 [D], dbias float32 [D])."""
    lib, what = load_library(), "moe_layernorm_bwd"
    code = _storage(x, what)
    if x.dim() == 0:
        raise MoeError(f"{what}: x needs a dimension to normalise")
    cols = x.shape[-1]
    rows, ldx = _mat(x, cols, x.dtype, what + " x")
    _, lddy = _mat(dy, cols, x.dtype, what + " dy", rows)
    ldadd = _mat(dx_add, cols, x.dtype, what + " dx_add", rows)[1] if dx_add is not None else cols
    if weight is not None:
        _need(weight, cols, x.dtype, what + " weight")
    _need(mean, rows, torch.float32, what + " mean")
    _need(rstd, rows, torch.float32, what + " rstd")
    if dx is None:
        dx = _like(x)
    else:
        _need(dx, rows * cols, x.dtype, what + " dx")
    if dweight is None:
        dweight = _flat(x, (cols,), (1,), torch.float32)
    else:
        _need(dweight, cols, torch.float32, what + " dweight")
    if dbias is None:
        dbias = _flat(x, (cols,), (1,), torch.float32)
    else:
        _need(dbias, cols, torch.float32, what + " dbias")
    ws, nb = _dense_ws(_norm_ws(rows, cols), ws, x)
    _run(what, lib.moe_layernorm_bwd,
         (dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(), _ptr(dx_add), code, rows, cols,
          lddy, ldx, ldadd, dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr(), _ptr(ws), nb, shuffle_seed),
         x, dy, weight, mean, rstd, dx_add, dx, dweight, dbias, ws)
    return dx, dweight, dbias


_norm_ws = functools.lru_cache(maxsize=4096)(moe_layernorm_workspace_size)


def _ws_bytes(ws: torch.Tensor) -> int:
    if not ws.is_contiguous():
        raise MoeError("the workspace must be contiguous")
    return ws.numel() * ws.element_size()


@functools.lru_cache(maxsize=4096)
def _dense_plan(kind: str, rows: int, d_in: int, d_out: int, dtype: int, grad_dtype: int, z_dtype: int, act: int, ldx: int,
                ldw: int, ldy: int, ldz: int, ldr: int, seed: int):
    """The C description of a call (read-only) and its workspace sizes."""
    what = f"moe_{kind}_workspace_size"
    if max(rows, ldx, ldw, ldy, ldz, ldr) >= 1 << 31:
        raise MoeError(f"{what}: sizes beyond 2^31")
    c = _CDense(rows, d_in, d_out, dtype, grad_dtype, z_dtype, act, ldx, ldw, ldy, ldz, ldr, seed & 0xFFFFFFFFFFFFFFFF)
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(getattr(load_library(), what)(ctypes.byref(c), ctypes.byref(f), ctypes.byref(b)), what)
    return c, f.value, b.value


def _dense_key(what, rows, d_in, d_out, dtype, act, grad_dtype, ldx, ldw, ldy, unaligned):
    """_dense_plan's arguments after its first."""
    if grad_dtype is None:
        grad_dtype = dtype
    for t in (dtype, grad_dtype):
        if t not in ("f32", "bf16"):
            raise MoeError(f"{what}: dtypes are f32 and bf16, got {t!r}")
    a = _act_code(act, what)
    for n in unaligned:
        if n not in ("x", "w", "y"):
            raise MoeError(f"{what}: unaligned names x, w or y, got {n!r}")
        a |= _ANY[n]
    ld = [d if v is None else v for v, d in ((ldx, d_in), (ldw, d_out), (ldy, d_out))]
    return (rows, d_in, d_out, DTYPE_CODE[dtype], DTYPE_CODE[grad_dtype], 0, a, *ld, d_out, 0, 0)


def moe_linear_workspace_size(rows: int, d_in: int, d_out: int, dtype: str = "bf16", act: str = "none",
                              grad_dtype: Optional[str] = "f32", ldx: Optional[int] = None, ldw: Optional[int] = None,
                              ldy: Optional[int] = None, unaligned=()):
    """Bytes of workspace for (moe_linear_fwd, moe_linear_bwd): ldx, ldw and ldy
    the row distances of x, w and y (in the backward dy), where they are not
    contiguous; unaligned names those of "x", "w" and "y" whose address is not a
    multiple of 16 bytes."""
    return _dense_plan("linear", *_dense_key("moe_linear_workspace_size", rows, d_in, d_out, dtype, act, grad_dtype, ldx, ldw,
                                             ldy, unaligned))[1:]


def moe_glu_workspace_size(rows: int, d_in: int, d_out: int, dtype: str = "bf16", act: str = "silu",
                           grad_dtype: Optional[str] = "f32", ldx: Optional[int] = None, ldw: Optional[int] = None,
                           ldy: Optional[int] = None, unaligned=()):
    """Bytes of workspace for (moe_glu_fwd, moe_glu_bwd); ldx, ldw (of wg and wu),
    ldy (of a, in the backward da) and unaligned as in moe_linear_workspace_size."""
    return _dense_plan("glu", *_dense_key("moe_glu_workspace_size", rows, d_in, d_out, dtype, act, grad_dtype, ldx, ldw, ldy,
                                          unaligned))[1:]


def _dense_names(kind, call, *key):
    what = f"moe_{kind}_stage_names"
    b = ctypes.create_string_buffer(256)
    c = _dense_plan(kind, *_dense_key(what, *key))[0]
    _check(getattr(load_library(), what)(ctypes.byref(c), call, b, len(b)), what)
    return b.value.decode().split(",") if b.value else []


def moe_linear_stage_names(rows: int, d_in: int, d_out: int, call: int, dtype: str = "bf16", act: str = "none",
                           grad_dtype: Optional[str] = "f32", ldx: Optional[int] = None, ldw: Optional[int] = None,
                           ldy: Optional[int] = None, unaligned=()):
    """Names of the kernels that a call enqueues, with the tile and the number of
    chunks of each product: call 0 moe_linear_fwd, 1 moe_linear_bwd, 2 the same
    without db; the other arguments as in moe_linear_workspace_size."""
    return _dense_names("linear", call, rows, d_in, d_out, dtype, act, grad_dtype, ldx, ldw, ldy, unaligned)


def moe_glu_stage_names(rows: int, d_in: int, d_out: int, call: int, dtype: str = "bf16", act: str = "silu",
                        grad_dtype: Optional[str] = "f32", ldx: Optional[int] = None, ldw: Optional[int] = None,
                        ldy: Optional[int] = None, unaligned=()):
    """The same for moe_glu_fwd (call 0) and moe_glu_bwd (1)."""
    return _dense_names("glu", call, rows, d_in, d_out, dtype, act, grad_dtype, ldx, ldw, ldy, unaligned)


def _dense_ws(nbytes: int, ws, like):
    """(workspace or None, bytes) of a call."""
    if ws is not None:
        return ws, _ws_bytes(ws)
    if nbytes == 0:
        return None, 0
    return _flat(like, (nbytes,), (1,), torch.uint8), nbytes


def _dense_in(x, w, what: str):
    """Sizes of x [..., D] and w [D, F]."""
    code = _storage(x, what)
    if w.dim() != 2:
        raise MoeError(f"{what}: weights must be [d_in, d_out], got {tuple(w.shape)}")
    d, f = w.shape
    if d < 1 or f < 1:
        raise MoeError(f"{what}: weights without elements: {tuple(w.shape)}")
    rows, ldx = _mat(x, d, x.dtype, what + " x")
    ldw = _mat(w, f, x.dtype, what + " weight")[1]
    return code, rows, d, f, ldx, ldw


def moe_linear_fwd(x: torch.Tensor, w: torch.Tensor, bias=None, residual=None, act: str = "none", y=None, z=None,
                   save_z: bool = False, ws=None, shuffle_seed: int = 0):
    """y = act(x w + bias) + residual for x [..., D], w [D, F] (float32 or
    bf16), bias [F], residual [..., F].  Returns (y, z): z the
    pre-activation x w + bias for the backward, in the tensor given (float32 or
    x's type), with save_z in a new float32 one, else None.  y may be the
    residual itself."""
    lib, what = load_library(), "moe_linear_fwd"
    code, rows, d, f, ldx, ldw = _dense_in(x, w, what)
    a = _act_code(act, what)
    dt = x.dtype
    if bias is not None:
        _need(bias, f, dt, what + " bias")
    ldr = _mat(residual, f, dt, what + " residual", rows)[1] if residual is not None else 0
    if y is None:
        y, ldy = _new(x, f, dt), f
    else:
        ldy = _mat(y, f, dt, what + " y", rows)[1]
    zc, ldz = 0, f
    if z is not None:
        zc, ldz = _z_mat(z, f, dt, what + " z", rows)
    elif save_z:
        z = _new(x, f, torch.float32)
    px, pw, py, pr, pz = x.data_ptr(), w.data_ptr(), y.data_ptr(), _ptr(residual), _ptr(z)
    rest = (pr or 0) | (pz or 0)
    if (px | pw | py | rest) & 15:
        a |= _any_code(px, pw, py, rest)
    c, need, _ = _dense_plan("linear", rows, d, f, code, code, zc, a, ldx, ldw, ldy, ldz, ldr, shuffle_seed)
    ws, nb = _dense_ws(need, ws, x)
    _run(what, lib.moe_linear_fwd, (c, px, pw, _ptr(bias), pr, py, pz, _ptr(ws), nb), x, w, bias, residual, y, z, ws)
    return y, z


def moe_linear_bwd(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, z=None, act: str = "none", dx_add=None,
                   need_db: bool = True, grad_dtype=torch.float32, dx=None, dw=None, db=None, ws=None,
                   shuffle_seed: int = 0):
    """Backward of moe_linear_fwd from dy [..., F], its inputs and the saved z
    (unread with act "none"); dx_add [..., D] is added to dx.  The
    residual's gradient is dy.  Returns (dx, dw, db): the weight gradients in
    grad_dtype (float32 or the storage type), db None with need_db False."""
    lib, what = load_library(), "moe_linear_bwd"
    code, rows, d, f, ldx, ldw = _dense_in(x, w, what)
    a = _act_code(act, what)
    dt = x.dtype
    g = _grad_code(grad_dtype, dt, what)
    ldy = _mat(dy, f, dt, what + " dy", rows)[1]
    zc, ldz = 0, f
    if a:
        if z is None:
            raise MoeError(f"{what}: act {act!r} needs the saved z")
        zc, ldz = _z_mat(z, f, dt, what + " z", rows)
    else:
        z = None
    ldr = _mat(dx_add, d, dt, what + " dx_add", rows)[1] if dx_add is not None else 0
    if dx is None:
        dx = _like(x)
    else:
        _need(dx, rows * d, dt, what + " dx")
    if dw is None:
        dw = _flat(x, (d, f), (f, 1), grad_dtype)
    else:
        _need(dw, d * f, grad_dtype, what + " dw")
    if db is not None:
        _need(db, f, grad_dtype, what + " db")
    elif need_db:
        db = _flat(x, (f,), (1,), grad_dtype)
    py, px, pw, pz, pa, pdx, pdw = (dy.data_ptr(), x.data_ptr(), w.data_ptr(), _ptr(z), _ptr(dx_add), dx.data_ptr(),
                                    dw.data_ptr())
    rest = (pz or 0) | (pa or 0) | pdx | pdw
    if (px | pw | py | rest) & 15:
        a |= _any_code(px, pw, py, rest)
    c, _, need = _dense_plan("linear", rows, d, f, code, g, zc, a, ldx, ldw, ldy, ldz, ldr, shuffle_seed)
    ws, nb = _dense_ws(need, ws, x)
    _run(what, lib.moe_linear_bwd, (c, py, px, pw, pz, pa, pdx, pdw, _ptr(db), _ptr(ws), nb), x, dy, w, z, dx_add, dx, dw,
         db, ws)
    return dx, dw, db


def moe_glu_fwd(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, act: str = "silu", save: bool = False, a=None,
                g=None, u=None, ws=None, shuffle_seed: int = 0):
    """Gated feed-forward product a = act(x wg) * (x wu) for x [..., D], wg
    and wu [D, F] (two matrices, or the halves of one).  Returns (a, g, u): x wg
    and x wu for the backward in the tensors given (float32 or x's type), with
    save in new float32 ones, else None."""
    lib, what = load_library(), "moe_glu_fwd"
    code, rows, d, f, ldx, ldw = _dense_in(x, wg, what)
    ac = _act_code(act, what)
    dt = x.dtype
    if wu.dim() != 2 or _mat(wu, f, dt, what + " wu", d)[1] != ldw:
        raise MoeError(f"{what}: wg and wu need the same shape and row distance")
    if a is None:
        a, ldy = _new(x, f, dt), f
    else:
        ldy = _mat(a, f, dt, what + " a", rows)[1]
    if (g is None) != (u is None):
        raise MoeError(f"{what}: g and u are given together")
    zc, ldz = 0, f
    if g is not None:
        zc, ldz = _z_mat(g, f, dt, what + " g", rows)
        if _z_mat(u, f, dt, what + " u", rows) != (zc, ldz):
            raise MoeError(f"{what}: g and u need the same type and row distance")
    elif save:
        g = _new(x, f, torch.float32)
        u = _new(x, f, torch.float32)
    px, pg, pu, pa, zg, zu = x.data_ptr(), wg.data_ptr(), wu.data_ptr(), a.data_ptr(), _ptr(g), _ptr(u)
    rest = (zg or 0) | (zu or 0)
    if (px | pg | pu | pa | rest) & 15:
        ac |= _any_code(px, pg | pu, pa, rest)
    c, need, _ = _dense_plan("glu", rows, d, f, code, code, zc, ac, ldx, ldw, ldy, ldz, 0, shuffle_seed)
    ws, nb = _dense_ws(need, ws, x)
    _run(what, lib.moe_glu_fwd, (c, px, pg, pu, pa, zg, zu, _ptr(ws), nb), x, wg, wu, a, g, u, ws)
    return a, g, u


def moe_glu_bwd(da: torch.Tensor, x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, g: torch.Tensor, u: torch.Tensor,
                act: str = "silu", dx_add=None, grad_dtype=torch.float32, dx=None, dwg=None, dwu=None, ws=None,
                shuffle_seed: int = 0):
    """Backward of moe_glu_fwd from da [..., F], its inputs and the saved g
    and u; dx_add [..., D] is added to dx.  Returns (dx, dwg, dwu), the weight
    gradients in grad_dtype (float32 or the storage type)."""
    lib, what = load_library(), "moe_glu_bwd"
    code, rows, d, f, ldx, ldw = _dense_in(x, wg, what)
    ac = _act_code(act, what)
    dt = x.dtype
    gc = _grad_code(grad_dtype, dt, what)
    if wu.dim() != 2 or _mat(wu, f, dt, what + " wu", d)[1] != ldw:
        raise MoeError(f"{what}: wg and wu need the same shape and row distance")
    ldy = _mat(da, f, dt, what + " da", rows)[1]
    zc, ldz = _z_mat(g, f, dt, what + " g", rows)
    if _z_mat(u, f, dt, what + " u", rows) != (zc, ldz):
        raise MoeError(f"{what}: g and u need the same type and row distance")
    ldr = _mat(dx_add, d, dt, what + " dx_add", rows)[1] if dx_add is not None else 0
    if dx is None:
        dx = _like(x)
    else:
        _need(dx, rows * d, dt, what + " dx")
    if dwg is None:
        dwg = _flat(x, (d, f), (f, 1), grad_dtype)
    else:
        _need(dwg, d * f, grad_dtype, what + " dwg")
    if dwu is None:
        dwu = _flat(x, (d, f), (f, 1), grad_dtype)
    else:
        _need(dwu, d * f, grad_dtype, what + " dwu")
    py, px, pg, pu, zg, zu, pa = (da.data_ptr(), x.data_ptr(), wg.data_ptr(), wu.data_ptr(), g.data_ptr(), u.data_ptr(),
                                  _ptr(dx_add))
    pdx, dg, du = dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr()
    rest = zg | zu | (pa or 0) | pdx | dg | du
    if (px | pg | pu | py | rest) & 15:
        ac |= _any_code(px, pg | pu, py, rest)
    c, _, need = _dense_plan("glu", rows, d, f, code, gc, zc, ac, ldx, ldw, ldy, ldz, ldr, shuffle_seed)
    ws, nb = _dense_ws(need, ws, x)
    _run(what, lib.moe_glu_bwd, (c, py, px, pg, pu, zg, zu, pa, pdx, dg, du, _ptr(ws), nb), x, da, wg, wu, g, u, dx_add, dx,
         dwg, dwu, ws)
    return dx, dwg, dwu
