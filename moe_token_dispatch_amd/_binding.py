"""ctypes binding of the dispatch C ABI (``include/moe_dispatch.h``).

Argument marshalling only: every operator runs in the HIP kernels of
``libmoe_dispatch.so``. torch supplies device memory and the current stream.
The library must have been built (``python -m moe_token_dispatch_amd.build``);
loading fails loudly otherwise, and there is no fallback path.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional, Tuple

import torch  # load torch's HIP runtime first so the library binds to the same one

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_dispatch.so")

ABI_VERSION = 6
MAX_TOPK = 32
MAX_EXPERTS = 4096
MAX_RANKS = 1024

OK = 0
ERR_NULL = -1
ERR_ARG = -2
ERR_ALIGN = -3
ERR_WORKSPACE = -4
ERR_HIP = -5

STATUS_BAD_EXPERT = 1
STATUS_RECV_OVERFLOW = 2
STATUS_RANK_OVERFLOW = 4
STATUS_DUP_EXPERT = 8
STATUS_BAD_COUNT = 16
STATUS_TIMEOUT = 32
DEFAULT_WAIT_LIMIT = 1 << 20

RANK_CONTIG = 1
EXPERT_MAJOR = 2
ZERO_PAD = 4
ALL_OUTPUTS = RANK_CONTIG | EXPERT_MAJOR | ZERO_PAD
ROWS_READ_AHEAD = 8  # scatter hint: the rows were just read ahead (changes no result)

GATE_SOFTMAX = 0
GATE_SIGMOID = 1
GATE_NORMALIZE = 1
MAX_GATE_GROUPS = 64
MAX_NORM_WIDTH = 65536
SF_BLOCK = 128  # channels per scale factor


class DispatchError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {dispatch_strerror(code)} (code {code})")


class Problem(ctypes.Structure):
    """dispatch_problem_t."""

    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_topk", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("num_ranks", ctypes.c_int32),
        ("expert_alignment", ctypes.c_int32),
        ("topk_idx_bytes", ctypes.c_int32),
        ("sf_per_token", ctypes.c_int32),
        ("row_bytes", ctypes.c_int64),
        ("recv_capacity_rows", ctypes.c_int64),
        ("rank_capacity_rows", ctypes.c_int64),
        ("flags", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32),
    ]


class LayoutPtrs(ctypes.Structure):
    """dispatch_layout_t."""

    _fields_ = [(name, ctypes.c_void_p) for name in (
        "expert_count", "rank_count", "expert_psum", "rank_psum", "expert_slot", "rank_slot",
        "recv_src_token_idx", "rank_src_token_idx", "status", "expert_count_cumulative")]


class ExpandProblem(ctypes.Structure):
    """dispatch_expand_problem_t."""

    _fields_ = [
        ("num_sources", ctypes.c_int32),
        ("rows_per_source", ctypes.c_int32),
        ("num_topk", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("num_ranks", ctypes.c_int32),
        ("local_rank", ctypes.c_int32),
        ("expert_alignment", ctypes.c_int32),
        ("topk_idx_bytes", ctypes.c_int32),
        ("sf_per_token", ctypes.c_int32),
        ("reserved", ctypes.c_uint32),
        ("row_bytes", ctypes.c_int64),
        ("recv_capacity_rows", ctypes.c_int64),
    ]


class CombineProblem(ctypes.Structure):
    """dispatch_combine_problem_t."""

    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_topk", ctypes.c_int32),
        ("reserved", ctypes.c_uint32),
        ("hidden", ctypes.c_int64),
        ("expert_rows", ctypes.c_int64),
    ]


class GateProblem(ctypes.Structure):
    """dispatch_gate_problem_t."""

    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_experts", ctypes.c_int32),
        ("num_topk", ctypes.c_int32),
        ("scoring", ctypes.c_int32),
        ("logits_bytes", ctypes.c_int32),
        ("topk_idx_bytes", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("route_scale", ctypes.c_float),
        ("loss_coef", ctypes.c_float),
    ]


class GateGroups(ctypes.Structure):
    """dispatch_gate_groups_t."""

    _fields_ = [
        ("num_groups", ctypes.c_int32),
        ("topk_groups", ctypes.c_int32),
        ("score_experts", ctypes.c_int32),
        ("reserved", ctypes.c_uint32),
    ]


class GateOutPtrs(ctypes.Structure):
    """dispatch_gate_out_t."""

    _fields_ = [(name, ctypes.c_void_p) for name in (
        "topk_idx", "topk_weights", "expert_count", "prob_sum", "live_tokens", "loss")]


class QuantizeProblem(ctypes.Structure):
    """dispatch_quantize_problem_t."""

    _fields_ = [("num_rows", ctypes.c_int64), ("width", ctypes.c_int64)]


class RmsNormProblem(ctypes.Structure):
    """dispatch_rms_norm_problem_t."""

    _fields_ = [
        ("num_rows", ctypes.c_int64),
        ("width", ctypes.c_int64),
        ("weight_bytes", ctypes.c_int32),
        ("eps", ctypes.c_float),
    ]


class ExpertProblem(ctypes.Structure):
    """dispatch_expert_problem_t."""

    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("reserved", ctypes.c_uint32),
        ("in_features", ctypes.c_int64),
        ("out_features", ctypes.c_int64),
        ("expert_rows", ctypes.c_int64),
        ("max_routed_rows", ctypes.c_int64),
    ]


_LIB = None

# Exported symbols of include/moe_dispatch.h.
SYMBOLS = ("dispatch_abi_version", "dispatch_strerror", "dispatch_workspace_size",
           "dispatch_max_rows", "dispatch_layout", "dispatch_layout_read_ahead",
           "dispatch_scatter", "dispatch_layout_and_scatter", "dispatch_layout_and_scatter_noalloc",
           "dispatch_kernel_count", "dispatch_set_wait_limit",
           "dispatch_expand_workspace_size", "dispatch_expand_max_rows", "dispatch_expand_layout",
           "dispatch_expand_scatter", "dispatch_expand_layout_and_scatter", "dispatch_combine",
           "dispatch_gate_workspace_size", "dispatch_gate", "dispatch_gate_backward", "dispatch_quantize",
           "dispatch_swiglu_quantize", "dispatch_swiglu_backward_quantize", "dispatch_expert_workspace_size",
           "dispatch_expert_product", "dispatch_expert_product_swiglu", "dispatch_gate_grouped", "dispatch_rms_norm",
           "dispatch_rms_norm_workspace_size", "dispatch_rms_norm_backward", "dispatch_combine_backward")


def load_library(path: str = LIB_PATH):
    """Load libmoe_dispatch.so (built in-tree) and declare its signatures."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m moe_token_dispatch_amd.build`")
    lib = ctypes.CDLL(path)
    p, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.dispatch_abi_version.argtypes = []
    lib.dispatch_abi_version.restype = i
    lib.dispatch_strerror.argtypes = [i]
    lib.dispatch_strerror.restype = ctypes.c_char_p
    lib.dispatch_workspace_size.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(sz)]
    lib.dispatch_workspace_size.restype = i
    lib.dispatch_max_rows.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(ctypes.c_int64),
                                      ctypes.POINTER(ctypes.c_int64)]
    lib.dispatch_max_rows.restype = i
    lib.dispatch_layout.argtypes = [ctypes.POINTER(Problem), p, ctypes.POINTER(LayoutPtrs), p, sz, p]
    lib.dispatch_layout.restype = i
    lib.dispatch_layout_read_ahead.argtypes = [ctypes.POINTER(Problem), p, ctypes.POINTER(LayoutPtrs), p, sz, p, p,
                                               p]
    lib.dispatch_layout_read_ahead.restype = i
    lib.dispatch_scatter.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(LayoutPtrs), p, p, p, p, p, p, p]
    lib.dispatch_scatter.restype = i
    lib.dispatch_layout_and_scatter.argtypes = [ctypes.POINTER(Problem), p, ctypes.POINTER(LayoutPtrs), p, sz,
                                                p, p, p, p, p, p, p]
    lib.dispatch_layout_and_scatter.restype = i
    lib.dispatch_layout_and_scatter_noalloc.argtypes = [ctypes.POINTER(Problem), p, ctypes.POINTER(LayoutPtrs),
                                                        p, p, p, p, p, p, p]
    lib.dispatch_layout_and_scatter_noalloc.restype = i
    lib.dispatch_kernel_count.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(i), ctypes.POINTER(i)]
    lib.dispatch_kernel_count.restype = i
    lib.dispatch_set_wait_limit.argtypes = [ctypes.c_int64]
    lib.dispatch_set_wait_limit.restype = i
    ep = ctypes.POINTER(ExpandProblem)
    lib.dispatch_expand_workspace_size.argtypes = [ep, ctypes.POINTER(sz)]
    lib.dispatch_expand_workspace_size.restype = i
    lib.dispatch_expand_max_rows.argtypes = [ep, ctypes.POINTER(ctypes.c_int64)]
    lib.dispatch_expand_max_rows.restype = i
    lib.dispatch_expand_layout.argtypes = [ep, p, p, ctypes.POINTER(LayoutPtrs), p, sz, p]
    lib.dispatch_expand_layout.restype = i
    lib.dispatch_expand_scatter.argtypes = [ep, ctypes.POINTER(LayoutPtrs), p, p, p, p, p]
    lib.dispatch_expand_layout_and_scatter.argtypes = [ep, p, p, ctypes.POINTER(LayoutPtrs), p, sz, p, p, p, p, p]
    lib.dispatch_expand_layout_and_scatter.restype = i
    lib.dispatch_expand_scatter.restype = i
    lib.dispatch_combine.argtypes = [ctypes.POINTER(CombineProblem), p, p, p, p, p]
    lib.dispatch_combine.restype = i
    gp, qp, xp = ctypes.POINTER(GateProblem), ctypes.POINTER(QuantizeProblem), ctypes.POINTER(ExpertProblem)
    np = ctypes.POINTER(RmsNormProblem)
    for name, args in (("dispatch_gate_workspace_size", [gp, ctypes.POINTER(sz)]),
                       ("dispatch_gate", [gp, p, p, p, ctypes.POINTER(GateOutPtrs), p, sz, p]),
                       ("dispatch_gate_backward", [gp, p, p, p, p, p, p, p, p, p]),
                       ("dispatch_quantize", [qp, p, p, p, p, p]),
                       ("dispatch_swiglu_quantize", [qp, p, p, p, p, p]),
                       ("dispatch_swiglu_backward_quantize", [qp, p, p, p, p, p, p]),
                       ("dispatch_expert_workspace_size", [xp, ctypes.POINTER(sz)]),
                       ("dispatch_expert_product", [xp, p, p, p, p, p, p, p, p, sz, p]),
                       ("dispatch_expert_product_swiglu", [xp, p, p, p, p, p, p, p, p, p, sz, p]),
                       ("dispatch_gate_grouped", [gp, ctypes.POINTER(GateGroups), p, p, p, ctypes.POINTER(GateOutPtrs),
                                                  p, sz, p]),
                       ("dispatch_rms_norm", [np, p, p, p, p, p, p, p, p, p]),
                       ("dispatch_rms_norm_workspace_size", [np, ctypes.POINTER(sz)]),
                       ("dispatch_rms_norm_backward", [np, p, p, p, p, p, p, p, p, sz, p]),
                       ("dispatch_combine_backward", [ctypes.POINTER(CombineProblem), p, p, p, p, p, p, p, p, p])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i
    if lib.dispatch_abi_version() != ABI_VERSION:
        raise ImportError(f"{path}: ABI version {lib.dispatch_abi_version()} != {ABI_VERSION}")
    _LIB = lib
    return lib


# ---------------------------------------------------------------- C ABI calls


def dispatch_abi_version() -> int:
    return load_library().dispatch_abi_version()


def dispatch_strerror(code: int) -> str:
    return load_library().dispatch_strerror(code).decode()


def dispatch_workspace_size(problem: Problem) -> int:
    out = ctypes.c_size_t(0)
    rc = load_library().dispatch_workspace_size(ctypes.byref(problem), ctypes.byref(out))
    if rc:
        raise DispatchError(rc, "dispatch_workspace_size")
    return int(out.value)


def dispatch_max_rows(problem: Problem) -> Tuple[int, int]:
    recv, rank = ctypes.c_int64(0), ctypes.c_int64(0)
    rc = load_library().dispatch_max_rows(ctypes.byref(problem), ctypes.byref(recv), ctypes.byref(rank))
    if rc:
        raise DispatchError(rc, "dispatch_max_rows")
    return int(recv.value), int(rank.value)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream: Optional[torch.cuda.Stream], device) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


@dataclasses.dataclass
class LayoutTensors:
    """Device int32 outputs of dispatch_layout (see dispatch_layout_t)."""

    expert_count: torch.Tensor
    rank_count: torch.Tensor
    expert_psum: torch.Tensor
    rank_psum: torch.Tensor
    expert_slot: torch.Tensor
    rank_slot: torch.Tensor
    recv_src_token_idx: torch.Tensor
    rank_src_token_idx: torch.Tensor
    status: torch.Tensor

    def ptrs(self, expert_count_cumulative: Optional[torch.Tensor] = None) -> LayoutPtrs:
        return LayoutPtrs(*[t.data_ptr() for t in (
            self.expert_count, self.rank_count, self.expert_psum, self.rank_psum, self.expert_slot,
            self.rank_slot, self.recv_src_token_idx, self.rank_src_token_idx, self.status)],
            _ptr(expert_count_cumulative))

    def tensors(self):
        """(name, tensor) of every output present."""
        return [(f.name, getattr(self, f.name)) for f in dataclasses.fields(self) if getattr(self, f.name) is not None]


def _fields_of(layout):
    """(name, tensor) of every layout output present (optional ones may be None)."""
    return [(f.name, getattr(layout, f.name)) for f in dataclasses.fields(layout) if getattr(layout, f.name) is not None]


def _check_device_tensor(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _check_cumulative(t: Optional[torch.Tensor], num_experts: int) -> None:
    if t is not None:
        _check_device_tensor(t, "expert_count_cumulative", torch.int32)
        if t.numel() < num_experts:
            raise ValueError(f"expert_count_cumulative needs {num_experts} entries, has {t.numel()}")


# The C ABI takes raw pointers and trusts their sizes; the binding knows every
# size from the problem and refuses a tensor too small for it, before any call.
def _need(t: Optional[torch.Tensor], name: str, nbytes: int) -> None:
    if t is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes; the problem needs {nbytes}")


def _check_dispatch_sizes(problem: Problem, topk_idx: Optional[torch.Tensor], layout: "LayoutTensors") -> None:
    t, k, e, r = problem.num_tokens, problem.num_topk, problem.num_experts, problem.num_ranks
    _need(topk_idx, "topk_idx", t * k * problem.topk_idx_bytes)
    for name, n in (("expert_count", e), ("rank_count", r), ("expert_psum", e + 1), ("rank_psum", r + 1),
                    ("expert_slot", t * k), ("rank_slot", t * k),
                    ("recv_src_token_idx", problem.recv_capacity_rows),
                    ("rank_src_token_idx", problem.rank_capacity_rows), ("status", 1)):
        _need(getattr(layout, name), name, 4 * n)


def _check_dispatch_rows(problem: Problem, x, x_sf, rank_x, rank_sf, recv_x, recv_sf) -> None:
    t, rb, s = problem.num_tokens, problem.row_bytes, problem.sf_per_token
    _need(x, "x", t * rb)
    _need(x_sf, "x_sf", 4 * t * s)
    if problem.flags & RANK_CONTIG:
        _need(rank_x, "rank_x", problem.rank_capacity_rows * rb)
        _need(rank_sf, "rank_sf", 4 * problem.rank_capacity_rows * s)
    if problem.flags & EXPERT_MAJOR:
        _need(recv_x, "recv_x", problem.recv_capacity_rows * rb)
        _need(recv_sf, "recv_sf", 4 * problem.recv_capacity_rows * s)


def _check_expand_sizes(problem: "ExpandProblem", recv_topk_idx, recv_count, layout, recv_buf, recv_sf_buf,
                        recv_x, recv_sf) -> None:
    rows = problem.num_sources * problem.rows_per_source
    local = problem.num_experts // problem.num_ranks
    cap, rb, s = problem.recv_capacity_rows, problem.row_bytes, problem.sf_per_token
    _need(recv_topk_idx, "recv_topk_idx", rows * problem.num_topk * problem.topk_idx_bytes)
    _need(recv_count, "recv_count", 4 * problem.num_sources)
    if layout is not None:
        for name, n in (("expert_count", local), ("expert_psum", local + 1), ("expert_slot", rows * problem.num_topk),
                        ("recv_src_row_idx", cap), ("status", 1)):
            _need(getattr(layout, name), name, 4 * n)
    _need(recv_buf, "recv_buf", rows * rb)
    _need(recv_sf_buf, "recv_sf_buf", 4 * rows * s)
    _need(recv_x, "recv_x", cap * rb)
    _need(recv_sf, "recv_sf", 4 * cap * s)


def dispatch_layout(problem: Problem, topk_idx: torch.Tensor, out: LayoutTensors,
                    workspace: torch.Tensor, stream: Optional[torch.cuda.Stream] = None,
                    expert_count_cumulative: Optional[torch.Tensor] = None) -> None:
    """Enqueue Count -> Prefix Sum -> slot assignment on the stream. When
    ``expert_count_cumulative`` (device int32 [E], kept by the caller) is given,
    a successful call adds its expert_count to it."""
    _check_device_tensor(topk_idx, "topk_idx")
    if topk_idx.element_size() != problem.topk_idx_bytes:
        raise ValueError("topk_idx element width does not match problem.topk_idx_bytes")
    _check_device_tensor(workspace, "workspace")
    for name, t in _fields_of(out):
        _check_device_tensor(t, name, torch.int32)
    _check_cumulative(expert_count_cumulative, problem.num_experts)
    _check_dispatch_sizes(problem, topk_idx, out)
    lay = out.ptrs(expert_count_cumulative)
    rc = load_library().dispatch_layout(ctypes.byref(problem), _ptr(topk_idx), ctypes.byref(lay),
                                        _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream_handle(stream, topk_idx.device))
    if rc:
        raise DispatchError(rc, "dispatch_layout")


def dispatch_layout_read_ahead(problem: Problem, topk_idx: torch.Tensor, out: LayoutTensors,
                               workspace: torch.Tensor, x: torch.Tensor, x_sf: Optional[torch.Tensor] = None,
                               stream: Optional[torch.cuda.Stream] = None,
                               expert_count_cumulative: Optional[torch.Tensor] = None) -> None:
    """dispatch_layout, reading the token rows ``x`` (and ``x_sf``) into the
    Infinity Cache while it runs, for a dispatch_scatter of them that follows."""
    _check_device_tensor(topk_idx, "topk_idx")
    if topk_idx.element_size() != problem.topk_idx_bytes:
        raise ValueError("topk_idx element width does not match problem.topk_idx_bytes")
    _check_device_tensor(workspace, "workspace")
    _check_device_tensor(x, "x")
    if x_sf is not None:
        _check_device_tensor(x_sf, "x_sf")
    for name, t in _fields_of(out):
        _check_device_tensor(t, name, torch.int32)
    _check_cumulative(expert_count_cumulative, problem.num_experts)
    _check_dispatch_sizes(problem, topk_idx, out)
    _need(x, "x", problem.num_tokens * problem.row_bytes)
    _need(x_sf, "x_sf", 4 * problem.num_tokens * problem.sf_per_token)
    lay = out.ptrs(expert_count_cumulative)
    rc = load_library().dispatch_layout_read_ahead(ctypes.byref(problem), _ptr(topk_idx), ctypes.byref(lay),
                                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                   _ptr(x), _ptr(x_sf), _stream_handle(stream, topk_idx.device))
    if rc:
        raise DispatchError(rc, "dispatch_layout_read_ahead")


def dispatch_scatter(problem: Problem, layout: LayoutTensors, x: torch.Tensor,
                     x_sf: Optional[torch.Tensor], rank_x: Optional[torch.Tensor],
                     rank_sf: Optional[torch.Tensor], recv_x: Optional[torch.Tensor],
                     recv_sf: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue the row scatter of a layout on the stream."""
    _check_device_tensor(x, "x")
    for name, t in (("x_sf", x_sf), ("rank_x", rank_x), ("rank_sf", rank_sf), ("recv_x", recv_x),
                    ("recv_sf", recv_sf)):
        if t is not None:
            _check_device_tensor(t, name)
    for name, t in _fields_of(layout):
        _check_device_tensor(t, name, torch.int32)
    _check_dispatch_sizes(problem, None, layout)
    _check_dispatch_rows(problem, x, x_sf, rank_x, rank_sf, recv_x, recv_sf)
    lay = layout.ptrs()
    rc = load_library().dispatch_scatter(ctypes.byref(problem), ctypes.byref(lay), _ptr(x), _ptr(x_sf),
                                         _ptr(rank_x), _ptr(rank_sf), _ptr(recv_x), _ptr(recv_sf),
                                         _stream_handle(stream, x.device))
    if rc:
        raise DispatchError(rc, "dispatch_scatter")


def dispatch_kernel_count(problem: Problem) -> tuple:
    """(kernels of dispatch_layout, kernels of dispatch_layout_and_scatter) for this problem."""
    lay, both = ctypes.c_int(0), ctypes.c_int(0)
    rc = load_library().dispatch_kernel_count(ctypes.byref(problem), ctypes.byref(lay), ctypes.byref(both))
    if rc:
        raise DispatchError(rc, "dispatch_kernel_count")
    return lay.value, both.value


def dispatch_set_wait_limit(polls: int) -> None:
    """Bound the one-launch layout's in-kernel wait to `polls` polls (0: the default); process-wide."""
    rc = load_library().dispatch_set_wait_limit(int(polls))
    if rc:
        raise DispatchError(rc, "dispatch_set_wait_limit")


def dispatch_layout_and_scatter(problem: Problem, topk_idx: torch.Tensor, out: LayoutTensors,
                                workspace: torch.Tensor, x: torch.Tensor, x_sf: Optional[torch.Tensor],
                                rank_x: Optional[torch.Tensor], rank_sf: Optional[torch.Tensor],
                                recv_x: Optional[torch.Tensor], recv_sf: Optional[torch.Tensor],
                                stream: Optional[torch.cuda.Stream] = None,
                                expert_count_cumulative: Optional[torch.Tensor] = None) -> None:
    """Enqueue dispatch_layout then dispatch_scatter as one call (one kernel
    for a batch that fits one layout tile)."""
    _check_device_tensor(topk_idx, "topk_idx")
    if topk_idx.element_size() != problem.topk_idx_bytes:
        raise ValueError("topk_idx element width does not match problem.topk_idx_bytes")
    _check_device_tensor(workspace, "workspace")
    for name, t in _fields_of(out):
        _check_device_tensor(t, name, torch.int32)
    _check_cumulative(expert_count_cumulative, problem.num_experts)
    _check_device_tensor(x, "x")
    for name, t in (("x_sf", x_sf), ("rank_x", rank_x), ("rank_sf", rank_sf), ("recv_x", recv_x),
                    ("recv_sf", recv_sf)):
        if t is not None:
            _check_device_tensor(t, name)
    _check_dispatch_sizes(problem, topk_idx, out)
    _check_dispatch_rows(problem, x, x_sf, rank_x, rank_sf, recv_x, recv_sf)
    lay = out.ptrs(expert_count_cumulative)
    rc = load_library().dispatch_layout_and_scatter(
        ctypes.byref(problem), _ptr(topk_idx), ctypes.byref(lay), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(x), _ptr(x_sf), _ptr(rank_x), _ptr(rank_sf),
        _ptr(recv_x), _ptr(recv_sf), _stream_handle(stream, topk_idx.device))
    if rc:
        raise DispatchError(rc, "dispatch_layout_and_scatter")


def dispatch_layout_and_scatter_noalloc(problem: Problem, topk_idx: torch.Tensor, out: LayoutTensors,
                                        x: torch.Tensor, x_sf: Optional[torch.Tensor],
                                        rank_x: Optional[torch.Tensor], rank_sf: Optional[torch.Tensor],
                                        recv_x: Optional[torch.Tensor], recv_sf: Optional[torch.Tensor],
                                        stream: Optional[torch.cuda.Stream] = None,
                                        expert_count_cumulative: Optional[torch.Tensor] = None) -> None:
    """dispatch_layout_and_scatter with the library's own fixed workspace (no
    workspace argument, nothing allocated). Calls that overlap on one GPU race."""
    _check_device_tensor(topk_idx, "topk_idx")
    if topk_idx.element_size() != problem.topk_idx_bytes:
        raise ValueError("topk_idx element width does not match problem.topk_idx_bytes")
    for name, t in _fields_of(out):
        _check_device_tensor(t, name, torch.int32)
    _check_cumulative(expert_count_cumulative, problem.num_experts)
    _check_device_tensor(x, "x")
    for name, t in (("x_sf", x_sf), ("rank_x", rank_x), ("rank_sf", rank_sf), ("recv_x", recv_x),
                    ("recv_sf", recv_sf)):
        if t is not None:
            _check_device_tensor(t, name)
    _check_dispatch_sizes(problem, topk_idx, out)
    _check_dispatch_rows(problem, x, x_sf, rank_x, rank_sf, recv_x, recv_sf)
    lay = out.ptrs(expert_count_cumulative)
    rc = load_library().dispatch_layout_and_scatter_noalloc(
        ctypes.byref(problem), _ptr(topk_idx), ctypes.byref(lay), _ptr(x), _ptr(x_sf), _ptr(rank_x),
        _ptr(rank_sf), _ptr(recv_x), _ptr(recv_sf), _stream_handle(stream, topk_idx.device))
    if rc:
        raise DispatchError(rc, "dispatch_layout_and_scatter_noalloc")


# ------------------------------------------------- allocation helpers (plumbing)


def make_problem(num_tokens: int, num_topk: int, num_experts: int, num_ranks: int,
                 expert_alignment: int = 1, topk_idx_bytes: int = 8, row_bytes: int = 0,
                 sf_per_token: int = 0, recv_capacity_rows: Optional[int] = None,
                 rank_capacity_rows: Optional[int] = None, flags: int = ALL_OUTPUTS) -> Problem:
    """A problem; capacities default to the library's worst-case row counts."""
    p = Problem(num_tokens, num_topk, num_experts, num_ranks, expert_alignment, topk_idx_bytes,
                sf_per_token, row_bytes, 0, 0, flags, 0)
    max_recv, max_rank = dispatch_max_rows(p)
    p.recv_capacity_rows = max_recv if recv_capacity_rows is None else recv_capacity_rows
    p.rank_capacity_rows = max_rank if rank_capacity_rows is None else rank_capacity_rows
    return p


def alloc_layout(problem: Problem, device) -> LayoutTensors:
    i32 = dict(dtype=torch.int32, device=device)
    t, k = problem.num_tokens, problem.num_topk
    return LayoutTensors(
        expert_count=torch.empty(problem.num_experts, **i32),
        rank_count=torch.empty(problem.num_ranks, **i32),
        expert_psum=torch.empty(problem.num_experts + 1, **i32),
        rank_psum=torch.empty(problem.num_ranks + 1, **i32),
        expert_slot=torch.empty((t, k), **i32),
        rank_slot=torch.empty((t, k), **i32),
        recv_src_token_idx=torch.empty(max(problem.recv_capacity_rows, 1), **i32),
        rank_src_token_idx=torch.empty(max(problem.rank_capacity_rows, 1), **i32),
        status=torch.empty(1, **i32))


def alloc_workspace(problem: Problem, device) -> torch.Tensor:
    """Workspace for the layout calls: zero-filled, as its first use requires (torch allocations are
    256-byte aligned)."""
    n = dispatch_workspace_size(problem)
    return torch.zeros((n + 255) // 256 * 256, dtype=torch.uint8, device=device)


@dataclasses.dataclass
class RowBuffers:
    rank_x: Optional[torch.Tensor]   # uint8 [rank_capacity_rows, row_bytes]
    rank_sf: Optional[torch.Tensor]  # float32 [rank_capacity_rows, S]
    recv_x: Optional[torch.Tensor]   # uint8 [recv_capacity_rows, row_bytes]
    recv_sf: Optional[torch.Tensor]  # float32 [recv_capacity_rows, S]


def alloc_rows(problem: Problem, device) -> RowBuffers:
    rb, s = problem.row_bytes, problem.sf_per_token
    want_rank = bool(problem.flags & RANK_CONTIG)
    want_expert = bool(problem.flags & EXPERT_MAJOR)

    def rows(n, width, dtype, on):
        return torch.empty((max(n, 1), width), dtype=dtype, device=device) if on and width > 0 else None

    return RowBuffers(rank_x=rows(problem.rank_capacity_rows, rb, torch.uint8, want_rank),
                      rank_sf=rows(problem.rank_capacity_rows, s, torch.float32, want_rank),
                      recv_x=rows(problem.recv_capacity_rows, rb, torch.uint8, want_expert),
                      recv_sf=rows(problem.recv_capacity_rows, s, torch.float32, want_expert))


class Plan:
    """A prepared dispatch: the problem, the tensors and the stream are checked
    once and the C arguments are built once, so each call is a single C call.

    ``layout()`` enqueues dispatch_layout, ``scatter()`` enqueues
    dispatch_scatter, ``__call__`` enqueues both as one
    dispatch_layout_and_scatter call; ``layout_read_ahead()`` followed by
    ``scatter(read_ahead=True)`` is that call's two halves. The tensors must stay alive and keep
    their storage while the plan is used.
    """

    def __init__(self, problem: Problem, topk_idx: torch.Tensor, layout: LayoutTensors,
                 workspace: torch.Tensor, x: Optional[torch.Tensor] = None,
                 x_sf: Optional[torch.Tensor] = None, rows: Optional[RowBuffers] = None,
                 stream: Optional[torch.cuda.Stream] = None,
                 expert_count_cumulative: Optional[torch.Tensor] = None):
        _check_device_tensor(topk_idx, "topk_idx")
        if topk_idx.element_size() != problem.topk_idx_bytes:
            raise ValueError("topk_idx element width does not match problem.topk_idx_bytes")
        _check_device_tensor(workspace, "workspace")
        for name, t in _fields_of(layout):
            _check_device_tensor(t, name, torch.int32)
        _check_cumulative(expert_count_cumulative, problem.num_experts)
        _check_dispatch_sizes(problem, topk_idx, layout)
        # The plan keeps its own copy of the problem: the tensor sizes were
        # checked against these values, and a later change to the caller's
        # struct must not reach the C calls.
        problem = Problem.from_buffer_copy(problem)
        self._problem = problem
        self._lib = load_library()
        self._keep = (problem, topk_idx, layout, workspace, x, x_sf, rows, expert_count_cumulative)
        self._lay = layout.ptrs(expert_count_cumulative)
        handle = _stream_handle(stream, topk_idx.device)
        self._layout_args = (ctypes.byref(problem), _ptr(topk_idx), ctypes.byref(self._lay), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), handle)
        self._scatter_args = self._scatter_ra_args = self._both_args = self._layout_ra_args = None
        if x is not None:
            _check_device_tensor(x, "x")
            rows = rows if rows is not None else RowBuffers(None, None, None, None)
            for name in ("rank_x", "rank_sf", "recv_x", "recv_sf"):
                t = getattr(rows, name)
                if t is not None:
                    _check_device_tensor(t, name)
            if x_sf is not None:
                _check_device_tensor(x_sf, "x_sf")
            _check_dispatch_rows(problem, x, x_sf, rows.rank_x, rows.rank_sf, rows.recv_x, rows.recv_sf)
            row_ptrs = (_ptr(x), _ptr(x_sf), _ptr(rows.rank_x), _ptr(rows.rank_sf), _ptr(rows.recv_x),
                        _ptr(rows.recv_sf))
            self._scatter_args = (ctypes.byref(problem), ctypes.byref(self._lay), *row_ptrs, handle)
            # The same problem with the read-ahead hint, for the scatter that
            # follows layout_read_ahead().
            ra_problem = Problem.from_buffer_copy(problem)
            ra_problem.flags |= ROWS_READ_AHEAD
            self._keep += (ra_problem,)
            self._scatter_ra_args = (ctypes.byref(ra_problem), *self._scatter_args[1:])
            self._both_args = (*self._layout_args[:-1], *row_ptrs, handle)
            self._layout_ra_args = (*self._layout_args[:-1], _ptr(x), _ptr(x_sf), handle)

    def layout(self) -> None:
        rc = self._lib.dispatch_layout(*self._layout_args)
        if rc:
            raise DispatchError(rc, "dispatch_layout")

    def layout_read_ahead(self) -> None:
        """dispatch_layout_read_ahead: the layout, reading the plan's token rows
        into the Infinity Cache for the scatter that follows."""
        if self._layout_ra_args is None:
            raise ValueError("this plan has no token batch to read ahead")
        rc = self._lib.dispatch_layout_read_ahead(*self._layout_ra_args)
        if rc:
            raise DispatchError(rc, "dispatch_layout_read_ahead")

    def scatter(self, read_ahead: bool = False) -> None:
        """dispatch_scatter; ``read_ahead``: right after layout_read_ahead()
        (sets DISPATCH_ROWS_READ_AHEAD)."""
        if self._scatter_args is None:
            raise ValueError("this plan has no token batch to scatter")
        rc = self._lib.dispatch_scatter(*(self._scatter_ra_args if read_ahead else self._scatter_args))
        if rc:
            raise DispatchError(rc, "dispatch_scatter")

    def __call__(self) -> None:
        if self._scatter_args is None:
            raise ValueError("this plan has no token batch to scatter")
        rc = self._lib.dispatch_layout_and_scatter(*self._both_args)
        if rc:
            raise DispatchError(rc, "dispatch_layout_and_scatter")


# ------------------------------------------------------------ receiver-side expand


def make_expand_problem(num_sources: int, rows_per_source: int, num_topk: int, num_experts: int,
                        num_ranks: int, local_rank: int, expert_alignment: int = 1, topk_idx_bytes: int = 8,
                        row_bytes: int = 16, sf_per_token: int = 0,
                        recv_capacity_rows: Optional[int] = None) -> ExpandProblem:
    """An expand problem; the capacity defaults to the library's worst case."""
    q = ExpandProblem(num_sources, rows_per_source, num_topk, num_experts, num_ranks, local_rank,
                      expert_alignment, topk_idx_bytes, sf_per_token, 0, row_bytes, 0)
    cap = ctypes.c_int64(0)
    rc = load_library().dispatch_expand_max_rows(ctypes.byref(q), ctypes.byref(cap))
    if rc:
        raise DispatchError(rc, "dispatch_expand_max_rows")
    q.recv_capacity_rows = int(cap.value) if recv_capacity_rows is None else recv_capacity_rows
    return q


def dispatch_expand_workspace_size(problem: ExpandProblem) -> int:
    out = ctypes.c_size_t(0)
    rc = load_library().dispatch_expand_workspace_size(ctypes.byref(problem), ctypes.byref(out))
    if rc:
        raise DispatchError(rc, "dispatch_expand_workspace_size")
    return int(out.value)


@dataclasses.dataclass
class ExpandLayoutTensors:
    """Device int32 outputs of dispatch_expand_layout."""

    expert_count: torch.Tensor        # [E/R]
    expert_psum: torch.Tensor         # [E/R + 1]
    expert_slot: torch.Tensor         # [S*M, K]
    recv_src_row_idx: torch.Tensor    # [recv_capacity_rows]
    status: torch.Tensor              # [1]

    def ptrs(self, expert_count_cumulative: Optional[torch.Tensor] = None) -> LayoutPtrs:
        return LayoutPtrs(self.expert_count.data_ptr(), None, self.expert_psum.data_ptr(), None,
                          self.expert_slot.data_ptr(), None, self.recv_src_row_idx.data_ptr(), None,
                          self.status.data_ptr(), _ptr(expert_count_cumulative))


def alloc_expand_layout(problem: ExpandProblem, device) -> ExpandLayoutTensors:
    i32 = dict(dtype=torch.int32, device=device)
    local = problem.num_experts // problem.num_ranks
    rows = problem.num_sources * problem.rows_per_source
    return ExpandLayoutTensors(
        expert_count=torch.empty(local, **i32), expert_psum=torch.empty(local + 1, **i32),
        expert_slot=torch.empty((rows, problem.num_topk), **i32),
        recv_src_row_idx=torch.empty(max(problem.recv_capacity_rows, 1), **i32),
        status=torch.empty(1, **i32))


def alloc_expand_workspace(problem: ExpandProblem, device) -> torch.Tensor:
    """Workspace for the expand layout calls: zero-filled, as its first use requires."""
    n = dispatch_expand_workspace_size(problem)
    return torch.zeros((n + 255) // 256 * 256, dtype=torch.uint8, device=device)


def dispatch_expand_layout(problem: ExpandProblem, recv_topk_idx: torch.Tensor, recv_count: torch.Tensor,
                           out: ExpandLayoutTensors, workspace: torch.Tensor,
                           stream: Optional[torch.cuda.Stream] = None,
                           expert_count_cumulative: Optional[torch.Tensor] = None) -> None:
    """Enqueue the receiver's expert-major layout of a receive buffer. When
    ``expert_count_cumulative`` (device int32 [E/R], kept by the caller) is
    given, a successful call adds the local experts' received rows to it."""
    _check_device_tensor(recv_topk_idx, "recv_topk_idx")
    if recv_topk_idx.element_size() != problem.topk_idx_bytes:
        raise ValueError("recv_topk_idx element width does not match problem.topk_idx_bytes")
    _check_device_tensor(recv_count, "recv_count", torch.int32)
    _check_device_tensor(workspace, "workspace")
    for name, t in _fields_of(out):
        _check_device_tensor(t, name, torch.int32)
    _check_cumulative(expert_count_cumulative, problem.num_experts // problem.num_ranks)
    _check_expand_sizes(problem, recv_topk_idx, recv_count, out, None, None, None, None)
    lay = out.ptrs(expert_count_cumulative)
    rc = load_library().dispatch_expand_layout(
        ctypes.byref(problem), _ptr(recv_topk_idx), _ptr(recv_count), ctypes.byref(lay), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream_handle(stream, recv_topk_idx.device))
    if rc:
        raise DispatchError(rc, "dispatch_expand_layout")


def dispatch_expand_layout_and_scatter(problem: ExpandProblem, recv_topk_idx: torch.Tensor,
                                       recv_count: torch.Tensor, out: ExpandLayoutTensors, workspace: torch.Tensor,
                                       recv_buf: torch.Tensor, recv_sf_buf: Optional[torch.Tensor],
                                       recv_x: torch.Tensor, recv_sf: Optional[torch.Tensor],
                                       stream: Optional[torch.cuda.Stream] = None,
                                       expert_count_cumulative: Optional[torch.Tensor] = None) -> None:
    """Enqueue dispatch_expand_layout then dispatch_expand_scatter as one call
    (one kernel for a small receive buffer)."""
    _check_device_tensor(recv_topk_idx, "recv_topk_idx")
    if recv_topk_idx.element_size() != problem.topk_idx_bytes:
        raise ValueError("recv_topk_idx element width does not match problem.topk_idx_bytes")
    _check_device_tensor(recv_count, "recv_count", torch.int32)
    _check_device_tensor(workspace, "workspace")
    for name, t in _fields_of(out):
        _check_device_tensor(t, name, torch.int32)
    _check_cumulative(expert_count_cumulative, problem.num_experts // problem.num_ranks)
    _check_device_tensor(recv_buf, "recv_buf")
    for name, t in (("recv_sf_buf", recv_sf_buf), ("recv_x", recv_x), ("recv_sf", recv_sf)):
        if t is not None:
            _check_device_tensor(t, name)
    _check_expand_sizes(problem, recv_topk_idx, recv_count, out, recv_buf, recv_sf_buf, recv_x, recv_sf)
    lay = out.ptrs(expert_count_cumulative)
    rc = load_library().dispatch_expand_layout_and_scatter(
        ctypes.byref(problem), _ptr(recv_topk_idx), _ptr(recv_count), ctypes.byref(lay), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(recv_buf), _ptr(recv_sf_buf), _ptr(recv_x), _ptr(recv_sf),
        _stream_handle(stream, recv_topk_idx.device))
    if rc:
        raise DispatchError(rc, "dispatch_expand_layout_and_scatter")


def dispatch_expand_scatter(problem: ExpandProblem, layout: ExpandLayoutTensors, recv_buf: torch.Tensor,
                            recv_sf_buf: Optional[torch.Tensor], recv_x: torch.Tensor,
                            recv_sf: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue the copy of received rows into the expert-major buffer."""
    _check_device_tensor(recv_buf, "recv_buf")
    for name, t in (("recv_sf_buf", recv_sf_buf), ("recv_x", recv_x), ("recv_sf", recv_sf)):
        if t is not None:
            _check_device_tensor(t, name)
    for name, t in _fields_of(layout):
        _check_device_tensor(t, name, torch.int32)
    _check_expand_sizes(problem, None, None, layout, recv_buf, recv_sf_buf, recv_x, recv_sf)
    lay = layout.ptrs()
    rc = load_library().dispatch_expand_scatter(ctypes.byref(problem), ctypes.byref(lay), _ptr(recv_buf),
                                                _ptr(recv_sf_buf), _ptr(recv_x), _ptr(recv_sf),
                                                _stream_handle(stream, recv_buf.device))
    if rc:
        raise DispatchError(rc, "dispatch_expand_scatter")


class ExpandPlan:
    """A prepared receiver-side expand, like Plan: the tensors and the stream
    are checked once and the C arguments built once. ``layout()`` enqueues
    dispatch_expand_layout, ``scatter()`` dispatch_expand_scatter and
    ``__call__`` both as one dispatch_expand_layout_and_scatter call."""

    def __init__(self, problem: ExpandProblem, recv_topk_idx: torch.Tensor, recv_count: torch.Tensor,
                 layout: ExpandLayoutTensors, workspace: torch.Tensor, recv_buf: torch.Tensor,
                 recv_sf_buf: Optional[torch.Tensor], recv_x: torch.Tensor, recv_sf: Optional[torch.Tensor],
                 stream: Optional[torch.cuda.Stream] = None,
                 expert_count_cumulative: Optional[torch.Tensor] = None):
        _check_device_tensor(recv_topk_idx, "recv_topk_idx")
        if recv_topk_idx.element_size() != problem.topk_idx_bytes:
            raise ValueError("recv_topk_idx element width does not match problem.topk_idx_bytes")
        _check_device_tensor(recv_count, "recv_count", torch.int32)
        _check_device_tensor(workspace, "workspace")
        for name, t in _fields_of(layout):
            _check_device_tensor(t, name, torch.int32)
        _check_cumulative(expert_count_cumulative, problem.num_experts // problem.num_ranks)
        _check_device_tensor(recv_buf, "recv_buf")
        for name, t in (("recv_sf_buf", recv_sf_buf), ("recv_x", recv_x), ("recv_sf", recv_sf)):
            if t is not None:
                _check_device_tensor(t, name)
        _check_expand_sizes(problem, recv_topk_idx, recv_count, layout, recv_buf, recv_sf_buf, recv_x, recv_sf)
        # Its own copy of the problem, as in Plan.
        problem = ExpandProblem.from_buffer_copy(problem)
        self._problem = problem
        self._lib = load_library()
        self._keep = (problem, recv_topk_idx, recv_count, layout, workspace, recv_buf, recv_sf_buf, recv_x, recv_sf,
                      expert_count_cumulative)
        self._lay = layout.ptrs(expert_count_cumulative)
        handle = _stream_handle(stream, recv_topk_idx.device)
        rows = (_ptr(recv_buf), _ptr(recv_sf_buf), _ptr(recv_x), _ptr(recv_sf))
        self._layout_args = (ctypes.byref(problem), _ptr(recv_topk_idx), _ptr(recv_count), ctypes.byref(self._lay),
                             _ptr(workspace), workspace.numel() * workspace.element_size(), handle)
        self._scatter_args = (ctypes.byref(problem), ctypes.byref(self._lay), *rows, handle)
        self._both_args = (*self._layout_args[:-1], *rows, handle)

    def layout(self) -> None:
        rc = self._lib.dispatch_expand_layout(*self._layout_args)
        if rc:
            raise DispatchError(rc, "dispatch_expand_layout")

    def scatter(self) -> None:
        rc = self._lib.dispatch_expand_scatter(*self._scatter_args)
        if rc:
            raise DispatchError(rc, "dispatch_expand_scatter")

    def __call__(self) -> None:
        rc = self._lib.dispatch_expand_layout_and_scatter(*self._both_args)
        if rc:
            raise DispatchError(rc, "dispatch_expand_layout_and_scatter")


# ------------------------------------------------------------------- combine


def dispatch_combine(expert_slot: torch.Tensor, topk_weights: torch.Tensor, y: torch.Tensor,
                     out: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue out[t] = sum_k topk_weights[t, k] * y[expert_slot[t, k]] (bf16 rows, fp32 sums)."""
    _check_device_tensor(expert_slot, "expert_slot", torch.int32)
    _check_device_tensor(topk_weights, "topk_weights", torch.float32)
    _check_device_tensor(y, "y", torch.bfloat16)
    _check_device_tensor(out, "out", torch.bfloat16)
    t, k = expert_slot.shape
    if topk_weights.shape != (t, k) or out.shape[0] != t or out.shape[1] != y.shape[1]:
        raise ValueError("combine: shapes do not line up")
    problem = CombineProblem(t, k, 0, y.shape[1], y.shape[0])
    rc = load_library().dispatch_combine(ctypes.byref(problem), _ptr(expert_slot), _ptr(topk_weights), _ptr(y),
                                         _ptr(out), _stream_handle(stream, y.device))
    if rc:
        raise DispatchError(rc, "dispatch_combine")


class CombinePlan:
    """A prepared combine: the tensors and the stream are checked once and the
    C arguments built once, so each call is a single C call."""

    def __init__(self, expert_slot: torch.Tensor, topk_weights: torch.Tensor, y: torch.Tensor, out: torch.Tensor,
                 stream: Optional[torch.cuda.Stream] = None):
        _check_device_tensor(expert_slot, "expert_slot", torch.int32)
        _check_device_tensor(topk_weights, "topk_weights", torch.float32)
        _check_device_tensor(y, "y", torch.bfloat16)
        _check_device_tensor(out, "out", torch.bfloat16)
        t, k = expert_slot.shape
        if topk_weights.shape != (t, k) or out.shape[0] != t or out.shape[1] != y.shape[1]:
            raise ValueError("combine: shapes do not line up")
        self._lib = load_library()
        self._problem = CombineProblem(t, k, 0, y.shape[1], y.shape[0])
        self._keep = (expert_slot, topk_weights, y, out)
        self._args = (ctypes.byref(self._problem), _ptr(expert_slot), _ptr(topk_weights), _ptr(y), _ptr(out),
                      _stream_handle(stream, y.device))

    def __call__(self) -> None:
        rc = self._lib.dispatch_combine(*self._args)
        if rc:
            raise DispatchError(rc, "dispatch_combine")


FP8 = torch.float8_e4m3fn


def _check_one_device(tensors) -> torch.device:
    """The device that all tensors present are on."""
    devices = {t.device for t in tensors if t is not None}
    if len(devices) != 1:
        raise ValueError(f"tensors must be on one device, got {sorted(str(d) for d in devices)}")
    return devices.pop()


class _Prepared:
    """C arguments built once for one C function; with several GPUs a call makes
    the tensors' device the current one where it is not (a null stream is the
    current device's)."""

    def __init__(self, name: str, args, device: torch.device, keep):
        self._name, self._args, self._keep = name, args, keep
        self._call = getattr(load_library(), name)
        self._device = device.index if torch.cuda.device_count() > 1 else None

    def __call__(self) -> None:
        if self._device is None or torch.cuda.current_device() == self._device:
            rc = self._call(*self._args)
        else:
            with torch.cuda.device(self._device):
                rc = self._call(*self._args)
        if rc:
            raise DispatchError(rc, self._name)


class CombineBackwardPlan(_Prepared):
    """A prepared dispatch_combine_backward, like Plan."""

    def __init__(self, expert_slot: torch.Tensor, topk_weights: torch.Tensor, y: Optional[torch.Tensor],
                 grad_out: torch.Tensor, grad_weights: Optional[torch.Tensor] = None,
                 grad_y: Optional[torch.Tensor] = None, grad_q: Optional[torch.Tensor] = None,
                 grad_sf: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        _check_device_tensor(expert_slot, "expert_slot", torch.int32)
        _check_device_tensor(topk_weights, "topk_weights", torch.float32)
        _check_device_tensor(grad_out, "grad_out", torch.bfloat16)
        rows = [t for t in (y, grad_y, grad_q) if t is not None]
        if expert_slot.dim() != 2 or grad_out.dim() != 2 or not rows or any(r.dim() != 2 for r in rows):
            raise ValueError("combine_backward: expert_slot, grad_out and the expert-major rows must be matrices")
        t, k = expert_slot.shape
        n, width = rows[0].shape
        if topk_weights.shape != (t, k) or grad_out.shape != (t, width) or any(r.shape != (n, width) for r in rows):
            raise ValueError("combine_backward: shapes do not line up")
        _check_sized(y, "y", n * width, torch.bfloat16)
        _check_sized(grad_weights, "grad_weights", t * k, torch.float32)
        _check_sized(grad_y, "grad_y", n * width, torch.bfloat16)
        _check_sized(grad_q, "grad_q", n * width, FP8, torch.uint8)
        _check_sized(grad_sf, "grad_sf", n * _sf_blocks(width), torch.float32)
        tensors = (expert_slot, topk_weights, y, grad_out, grad_weights, grad_y, grad_q, grad_sf)
        device = _check_one_device(tensors)
        problem = CombineProblem(t, k, 0, width, n)
        super().__init__("dispatch_combine_backward", (ctypes.byref(problem), *map(_ptr, tensors),
                                                       _stream_handle(stream, device)), device,
                         (problem, tensors, stream))


def dispatch_combine_backward(expert_slot: torch.Tensor, topk_weights: torch.Tensor, y: Optional[torch.Tensor],
                              grad_out: torch.Tensor, grad_weights: Optional[torch.Tensor] = None,
                              grad_y: Optional[torch.Tensor] = None, grad_q: Optional[torch.Tensor] = None,
                              grad_sf: Optional[torch.Tensor] = None,
                              stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue the combine's gradient from grad_out [T, H]: grad_weights [T, K]
    (needs y), and the expert-major rows' gradient, bf16 grad_y or fp8 grad_q
    with its scales grad_sf. Rows that no entry has are not written."""
    CombineBackwardPlan(expert_slot, topk_weights, y, grad_out, grad_weights, grad_y, grad_q, grad_sf, stream)()


# ---------------------------------------------------------------------- gate

_LOGIT_TYPES = {torch.bfloat16: 2, torch.float32: 4}
_INDEX_TYPES = {4: torch.int32, 8: torch.int64}


def make_gate_problem(num_tokens: int, num_experts: int, num_topk: int, scoring: int = GATE_SOFTMAX,
                      logits_dtype: torch.dtype = torch.bfloat16, normalize: bool = True, route_scale: float = 1.0,
                      loss_coef: float = 0.0, topk_idx_bytes: int = 8) -> GateProblem:
    if logits_dtype not in _LOGIT_TYPES:
        raise ValueError(f"logits must be bfloat16 or float32, got {logits_dtype}")
    p = GateProblem(num_tokens, num_experts, num_topk, scoring, _LOGIT_TYPES[logits_dtype], topk_idx_bytes,
                    GATE_NORMALIZE if normalize else 0, route_scale, loss_coef)
    dispatch_gate_workspace_size(p)  # checks the problem
    return p


def dispatch_gate_workspace_size(problem: GateProblem) -> int:
    out = ctypes.c_size_t(0)
    rc = load_library().dispatch_gate_workspace_size(ctypes.byref(problem), ctypes.byref(out))
    if rc:
        raise DispatchError(rc, "dispatch_gate_workspace_size")
    return int(out.value)


@dataclasses.dataclass
class GateTensors:
    """Device outputs of dispatch_gate (see dispatch_gate_out_t); the last four are None without balance outputs."""

    topk_idx: torch.Tensor                  # int64 or int32 [T, K]
    topk_weights: torch.Tensor              # float32 [T, K]
    expert_count: Optional[torch.Tensor]    # int32 [E]
    prob_sum: Optional[torch.Tensor]        # float32 [E]
    live_tokens: Optional[torch.Tensor]     # int32 [1]
    loss: Optional[torch.Tensor]            # float32 [1]

    def ptrs(self) -> GateOutPtrs:
        return GateOutPtrs(*[_ptr(getattr(self, f.name)) for f in dataclasses.fields(self)])


def alloc_gate(problem: GateProblem, device, balance: bool = True) -> GateTensors:
    t, e, k = problem.num_tokens, problem.num_experts, problem.num_topk

    def new(shape, dtype, on=True):
        return torch.empty(shape, dtype=dtype, device=device) if on else None

    return GateTensors(topk_idx=new((t, k), _INDEX_TYPES[problem.topk_idx_bytes]),
                       topk_weights=new((t, k), torch.float32), expert_count=new(e, torch.int32, balance),
                       prob_sum=new(e, torch.float32, balance), live_tokens=new(1, torch.int32, balance),
                       loss=new(1, torch.float32, balance))


def alloc_gate_workspace(problem: GateProblem, device) -> torch.Tensor:
    """Workspace for dispatch_gate with balance outputs (it need not be initialised)."""
    return torch.empty(dispatch_gate_workspace_size(problem), dtype=torch.uint8, device=device)


def _check_sized(t: Optional[torch.Tensor], name: str, count: int, *dtypes) -> None:
    """A device tensor of one of the types with at least `count` elements (None passes)."""
    if t is None:
        return
    _check_device_tensor(t, name)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    _need(t, name, count * t.element_size())


def _logit_type(problem: GateProblem) -> torch.dtype:
    return torch.bfloat16 if problem.logits_bytes == 2 else torch.float32


def _gate_args(problem: GateProblem, logits, out: GateTensors, workspace, select_bias, token_mask, stream):
    t, e, k = problem.num_tokens, problem.num_experts, problem.num_topk
    _check_sized(logits, "logits", t * e, _logit_type(problem))
    _check_sized(out.topk_idx, "topk_idx", t * k, _INDEX_TYPES[problem.topk_idx_bytes])
    _check_sized(out.topk_weights, "topk_weights", t * k, torch.float32)
    _check_sized(out.expert_count, "expert_count", e, torch.int32)
    _check_sized(out.prob_sum, "prob_sum", e, torch.float32)
    _check_sized(out.live_tokens, "live_tokens", 1, torch.int32)
    _check_sized(out.loss, "loss", 1, torch.float32)
    _check_sized(select_bias, "select_bias", e, torch.float32)
    _check_sized(token_mask, "token_mask", t, torch.bool, torch.uint8)
    nbytes = 0
    if workspace is not None:
        _check_device_tensor(workspace, "workspace")
        nbytes = workspace.numel() * workspace.element_size()
    ptrs = out.ptrs()
    return (ctypes.byref(problem), _ptr(logits), _ptr(select_bias), _ptr(token_mask), ctypes.byref(ptrs),
            _ptr(workspace), nbytes, _stream_handle(stream, logits.device)), ptrs


def dispatch_gate(problem: GateProblem, logits: torch.Tensor, out: GateTensors,
                  workspace: Optional[torch.Tensor] = None, select_bias: Optional[torch.Tensor] = None,
                  token_mask: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue the gate: logits [T, E] to out.topk_idx and out.topk_weights,
    and, where ``out`` has them, the balance outputs (these need a workspace)."""
    args, _keep = _gate_args(problem, logits, out, workspace, select_bias, token_mask, stream)
    rc = load_library().dispatch_gate(*args)
    if rc:
        raise DispatchError(rc, "dispatch_gate")


class GatePlan:
    """A prepared gate, like Plan: checked once, one C call per step."""

    def __init__(self, problem: GateProblem, logits: torch.Tensor, out: GateTensors,
                 workspace: Optional[torch.Tensor] = None, select_bias: Optional[torch.Tensor] = None,
                 token_mask: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        problem = GateProblem.from_buffer_copy(problem)
        self._args, ptrs = _gate_args(problem, logits, out, workspace, select_bias, token_mask, stream)
        self._keep = (problem, logits, out, ptrs, workspace, select_bias, token_mask)
        self._call = load_library().dispatch_gate

    def __call__(self) -> None:
        rc = self._call(*self._args)
        if rc:
            raise DispatchError(rc, "dispatch_gate")


def make_gate_groups(num_groups: int, topk_groups: int, score_experts: int = 1) -> GateGroups:
    """``num_groups`` groups of neighbouring experts, ``topk_groups`` of them for
    a token, by their largest choice or (``score_experts`` 2, sigmoid scores
    only) by the sum of their two largest."""
    return GateGroups(num_groups, topk_groups, score_experts, 0)


class GroupedGatePlan(_Prepared):
    """A prepared dispatch_gate_grouped, like Plan."""

    def __init__(self, problem: GateProblem, groups: GateGroups, logits: torch.Tensor, out: GateTensors,
                 workspace: Optional[torch.Tensor] = None, select_bias: Optional[torch.Tensor] = None,
                 token_mask: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        problem, groups = GateProblem.from_buffer_copy(problem), GateGroups.from_buffer_copy(groups)
        (first, *rest), ptrs = _gate_args(problem, logits, out, workspace, select_bias, token_mask, stream)
        outs = [getattr(out, f.name) for f in dataclasses.fields(out)]
        device = _check_one_device((logits, workspace, select_bias, token_mask, *outs))
        super().__init__("dispatch_gate_grouped", (first, ctypes.byref(groups), *rest), device,
                         (problem, groups, logits, outs, ptrs, workspace, select_bias, token_mask, stream))


def dispatch_gate_grouped(problem: GateProblem, groups: GateGroups, logits: torch.Tensor, out: GateTensors,
                          workspace: Optional[torch.Tensor] = None, select_bias: Optional[torch.Tensor] = None,
                          token_mask: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue the gate with each token's experts from its best groups (see
    make_gate_groups); all else as dispatch_gate."""
    GroupedGatePlan(problem, groups, logits, out, workspace, select_bias, token_mask, stream)()


def _gate_backward_args(problem: GateProblem, logits, out: GateTensors, grad_weights, grad_loss, grad_logits,
                        token_mask, stream):
    t, e, k = problem.num_tokens, problem.num_experts, problem.num_topk
    _check_sized(logits, "logits", t * e, _logit_type(problem))
    _check_sized(out.topk_idx, "topk_idx", t * k, _INDEX_TYPES[problem.topk_idx_bytes])
    _check_sized(out.expert_count, "expert_count", e, torch.int32)
    _check_sized(out.live_tokens, "live_tokens", 1, torch.int32)
    _check_sized(grad_weights, "grad_weights", t * k, torch.float32)
    _check_sized(grad_loss, "grad_loss", 1, torch.float32)
    _check_sized(grad_logits, "grad_logits", t * e, _logit_type(problem))
    _check_sized(token_mask, "token_mask", t, torch.bool, torch.uint8)
    return (ctypes.byref(problem), _ptr(logits), _ptr(token_mask), _ptr(out.topk_idx), _ptr(grad_weights),
            _ptr(out.expert_count), _ptr(out.live_tokens), _ptr(grad_loss), _ptr(grad_logits),
            _stream_handle(stream, logits.device))


def dispatch_gate_backward(problem: GateProblem, logits: torch.Tensor, out: GateTensors,
                           grad_weights: Optional[torch.Tensor], grad_loss: Optional[torch.Tensor],
                           grad_logits: torch.Tensor, token_mask: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue the gradient of the logits from those of out.topk_weights and
    out.loss (None = zero). ``out`` holds dispatch_gate's outputs for them."""
    rc = load_library().dispatch_gate_backward(*_gate_backward_args(problem, logits, out, grad_weights, grad_loss,
                                                                    grad_logits, token_mask, stream))
    if rc:
        raise DispatchError(rc, "dispatch_gate_backward")


class GateBackwardPlan:
    """A prepared gate gradient, like Plan."""

    def __init__(self, problem: GateProblem, logits: torch.Tensor, out: GateTensors,
                 grad_weights: Optional[torch.Tensor], grad_loss: Optional[torch.Tensor], grad_logits: torch.Tensor,
                 token_mask: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        problem = GateProblem.from_buffer_copy(problem)
        self._args = _gate_backward_args(problem, logits, out, grad_weights, grad_loss, grad_logits, token_mask, stream)
        self._keep = (problem, logits, out, grad_weights, grad_loss, grad_logits, token_mask)
        self._call = load_library().dispatch_gate_backward

    def __call__(self) -> None:
        rc = self._call(*self._args)
        if rc:
            raise DispatchError(rc, "dispatch_gate_backward")


# -------------------------------------------------------------- quantisation


def _sf_blocks(width: int) -> int:
    return (width + SF_BLOCK - 1) // SF_BLOCK


def _check_grad(grad: Optional[torch.Tensor]) -> None:
    """SwiGLU's gradient needs one (None stands for the calls that have none)."""
    if grad is None:
        raise ValueError("grad must be a device tensor")


def _quantize_args(x, grad, q, sf, num_valid_rows, halves_in: int, halves_out: int, stream):
    """halves_in, halves_out: x's and q's channels in units of the problem's width."""
    _check_device_tensor(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.shape[1] % halves_in:
        raise ValueError("x must be [rows, channels], with as many gate as up channels for SwiGLU")
    rows, width = x.shape[0], x.shape[1] // halves_in
    if grad is not None:
        _check_sized(grad, "grad", rows * width, torch.bfloat16)
    _check_sized(q, "q", rows * width * halves_out, FP8, torch.uint8)
    _check_sized(sf, "sf", rows * _sf_blocks(width) * halves_out, torch.float32)
    _check_sized(num_valid_rows, "num_valid_rows", 1, torch.int32)
    problem = QuantizeProblem(rows, width)
    rows_ptrs = (_ptr(x),) if grad is None else (_ptr(x), _ptr(grad))
    return (ctypes.byref(problem), *rows_ptrs, _ptr(num_valid_rows), _ptr(q), _ptr(sf),
            _stream_handle(stream, x.device)), problem


def dispatch_quantize(x: torch.Tensor, q: torch.Tensor, sf: torch.Tensor,
                      num_valid_rows: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue bf16 rows [R, H] to fp8 q [R, H] and scales sf [R, ceil(H / 128)]."""
    args, _keep = _quantize_args(x, None, q, sf, num_valid_rows, 1, 1, stream)
    rc = load_library().dispatch_quantize(*args)
    if rc:
        raise DispatchError(rc, "dispatch_quantize")


def dispatch_swiglu_quantize(h: torch.Tensor, q: torch.Tensor, sf: torch.Tensor,
                             num_valid_rows: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue SwiGLU of bf16 h [R, 2I] to fp8 q [R, I] and scales sf [R, I / 128]."""
    args, _keep = _quantize_args(h, None, q, sf, num_valid_rows, 2, 1, stream)
    rc = load_library().dispatch_swiglu_quantize(*args)
    if rc:
        raise DispatchError(rc, "dispatch_swiglu_quantize")


def dispatch_swiglu_backward_quantize(h: torch.Tensor, grad: torch.Tensor, q: torch.Tensor, sf: torch.Tensor,
                                      num_valid_rows: Optional[torch.Tensor] = None,
                                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue SwiGLU's gradient with respect to h [R, 2I], from grad [R, I],
    to fp8 q [R, 2I] and scales sf [R, 2I / 128]."""
    _check_grad(grad)
    args, _keep = _quantize_args(h, grad, q, sf, num_valid_rows, 2, 2, stream)
    rc = load_library().dispatch_swiglu_backward_quantize(*args)
    if rc:
        raise DispatchError(rc, "dispatch_swiglu_backward_quantize")


class QuantizePlan:
    """A prepared dispatch_quantize, like Plan."""

    _name, _halves = "dispatch_quantize", (1, 1)

    def __init__(self, x: torch.Tensor, q: torch.Tensor, sf: torch.Tensor,
                 num_valid_rows: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        self._prepare(x, None, q, sf, num_valid_rows, stream)

    def _prepare(self, x, grad, q, sf, num_valid_rows, stream):
        self._args, problem = _quantize_args(x, grad, q, sf, num_valid_rows, *self._halves, stream)
        self._keep = (problem, x, grad, q, sf, num_valid_rows)
        self._call = getattr(load_library(), self._name)

    def __call__(self) -> None:
        rc = self._call(*self._args)
        if rc:
            raise DispatchError(rc, self._name)


class SwigluQuantizePlan(QuantizePlan):
    """A prepared dispatch_swiglu_quantize, like Plan."""

    _name, _halves = "dispatch_swiglu_quantize", (2, 1)


class SwigluBackwardQuantizePlan(QuantizePlan):
    """A prepared dispatch_swiglu_backward_quantize, like Plan."""

    _name, _halves = "dispatch_swiglu_backward_quantize", (2, 2)

    def __init__(self, h: torch.Tensor, grad: torch.Tensor, q: torch.Tensor, sf: torch.Tensor,
                 num_valid_rows: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        _check_grad(grad)
        self._prepare(h, grad, q, sf, num_valid_rows, stream)


# ------------------------------------------------------------------ RMS norm

_WEIGHT_TYPES = {torch.bfloat16: 2, torch.float32: 4}


def _rms_norm_problem(rows: torch.Tensor, name: str, weight: torch.Tensor, eps: float) -> RmsNormProblem:
    _check_device_tensor(rows, name, torch.bfloat16)
    if rows.dim() != 2:
        raise ValueError(f"{name} must be [rows, channels]")
    _check_sized(weight, "weight", rows.shape[1], *_WEIGHT_TYPES)
    return RmsNormProblem(rows.shape[0], rows.shape[1], _WEIGHT_TYPES[weight.dtype], eps)


class RmsNormPlan(_Prepared):
    """A prepared dispatch_rms_norm, like Plan."""

    def __init__(self, x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                 h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                 sf: Optional[torch.Tensor] = None, num_valid_rows: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
        problem = _rms_norm_problem(x, "x", weight, eps)
        size = x.numel()
        for t, name in ((residual, "residual"), (h, "h"), (y, "y")):
            _check_sized(t, name, size, torch.bfloat16)
        _check_sized(q, "q", size, FP8, torch.uint8)
        _check_sized(sf, "sf", x.shape[0] * _sf_blocks(x.shape[1]), torch.float32)
        _check_sized(num_valid_rows, "num_valid_rows", 1, torch.int32)
        tensors = (x, residual, weight, num_valid_rows, h, y, q, sf)
        device = _check_one_device(tensors)
        super().__init__("dispatch_rms_norm", (ctypes.byref(problem), *map(_ptr, tensors),
                                               _stream_handle(stream, device)), device,
                         (problem, tensors, stream))


def dispatch_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                      h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                      q: Optional[torch.Tensor] = None, sf: Optional[torch.Tensor] = None,
                      num_valid_rows: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue h = x + residual and its RMS norm times weight, to bf16 rows y
    [R, W], to fp8 rows q [R, W] with scales sf [R, ceil(W / 128)], or to both.
    Without a residual there is no h; h may be x or residual."""
    RmsNormPlan(x, weight, eps, residual, h, y, q, sf, num_valid_rows, stream)()


def dispatch_rms_norm_workspace_size(problem: RmsNormProblem) -> int:
    out = ctypes.c_size_t(0)
    rc = load_library().dispatch_rms_norm_workspace_size(ctypes.byref(problem), ctypes.byref(out))
    if rc:
        raise DispatchError(rc, "dispatch_rms_norm_workspace_size")
    return int(out.value)


def alloc_rms_norm_workspace(num_rows: int, width: int, device) -> torch.Tensor:
    """Workspace for the weight's gradient (it need not be initialised)."""
    problem = RmsNormProblem(num_rows, width, 4, 1.0)
    return torch.empty(dispatch_rms_norm_workspace_size(problem), dtype=torch.uint8, device=device)


class RmsNormBackwardPlan(_Prepared):
    """A prepared dispatch_rms_norm_backward, like Plan."""

    def __init__(self, h: torch.Tensor, weight: torch.Tensor, grad_y: torch.Tensor, eps: float, grad_x: torch.Tensor,
                 grad_h: Optional[torch.Tensor] = None, grad_weight: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, num_valid_rows: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
        problem = _rms_norm_problem(h, "h", weight, eps)
        for t, name in ((grad_y, "grad_y"), (grad_h, "grad_h"), (grad_x, "grad_x")):
            _check_sized(t, name, h.numel(), torch.bfloat16)
        _check_sized(grad_weight, "grad_weight", h.shape[1], torch.float32)
        _check_sized(num_valid_rows, "num_valid_rows", 1, torch.int32)
        nbytes = 0
        if workspace is not None:
            _check_device_tensor(workspace, "workspace")
            nbytes = workspace.numel() * workspace.element_size()
        tensors = (h, weight, grad_y, grad_h, num_valid_rows, grad_x, grad_weight, workspace)
        device = _check_one_device(tensors)
        super().__init__("dispatch_rms_norm_backward", (ctypes.byref(problem), *map(_ptr, tensors), nbytes,
                                                        _stream_handle(stream, device)), device,
                         (problem, tensors, stream))


def dispatch_rms_norm_backward(h: torch.Tensor, weight: torch.Tensor, grad_y: torch.Tensor, eps: float,
                               grad_x: torch.Tensor, grad_h: Optional[torch.Tensor] = None,
                               grad_weight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                               num_valid_rows: Optional[torch.Tensor] = None,
                               stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue the norm's gradient: grad_x [R, W], that of h (grad_h is added to
    it), and grad_weight [W] (needs a workspace)."""
    RmsNormBackwardPlan(h, weight, grad_y, eps, grad_x, grad_h, grad_weight, workspace, num_valid_rows, stream)()


# ---------------------------------------------------------- experts' product


def make_expert_problem(num_experts: int, in_features: int, out_features: int, expert_rows: int,
                        max_routed_rows: Optional[int] = None) -> ExpertProblem:
    """``expert_rows``: rows of the expert-major buffers (recv_capacity_rows).
    ``max_routed_rows``: about how many of them are routed at most (T * K; it
    picks the kernel, and defaults to expert_rows)."""
    return ExpertProblem(num_experts, 0, in_features, out_features, expert_rows,
                         expert_rows if max_routed_rows is None else max_routed_rows)


def dispatch_expert_workspace_size(problem: ExpertProblem) -> int:
    out = ctypes.c_size_t(0)
    rc = load_library().dispatch_expert_workspace_size(ctypes.byref(problem), ctypes.byref(out))
    if rc:
        raise DispatchError(rc, "dispatch_expert_workspace_size")
    return int(out.value)


def alloc_expert_workspace(problem: ExpertProblem, device) -> Optional[torch.Tensor]:
    """Workspace for the products of a problem: zero-filled, as its first use
    requires; None where the problem has no use for one."""
    n = dispatch_expert_workspace_size(problem)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def _expert_args(problem: ExpertProblem, expert_psum, expert_count, x, x_sf, w, w_sf, out, out_sf, swiglu, workspace,
                 stream):
    e, k, n, rows = problem.num_experts, problem.in_features, problem.out_features, problem.expert_rows
    _check_sized(expert_psum, "expert_psum", e + 1, torch.int32)
    _check_sized(expert_count, "expert_count", e, torch.int32)
    _check_sized(x, "x", rows * k, FP8, torch.uint8)
    _check_sized(x_sf, "x_sf", rows * _sf_blocks(k), torch.float32)
    _check_sized(w, "w", e * n * k, FP8, torch.uint8)
    _check_sized(w_sf, "w_sf", e * _sf_blocks(n) * _sf_blocks(k), torch.float32)
    if swiglu:
        _check_sized(out, "out_q", rows * (n // 2), FP8, torch.uint8)
        _check_sized(out_sf, "out_sf", rows * (n // 2 // SF_BLOCK), torch.float32)
    else:
        _check_sized(out, "out", rows * n, torch.bfloat16)
    nbytes = 0
    if workspace is not None:
        _check_device_tensor(workspace, "workspace")
        nbytes = workspace.numel() * workspace.element_size()
    outs = (_ptr(out), _ptr(out_sf)) if swiglu else (_ptr(out),)
    return (ctypes.byref(problem), _ptr(expert_psum), _ptr(expert_count), _ptr(x), _ptr(x_sf), _ptr(w), _ptr(w_sf),
            *outs, _ptr(workspace), nbytes, _stream_handle(stream, w.device))


def dispatch_expert_product(problem: ExpertProblem, expert_psum: torch.Tensor, expert_count: torch.Tensor,
                            x: torch.Tensor, x_sf: torch.Tensor, w: torch.Tensor, w_sf: torch.Tensor,
                            out: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue out[r] = x[r] @ w[e].T for the rows r of each expert e (fp8
    operands with block scales, bf16 out). ``workspace``: from
    alloc_expert_workspace, for few rows (optional)."""
    rc = load_library().dispatch_expert_product(*_expert_args(problem, expert_psum, expert_count, x, x_sf, w, w_sf,
                                                              out, None, False, workspace, stream))
    if rc:
        raise DispatchError(rc, "dispatch_expert_product")


def dispatch_expert_product_swiglu(problem: ExpertProblem, expert_psum: torch.Tensor, expert_count: torch.Tensor,
                                   x: torch.Tensor, x_sf: torch.Tensor, w: torch.Tensor, w_sf: torch.Tensor,
                                   out_q: torch.Tensor, out_sf: torch.Tensor,
                                   workspace: Optional[torch.Tensor] = None,
                                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """Enqueue SwiGLU of that product (w [E, 2I, K], gate rows first),
    quantised: out_q [expert_rows, I] and out_sf [expert_rows, I / 128]."""
    rc = load_library().dispatch_expert_product_swiglu(*_expert_args(problem, expert_psum, expert_count, x, x_sf, w,
                                                                     w_sf, out_q, out_sf, True, workspace, stream))
    if rc:
        raise DispatchError(rc, "dispatch_expert_product_swiglu")


class ExpertProductPlan:
    """A prepared dispatch_expert_product, like Plan. A plan of few rows makes
    a workspace of its own unless it is given one, so a plan's calls must not
    overlap in time."""

    def __init__(self, problem: ExpertProblem, expert_psum: torch.Tensor, expert_count: torch.Tensor,
                 x: torch.Tensor, x_sf: torch.Tensor, w: torch.Tensor, w_sf: torch.Tensor, out: torch.Tensor,
                 workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        self._prepare(False, problem, (expert_psum, expert_count, x, x_sf, w, w_sf), out, None, workspace, stream)
        self._call = load_library().dispatch_expert_product

    def _prepare(self, swiglu, problem, ins, out, out_sf, workspace, stream):
        problem = ExpertProblem.from_buffer_copy(problem)
        if workspace is None:
            # Cleared on the stream that the calls run on.
            with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(ins[4].device)):
                workspace = alloc_expert_workspace(problem, ins[4].device)
        self._args = _expert_args(problem, *ins, out, out_sf, swiglu, workspace, stream)
        self._keep = (problem, ins, out, out_sf, workspace)

    def __call__(self) -> None:
        rc = self._call(*self._args)
        if rc:
            raise DispatchError(rc, self._call.__name__)


class ExpertSwigluPlan(ExpertProductPlan):
    """A prepared dispatch_expert_product_swiglu, like ExpertProductPlan."""

    def __init__(self, problem: ExpertProblem, expert_psum: torch.Tensor, expert_count: torch.Tensor,
                 x: torch.Tensor, x_sf: torch.Tensor, w: torch.Tensor, w_sf: torch.Tensor, out_q: torch.Tensor,
                 out_sf: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
        self._prepare(True, problem, (expert_psum, expert_count, x, x_sf, w, w_sf), out_q, out_sf, workspace, stream)
        self._call = load_library().dispatch_expert_product_swiglu
