"""Single-GPU MoE expert-parallel token shuffle for GB300: Python binding.

A thin ctypes layer over the C ABI in include/ep.h (libep.so, hand-written
CUDA for sm_103a).  It only marshals arguments: it allocates output tensors
with torch and passes raw device pointers and the current CUDA stream.  Every
step of layout, dispatch and combine runs in the library's kernels.  There is
no CPU or PyTorch fallback.  If the library is missing or cannot be loaded,
every call raises.

The three steps follow the high-throughput expert-parallel kernels of
"[Not ready] MSCCLPP EP implementation" (mscclpp pull request 852), section
"Scope" (get_dispatch_layout, intranode_dispatch, intranode_combine), with the
kUseFP8 payload cast of its low-latency dispatch.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libep.so")

EP_OK = 0
EP_ERRBIT_BAD_EXPERT = 1
EP_ERRBIT_CAPACITY = 2
EP_ERRBIT_TIMEOUT = 4
EP_ERRBIT_SCHED = 8
EP_MAX_RANKS = 64
EP_MAX_TOPK = 32
EP_MAX_EXPERTS = 4096
EP_LAYER_MAX_TOKENS = 16
EP_LAYER_MAX_EXPERTS = 512
EP_NORM_MAX_HIDDEN = 16384

# ep_layout_path_t
LAYOUT_PATHS = {"auto": 0, "multi": 1, "single": 2}

# ep_score_t, ep_act_t
SCORES = {"softmax": 0, "sigmoid": 1}
ACTS = {"none": 0, "swiglu": 1}
# ep_gate_t
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = range(4)

# every entry point declared in include/ep.h
EXPORTED = ("ep_status_string", "ep_workspace_bytes", "ep_get_dispatch_layout",
            "ep_layout_single_launch_fits", "ep_layout_auto_single_launch",
            "ep_get_dispatch_layout_path",
            "ep_get_dispatch_layout_noalloc", "ep_layout_total_rows", "ep_dispatch",
            "ep_combine", "ep_ll_workspace_bytes", "ep_ll_get_dispatch_layout",
            "ep_ll_dispatch", "ep_ll_combine", "ep_debug_set_combine_stall",
            "ep_ll_layout_single_launch_fits", "ep_ll_layout_auto_single_launch",
            "ep_ll_get_dispatch_layout_path", "ep_combine_sched", "ep_ll_combine_sched",
            "ep_layout_dispatch_fused_fits", "ep_layout_dispatch_fused",
            "ep_layout_dispatch_fused_workspace_bytes", "ep_debug_set_fused_stall",
            "ep_shard_workspace_bytes", "ep_shard_layout", "ep_shard_offsets",
            "ep_shard_recv_tokens_per_expert", "ep_debug_e4m3_range",
            "ep_route", "ep_route_backward", "ep_combine_backward", "ep_ll_combine_backward",
            "ep_ll_experts_w4", "ep_debug_set_experts_stall",
            "ep_layer_w4", "ep_layer_w4_workspace_bytes", "ep_block_norm",
            "ep_block_norm_backward", "ep_block_norm_backward_workspace_bytes",
            "ep_ll_swiglu", "ep_ll_swiglu_backward")

# 64-bit words of a combine's scheduling counters (EP_COMBINE_SCHED_WORDS)
COMBINE_SCHED_WORDS = 2
# 64-bit words of the fused layout + dispatch's counters (EP_FUSED_SYNC_WORDS)
FUSED_SYNC_WORDS = 640

_lib = None


class EPError(RuntimeError):
    pass


def load(path: str | None = None) -> C.CDLL:
    """Load libep.so (built by combine_get_dispatch_04_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise EPError(f"CUDA library not built: {path} is missing "
                      "(run combine_get_dispatch_04_gb300.build.build())")
    L = C.CDLL(path)
    P, i32, i64, sz = C.c_void_p, C.c_int, C.c_int64, C.c_size_t
    L.ep_status_string.argtypes = [i32]
    L.ep_status_string.restype = C.c_char_p
    L.ep_workspace_bytes.argtypes = [i64, i32, i32]
    L.ep_workspace_bytes.restype = sz
    L.ep_get_dispatch_layout.argtypes = [P, i64, i32, i32, i32, P, P, P, P, P, P, P, sz, P]
    L.ep_layout_single_launch_fits.argtypes = [i64, i32, i32]
    L.ep_layout_single_launch_fits.restype = i32
    L.ep_layout_auto_single_launch.argtypes = [i64, i32, i32]
    L.ep_layout_auto_single_launch.restype = i32
    L.ep_get_dispatch_layout_path.argtypes = [P, i64, i32, i32, i32, P, P, P, P, P, P, P, sz,
                                              i32, P]
    L.ep_layout_total_rows.argtypes = [P, i32, P, P]
    L.ep_dispatch.argtypes = [P, i32, P, P, i64, i32, i32, i32, P, P, i64, i32, P, P, P, P, P,
                              P, P, P]
    L.ep_combine.argtypes = [P, i32, P, P, i64, i32, i32, i32, P, P, P, P]
    L.ep_debug_set_combine_stall.argtypes = [i32]
    L.ep_debug_set_combine_stall.restype = None
    L.ep_ll_workspace_bytes.argtypes = [i64, i32, i32]
    L.ep_ll_workspace_bytes.restype = sz
    L.ep_ll_get_dispatch_layout.argtypes = [P, i64, i32, i32, i32, i64, P, P, P, P, P, sz, P]
    L.ep_ll_get_dispatch_layout_path.argtypes = [P, i64, i32, i32, i32, i64, P, P, P, P, P, sz,
                                                 i32, P]
    for name in ("ep_ll_layout_single_launch_fits", "ep_ll_layout_auto_single_launch"):
        getattr(L, name).argtypes = [i64, i32, i32, i32]
        getattr(L, name).restype = i32
    L.ep_ll_dispatch.argtypes = [P, i32, i64, i32, P, i64, i32, P, P, P, P, P]
    L.ep_ll_combine.argtypes = [P, i32, P, i64, i32, P, P, P, P]
    L.ep_combine_sched.argtypes = [P, i32, P, P, i64, i32, i32, i32, P, P, P, P, P]
    L.ep_ll_combine_sched.argtypes = [P, i32, P, i64, i32, P, P, P, P, P]
    L.ep_layout_dispatch_fused_fits.argtypes = [i64, i32, i32]
    L.ep_layout_dispatch_fused_fits.restype = i32
    L.ep_layout_dispatch_fused_workspace_bytes.argtypes = [i64, i32, i32]
    L.ep_layout_dispatch_fused_workspace_bytes.restype = sz
    L.ep_layout_dispatch_fused.argtypes = [P, i32, P, P, i64, i32, i32, i32, P, P, P, P, P, i64,
                                           i32, P, P, P, P, P, P, P, sz, P, P, P]
    L.ep_debug_set_fused_stall.argtypes = [i32]
    L.ep_debug_set_fused_stall.restype = None
    L.ep_debug_e4m3_range.argtypes = [C.c_uint32, i64, P, P]
    L.ep_shard_workspace_bytes.argtypes = [i64, i32, i32]
    L.ep_shard_workspace_bytes.restype = sz
    L.ep_shard_layout.argtypes = [P, i64, i32, i32, i32, P, P, P, P, P, P, P, sz, P]
    L.ep_shard_offsets.argtypes = [P, i32, i32, P, P]
    L.ep_shard_recv_tokens_per_expert.argtypes = [P, i32, i32, i32, P]
    f32 = C.c_float
    L.ep_route.argtypes = [P, i32, i64, P, i64, i32, i32, i32, i32, i32, i32, f32, P, P, P]
    L.ep_route_backward.argtypes = [P, P, i32, i64, P, i64, i32, i32, i32, i32, f32, P, P, P]
    L.ep_combine_backward.argtypes = [P, P, i32, i64, P, P, i64, i32, i32, i32, P, P, P, P, P]
    L.ep_ll_combine_backward.argtypes = [P, P, i32, i64, P, i64, i32, P, P, P, P, P]
    L.ep_ll_experts_w4.argtypes = [P, i32, P, i32, P, i32, i64, P, P, P, i32, i32, i32, P, P, P]
    L.ep_debug_set_experts_stall.argtypes = [i32]
    L.ep_debug_set_experts_stall.restype = None
    L.ep_layer_w4_workspace_bytes.argtypes = [i64, i32, i32]
    L.ep_layer_w4_workspace_bytes.restype = sz
    L.ep_layer_w4.argtypes = [P, i32, i32, i64, P, i32, i64, P, i32, i32, i32, i32, i32, i32, f32,
                              P, P, P, i32, P, P, P, i32, P, P, P, P, sz, P]
    L.ep_block_norm.argtypes = [P, i32, P, i64, P, i32, P, i64, i32, P, i32, P, P, i32, f32, f32,
                                P, P, P, P, P]
    L.ep_block_norm_backward_workspace_bytes.argtypes = [i64, i32]
    L.ep_block_norm_backward_workspace_bytes.restype = sz
    L.ep_block_norm_backward.argtypes = [P, P, P, i32, P, i64, i32, P, i32, P, P, i32, f32, f32,
                                         P, P, P, P, P, P, sz, P]
    L.ep_ll_swiglu.argtypes = [P, i32, i64, P, i64, i32, P, P, P, P, P, P]
    L.ep_ll_swiglu_backward.argtypes = [P, P, P, P, i32, i64, P, i64, i32, P, P, P, P, P]
    for name in ("ep_route", "ep_route_backward", "ep_combine_backward",
                 "ep_ll_combine_backward", "ep_ll_experts_w4", "ep_layer_w4", "ep_block_norm",
                 "ep_block_norm_backward", "ep_ll_swiglu", "ep_ll_swiglu_backward"):
        getattr(L, name).restype = i32
    for name in ("ep_get_dispatch_layout", "ep_get_dispatch_layout_path",
                 "ep_layout_total_rows", "ep_dispatch", "ep_combine",
                 "ep_ll_get_dispatch_layout", "ep_ll_get_dispatch_layout_path",
                 "ep_ll_dispatch", "ep_ll_combine", "ep_combine_sched", "ep_ll_combine_sched",
                 "ep_layout_dispatch_fused", "ep_shard_layout", "ep_shard_offsets",
                 "ep_shard_recv_tokens_per_expert", "ep_debug_e4m3_range"):
        getattr(L, name).restype = i32
    _lib = L
    return L


def lib() -> C.CDLL:
    return load()


# Debug mode (environment EP_DEBUG=1, or set_debug(True)): every call waits
# for its stream and raises at once if the device error word it was given is
# non-zero or the kernels failed, naming the call.  Off by default: calls are
# asynchronous.
_debug = os.environ.get("EP_DEBUG", "0") not in ("", "0")

_ERRBITS = ((EP_ERRBIT_BAD_EXPERT, "an expert id outside [-1, E)"),
            (EP_ERRBIT_CAPACITY, "a row at or beyond the receive capacity"),
            (EP_ERRBIT_TIMEOUT, "a bounded pipeline wait ran out"),
            (EP_ERRBIT_SCHED, "a combine's scheduling counters were in use by another launch"))


def set_debug(on: bool) -> None:
    """Synchronise and check the error word after every call (see above)."""
    global _debug
    _debug = bool(on)


def describe_error_word(value: int) -> str:
    names = [text for bit, text in _ERRBITS if value & bit]
    return ", ".join(names) if names else "no error"


def _debug_check(what: str, err: torch.Tensor | None, device: torch.device):
    if not _debug:
        return
    torch.cuda.current_stream(device).synchronize()  # raises on a kernel fault
    if err is not None and int(err.item()) != 0:
        v = int(err.item())
        raise EPError(f"{what}: device error word {v} ({describe_error_word(v)})")


def _check(status: int, what: str):
    if status != EP_OK:
        msg = lib().ep_status_string(status).decode()
        raise EPError(f"{what} failed: {msg}")


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a Stream object (2 us a call on
# the host of a GB300), where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device):
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None):
    if not t.is_cuda:
        raise EPError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise EPError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise EPError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise EPError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


@dataclass
class Layout:
    """Outputs of get_dispatch_layout (all on the device)."""
    num_tokens_per_rank: torch.Tensor    # [R, R] int32, row = source rank
    num_tokens_per_expert: torch.Tensor  # [R, E] int32, row = source rank
    is_token_in_rank: torch.Tensor       # [T, R] bool
    slot: torch.Tensor                   # [T, R] int32, -1 = not sent
    recv_base: torch.Tensor              # [R + 1] int32, recv_base[R] = P
    num_experts: int
    num_ranks: int
    workspace: torch.Tensor | None = None
    # [2] int64 counters of the dynamically scheduled combine, zero between
    # launches; None: the static schedule.  They serve the combines of the
    # first stream that uses them; combines on any other stream get counters
    # of their own (sched_for), so that combines through one Layout on two
    # streams, or a graph replayed beside eager calls, never share them.
    sched: torch.Tensor | None = None
    # [FUSED_SYNC_WORDS] int64 counters and flags of the one-launch layout +
    # dispatch, zero between launches; per stream like sched
    fused_sync: torch.Tensor | None = None

    @property
    def num_tokens(self) -> int:
        return self.slot.shape[0]


def workspace_bytes(num_tokens: int, num_ranks: int, num_experts: int) -> int:
    return int(lib().ep_workspace_bytes(num_tokens, num_ranks, num_experts))


def single_launch_fits(num_tokens: int, num_ranks: int, num_experts: int) -> bool:
    """True if the one-launch (thread-block cluster) layout applies."""
    return bool(lib().ep_layout_single_launch_fits(num_tokens, num_ranks, num_experts))


def auto_single_launch(num_tokens: int, num_ranks: int, num_experts: int) -> bool:
    """True if path="auto" takes the one-launch layout for this batch."""
    return bool(lib().ep_layout_auto_single_launch(num_tokens, num_ranks, num_experts))


def alloc_combine_sched(device: torch.device) -> torch.Tensor:
    """Zeroed counters for the dynamically scheduled combine (each launch
    leaves them zero again)."""
    return torch.zeros(COMBINE_SCHED_WORDS, dtype=torch.int64, device=device)


def alloc_layout(num_tokens: int, num_experts: int, num_ranks: int,
                 device: torch.device) -> Layout:
    """Output tensors and the multi-launch workspace (allocated for every size,
    so that the same Layout serves either path)."""
    T, R, E = num_tokens, num_ranks, num_experts
    i32 = dict(dtype=torch.int32, device=device)
    # one workspace for the multi-launch layout and the one-launch layout + dispatch
    wsb = max(workspace_bytes(T, R, E),
              int(lib().ep_layout_dispatch_fused_workspace_bytes(T, R, E)), 16)
    ws = torch.empty(wsb, dtype=torch.uint8, device=device)
    return Layout(torch.empty((R, R), **i32), torch.empty((R, E), **i32),
                  torch.empty((T, R), dtype=torch.bool, device=device),
                  torch.empty((T, R), **i32), torch.empty(R + 1, **i32), E, R, ws,
                  alloc_combine_sched(device),
                  torch.zeros(FUSED_SYNC_WORDS, dtype=torch.int64, device=device))


def get_dispatch_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int, *,
                        err: torch.Tensor | None = None, out: Layout | None = None,
                        path: str = "auto") -> Layout:
    """Per-rank / per-expert counts, is_token_in_rank and the slot of every
    (token, destination rank) pair.  Enqueued on the current stream.
    path: "auto", "multi" (multi-launch) or "single" (one cluster launch,
    small batches only); all give the same outputs."""
    _need(topk_idx, "topk_idx", torch.int64)
    if topk_idx.dim() != 2:
        raise EPError("topk_idx must be [num_tokens, num_topk]")
    if path not in LAYOUT_PATHS:
        raise EPError(f"path must be one of {sorted(LAYOUT_PATHS)}")
    T, K = topk_idx.shape
    L = out if out is not None else alloc_layout(T, num_experts, num_ranks, topk_idx.device)
    if err is not None:
        _need(err, "err", torch.int32)
    args = (_ptr(topk_idx), T, K, num_experts, num_ranks, _ptr(L.num_tokens_per_rank),
            _ptr(L.num_tokens_per_expert), _ptr(L.is_token_in_rank), _ptr(L.slot),
            _ptr(L.recv_base), _ptr(err), _ptr(L.workspace),
            L.workspace.numel() if L.workspace is not None else 0)
    stream = _stream(topk_idx.device)
    if path == "auto":
        _check(lib().ep_get_dispatch_layout(*args, stream), "ep_get_dispatch_layout")
    else:
        _check(lib().ep_get_dispatch_layout_path(*args, LAYOUT_PATHS[path], stream),
               "ep_get_dispatch_layout_path")
    _debug_check("get_dispatch_layout", err, topk_idx.device)
    return L


def total_rows(layout: Layout) -> int:
    """P = rows of the receive buffer (copies one int32 and synchronises)."""
    v = C.c_int32(0)
    _check(lib().ep_layout_total_rows(_ptr(layout.recv_base), layout.num_ranks, C.byref(v),
                                      _stream(layout.recv_base.device)), "ep_layout_total_rows")
    return int(v.value)


@dataclass
class Dispatched:
    recv_x: torch.Tensor                # [cap, H] bf16, or [cap, H] uint8 E4M3 codes
    recv_scales: torch.Tensor | None    # [cap, H/128] float32 (FP8 only)
    recv_src_idx: torch.Tensor          # [cap] int32
    recv_topk_idx: torch.Tensor         # [cap, K] int64
    recv_topk_weights: torch.Tensor     # [cap, K] float32
    num_recv_tokens_per_expert: torch.Tensor  # [R, E/R] int32
    use_fp8: bool


def worst_case_rows(num_tokens: int, num_topk: int, num_ranks: int) -> int:
    return num_tokens * min(num_topk, num_ranks)


def alloc_dispatched(capacity: int, hidden: int, num_topk: int, num_experts: int,
                     num_ranks: int, use_fp8: bool, device: torch.device) -> Dispatched:
    if use_fp8:
        recv_x = torch.empty((capacity, hidden), dtype=torch.uint8, device=device)
        scales = torch.empty((capacity, hidden // 128), dtype=torch.float32, device=device)
    else:
        recv_x = torch.empty((capacity, hidden), dtype=torch.bfloat16, device=device)
        scales = None
    return Dispatched(recv_x, scales,
                      torch.empty(capacity, dtype=torch.int32, device=device),
                      torch.empty((capacity, num_topk), dtype=torch.int64, device=device),
                      torch.empty((capacity, num_topk), dtype=torch.float32, device=device),
                      torch.empty((num_ranks, num_experts // num_ranks), dtype=torch.int32,
                                  device=device), use_fp8)


def dispatch(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
             layout: Layout, *, use_fp8: bool = False, capacity: int | None = None,
             err: torch.Tensor | None = None, out: Dispatched | None = None) -> Dispatched:
    """Scatter every token row to its destination ranks' rows (bf16 copy or
    FP8 E4M3 with per-128-channel scales).  Enqueued on the current stream."""
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    K = topk_idx.shape[1]
    _need(topk_idx, "topk_idx", torch.int64, (T, K))
    _need(topk_weights, "topk_weights", torch.float32, (T, K))
    R, E = layout.num_ranks, layout.num_experts
    _need(layout.slot, "slot", torch.int32, (T, R))
    if out is None:
        cap = capacity if capacity is not None else worst_case_rows(T, K, R)
        out = alloc_dispatched(cap, H, K, E, R, use_fp8, x.device)
    elif out.use_fp8 != use_fp8:
        raise EPError("preallocated dispatch buffers have the wrong payload type")
    cap = out.recv_x.shape[0]
    if err is not None:
        _need(err, "err", torch.int32)
    # a shard's layout has no [R, E] per-source counts: no per-expert receive counts here
    ntpe = getattr(layout, "num_tokens_per_expert", None)
    nrpe = out.num_recv_tokens_per_expert if ntpe is not None else None
    _check(lib().ep_dispatch(
        _ptr(x), H, _ptr(topk_idx), _ptr(topk_weights), T, K, E, R, _ptr(layout.slot),
        _ptr(ntpe), cap, int(use_fp8), _ptr(out.recv_x),
        _ptr(out.recv_scales), _ptr(out.recv_src_idx), _ptr(out.recv_topk_idx),
        _ptr(out.recv_topk_weights), _ptr(nrpe), _ptr(err),
        _stream(x.device)), "ep_dispatch")
    _debug_check("dispatch", err, x.device)
    return out


def _per_stream(s: torch.Tensor, name: str, words: int, device: torch.device) -> torch.Tensor:
    """Counter state `s` serves the first stream that uses it (recorded on
    the tensor, so copies of a Layout agree); any other stream gets a state
    of its own, kept on `s` and zeroed when first needed."""
    _need(s, name, torch.int64, (words,))
    if s.device != device:
        raise EPError(f"the layout's {name} must be on the call's device")
    key = torch.cuda.current_stream(device).cuda_stream
    home = getattr(s, "_ep_home_stream", None)
    if home is None:
        s._ep_home_stream = home = key
    if key == home:
        return s
    others = s.__dict__.setdefault("_ep_other_streams", {})
    if key not in others:
        others[key] = torch.zeros(words, dtype=torch.int64, device=device)
    return others[key]


def sched_for(layout, device: torch.device) -> torch.Tensor | None:
    """The scheduling counters that a combine through `layout` on the current
    stream uses (see _per_stream).  None: the layout asks for the static
    schedule."""
    s = layout.sched
    return None if s is None else _per_stream(s, "sched", COMBINE_SCHED_WORDS, device)


def fused_fits(num_tokens: int, num_ranks: int, num_experts: int) -> bool:
    """True if layout_dispatch (one launch) applies to the batch."""
    return bool(lib().ep_layout_dispatch_fused_fits(num_tokens, num_ranks, num_experts))


def layout_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                    num_experts: int, num_ranks: int, *, use_fp8: bool = False,
                    capacity: int | None = None, err: torch.Tensor | None = None,
                    layout: Layout | None = None,
                    out: Dispatched | None = None) -> tuple[Layout, Dispatched]:
    """get_dispatch_layout and dispatch in one kernel launch (small batches:
    fused_fits).  Same outputs as the two calls.  Enqueued on the current
    stream."""
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    _need(topk_idx, "topk_idx", torch.int64)
    K = topk_idx.shape[1]
    _need(topk_idx, "topk_idx", torch.int64, (T, K))
    _need(topk_weights, "topk_weights", torch.float32, (T, K))
    R, E = num_ranks, num_experts
    L = layout if layout is not None else alloc_layout(T, E, R, x.device)
    _need(L.slot, "slot", torch.int32, (T, R))
    if L.fused_sync is None:
        raise EPError("the layout has no fused_sync state")
    sync = _per_stream(L.fused_sync, "fused_sync", FUSED_SYNC_WORDS, x.device)
    if out is None:
        cap = capacity if capacity is not None else worst_case_rows(T, K, R)
        out = alloc_dispatched(cap, H, K, E, R, use_fp8, x.device)
    elif out.use_fp8 != use_fp8:
        raise EPError("preallocated dispatch buffers have the wrong payload type")
    if err is not None:
        _need(err, "err", torch.int32)
    _check(lib().ep_layout_dispatch_fused(
        _ptr(x), H, _ptr(topk_idx), _ptr(topk_weights), T, K, E, R,
        _ptr(L.num_tokens_per_rank), _ptr(L.num_tokens_per_expert), _ptr(L.is_token_in_rank),
        _ptr(L.slot), _ptr(L.recv_base), out.recv_x.shape[0], int(use_fp8), _ptr(out.recv_x),
        _ptr(out.recv_scales), _ptr(out.recv_src_idx), _ptr(out.recv_topk_idx),
        _ptr(out.recv_topk_weights), _ptr(out.num_recv_tokens_per_expert), _ptr(L.workspace),
        L.workspace.numel(), _ptr(sync), _ptr(err), _stream(x.device)),
        "ep_layout_dispatch_fused")
    _debug_check("layout_dispatch", err, x.device)
    return L, out


def combine(y: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor | None,
            layout: Layout, *, err: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = bf16(sum_k w[t][k] * y[slot[t][rank(e_k)]]) accumulated in
    float32; with topk_weights=None, the unweighted sum of the token's
    destination-rank rows (each rank once).  Enqueued on the current stream."""
    _need(y, "y", torch.bfloat16)
    H = y.shape[1]
    T, K = topk_idx.shape
    _need(topk_idx, "topk_idx", torch.int64, (T, K))
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, (T, K))
    R, E = layout.num_ranks, layout.num_experts
    _need(layout.slot, "slot", torch.int32, (T, R))
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _need(out, "out", torch.bfloat16, (T, H))
    if err is not None:
        _need(err, "err", torch.int32)
    sched = sched_for(layout, y.device)
    _check(lib().ep_combine_sched(_ptr(y), H, _ptr(topk_idx), _ptr(topk_weights), T, K, E, R,
                                  _ptr(layout.slot), _ptr(out), _ptr(sched), _ptr(err),
                                  _stream(y.device)), "ep_combine_sched")
    _debug_check("combine", err, y.device)
    return out


# --------------------------------------------------------------------------
# sharded form: one rank's own tokens (the exchange is in .sharded)
# --------------------------------------------------------------------------
@dataclass
class ShardLayout:
    """Outputs of shard_layout (all on the device)."""
    send_counts: torch.Tensor       # [R] int32: tokens sent to each destination rank
    expert_counts: torch.Tensor     # [E] int32: slots naming each expert
    is_token_in_rank: torch.Tensor  # [T, R] bool
    send_slot: torch.Tensor         # [T, R] int32: row in the send buffer, -1 = not sent
    send_base: torch.Tensor         # [R + 1] int32: destination r's run starts here
    num_experts: int
    num_ranks: int
    workspace: torch.Tensor | None = None
    sched: torch.Tensor | None = None  # the local combine's counters (as Layout.sched)

    @property
    def slot(self) -> torch.Tensor:  # dispatch and combine read the send slots as slots
        return self.send_slot


def alloc_shard_layout(num_tokens: int, num_experts: int, num_ranks: int,
                       device: torch.device) -> ShardLayout:
    T, R, E = num_tokens, num_ranks, num_experts
    i32 = dict(dtype=torch.int32, device=device)
    ws = torch.empty(max(int(lib().ep_shard_workspace_bytes(T, R, E)), 16), dtype=torch.uint8,
                     device=device)
    return ShardLayout(torch.empty(R, **i32), torch.empty(E, **i32),
                       torch.empty((T, R), dtype=torch.bool, device=device),
                       torch.empty((T, R), **i32), torch.empty(R + 1, **i32), E, R, ws,
                       alloc_combine_sched(device))


def shard_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int, *,
                 err: torch.Tensor | None = None, out: ShardLayout | None = None) -> ShardLayout:
    """One rank's layout of its own tokens over num_ranks destinations (any
    number of tokens): its send buffer is packed destination-major in token
    order.  Enqueued on the current stream."""
    _need(topk_idx, "topk_idx", torch.int64)
    if topk_idx.dim() != 2:
        raise EPError("topk_idx must be [num_tokens, num_topk]")
    T, K = topk_idx.shape
    L = out if out is not None else alloc_shard_layout(T, num_experts, num_ranks,
                                                       topk_idx.device)
    if err is not None:
        _need(err, "err", torch.int32)
    _check(lib().ep_shard_layout(_ptr(topk_idx), T, K, num_experts, num_ranks,
                                 _ptr(L.send_counts), _ptr(L.expert_counts),
                                 _ptr(L.is_token_in_rank), _ptr(L.send_slot), _ptr(L.send_base),
                                 _ptr(err), _ptr(L.workspace), L.workspace.numel(),
                                 _stream(topk_idx.device)), "ep_shard_layout")
    _debug_check("shard_layout", err, topk_idx.device)
    return L


def shard_offsets(counts: np.ndarray, rank: int) -> tuple[np.ndarray, np.ndarray]:
    """Host: from the gathered counts [R, R] (counts[s][r] = tokens of rank s
    sent to rank r), this rank's send offsets (its runs in its send buffer)
    and receive offsets (where each source's run lands), both [R + 1] int64."""
    c = np.ascontiguousarray(counts, dtype=np.int32)
    R = c.shape[0]
    if c.shape != (R, R):
        raise EPError("counts must be [R, R]")
    send = np.empty(R + 1, np.int64)
    recv = np.empty(R + 1, np.int64)
    _check(lib().ep_shard_offsets(c.ctypes.data, R, rank, send.ctypes.data, recv.ctypes.data),
           "ep_shard_offsets")
    return send, recv


def shard_recv_tokens_per_expert(expert_counts: np.ndarray, rank: int) -> np.ndarray:
    """Host: from every rank's expert counts [R, E], the rows this rank
    receives per local expert, [E / R] int32."""
    c = np.ascontiguousarray(expert_counts, dtype=np.int32)
    R, E = c.shape
    out = np.empty(E // R if R and E % R == 0 else 0, np.int32)
    _check(lib().ep_shard_recv_tokens_per_expert(c.ctypes.data, E, R, rank, out.ctypes.data),
           "ep_shard_recv_tokens_per_expert")
    return out


# --------------------------------------------------------------------------
# low-latency (expert-major) layout
# --------------------------------------------------------------------------
@dataclass
class LLLayout:
    """Outputs of ll_get_dispatch_layout (all on the device)."""
    ll_slot: torch.Tensor        # [T, K] int32: row of each slot, -1 = none
    ll_count: torch.Tensor       # [E] int32: rows each expert receives
    ll_src_offset: torch.Tensor  # [E, R] int32: first row of each source within its expert
    num_experts: int
    num_ranks: int
    expert_capacity: int
    workspace: torch.Tensor | None = None
    sched: torch.Tensor | None = None  # as Layout.sched

    @property
    def num_rows(self) -> int:
        """Rows of the expert-major buffer: E * expert_capacity."""
        return self.num_experts * self.expert_capacity


def alloc_ll_layout(num_tokens: int, num_topk: int, num_experts: int, num_ranks: int,
                    expert_capacity: int, device: torch.device) -> LLLayout:
    ws = torch.empty(max(int(lib().ep_ll_workspace_bytes(num_tokens, num_ranks, num_experts)), 16),
                     dtype=torch.uint8, device=device)
    return LLLayout(torch.empty((num_tokens, num_topk), dtype=torch.int32, device=device),
                    torch.empty(num_experts, dtype=torch.int32, device=device),
                    torch.empty((num_experts, num_ranks), dtype=torch.int32, device=device),
                    num_experts, num_ranks, int(expert_capacity), ws,
                    alloc_combine_sched(device))


def ll_single_launch_fits(num_tokens: int, num_topk: int, num_ranks: int,
                          num_experts: int) -> bool:
    """True if the one-launch (thread-block cluster) expert-major layout applies."""
    return bool(lib().ep_ll_layout_single_launch_fits(num_tokens, num_topk, num_ranks,
                                                      num_experts))


def ll_auto_single_launch(num_tokens: int, num_topk: int, num_ranks: int,
                          num_experts: int) -> bool:
    """True if path="auto" takes the one-launch expert-major layout."""
    return bool(lib().ep_ll_layout_auto_single_launch(num_tokens, num_topk, num_ranks,
                                                      num_experts))


def ll_get_dispatch_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int,
                           expert_capacity: int | None = None, *,
                           err: torch.Tensor | None = None,
                           out: LLLayout | None = None, path: str = "auto") -> LLLayout:
    """Rows of the expert-major layout (default capacity: T rows per expert).
    path: "auto", "multi" or "single" (one cluster launch, small batches)."""
    _need(topk_idx, "topk_idx", torch.int64)
    if path not in LAYOUT_PATHS:
        raise EPError(f"path must be one of {sorted(LAYOUT_PATHS)}")
    T, K = topk_idx.shape
    if out is not None:
        L = out
        cap = L.expert_capacity
    else:
        cap = T if expert_capacity is None else int(expert_capacity)
        L = alloc_ll_layout(T, K, num_experts, num_ranks, cap, topk_idx.device)
    dev = topk_idx.device
    ws = L.workspace
    if err is not None:
        _need(err, "err", torch.int32)
    args = (_ptr(topk_idx), T, K, num_experts, num_ranks, cap, _ptr(L.ll_slot),
            _ptr(L.ll_count), _ptr(L.ll_src_offset), _ptr(err), _ptr(ws), ws.numel())
    if path == "auto":
        _check(lib().ep_ll_get_dispatch_layout(*args, _stream(dev)), "ep_ll_get_dispatch_layout")
    else:
        _check(lib().ep_ll_get_dispatch_layout_path(*args, LAYOUT_PATHS[path], _stream(dev)),
               "ep_ll_get_dispatch_layout_path")
    _debug_check("ll_get_dispatch_layout", err, dev)
    return L


@dataclass
class LLDispatched:
    recv_x: torch.Tensor              # [E*cap, H] bf16 or uint8 (E4M3)
    recv_scales: torch.Tensor | None  # [E*cap, H/128] float32 (FP8 only)
    recv_src_idx: torch.Tensor        # [E*cap] int32
    use_fp8: bool


def ll_dispatch(x: torch.Tensor, layout: LLLayout, *, use_fp8: bool = False,
                err: torch.Tensor | None = None, out: LLDispatched | None = None) -> LLDispatched:
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    K = layout.ll_slot.shape[1]
    _need(layout.ll_slot, "ll_slot", torch.int32, (T, K))
    rows = layout.num_rows
    if out is None:
        dev = x.device
        out = LLDispatched(
            torch.empty((rows, H), dtype=torch.uint8 if use_fp8 else torch.bfloat16, device=dev),
            torch.empty((rows, H // 128), dtype=torch.float32, device=dev) if use_fp8 else None,
            torch.empty(rows, dtype=torch.int32, device=dev), use_fp8)
    if err is not None:
        _need(err, "err", torch.int32)
    _check(lib().ep_ll_dispatch(_ptr(x), H, T, K, _ptr(layout.ll_slot), out.recv_x.shape[0],
                                int(use_fp8), _ptr(out.recv_x), _ptr(out.recv_scales),
                                _ptr(out.recv_src_idx), _ptr(err), _stream(x.device)),
           "ep_ll_dispatch")
    _debug_check("ll_dispatch", err, x.device)
    return out


def ll_combine(y: torch.Tensor, topk_weights: torch.Tensor | None, layout: LLLayout, *,
               err: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    _need(y, "y", torch.bfloat16)
    H = y.shape[1]
    T, K = layout.ll_slot.shape
    if y.shape[0] < layout.num_rows:
        raise EPError(f"y must have the layout's {layout.num_rows} rows (E * capacity), "
                      f"got {y.shape[0]}")
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, (T, K))
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _need(out, "out", torch.bfloat16, (T, H))
    if err is not None:
        _need(err, "err", torch.int32)
    sched = sched_for(layout, y.device)
    _check(lib().ep_ll_combine_sched(_ptr(y), H, _ptr(topk_weights), T, K, _ptr(layout.ll_slot),
                                     _ptr(out), _ptr(sched), _ptr(err), _stream(y.device)),
           "ep_ll_combine_sched")
    _debug_check("ll_combine", err, y.device)
    return out


def debug_e4m3_range(first: int, out: torch.Tensor) -> None:
    """Test hook: out[i] = the FP8 dispatch's E4M3 code for the float32 with
    bit pattern first + i (out: uint8, a multiple of 4 elements).  Enqueued on
    the current stream."""
    _need(out, "out", torch.uint8)
    _check(lib().ep_debug_e4m3_range(int(first), out.numel(), _ptr(out), _stream(out.device)),
           "ep_debug_e4m3_range")


# --------------------------------------------------------------------------
# the router and its gradient
# --------------------------------------------------------------------------
def _need_logits(logits: torch.Tensor) -> int:
    """Checks router logits (rows may be strided); returns the row stride."""
    if not logits.is_cuda:
        raise EPError("logits must be a CUDA tensor")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise EPError(f"logits must be torch.float32 or torch.bfloat16, got {logits.dtype}")
    if logits.dim() != 2:
        raise EPError("logits must be [num_tokens, num_experts]")
    T, E = logits.shape
    if E > 1 and logits.stride(1) != 1:
        raise EPError("logits must be contiguous along the experts")
    stride = logits.stride(0) if T > 1 else E
    if stride < E:
        raise EPError("the rows of logits must not overlap")
    return stride


def _enum(table: dict, value: str, name: str) -> int:
    if value not in table:
        raise EPError(f"{name} must be one of {sorted(table)}")
    return table[value]


def route(logits: torch.Tensor, num_topk: int, *, score: str = "softmax",
          bias: torch.Tensor | None = None, num_groups: int = 1, topk_groups: int = 1,
          renormalize: bool = True, scale: float = 1.0,
          out: tuple[torch.Tensor, torch.Tensor] | None = None
          ) -> tuple[torch.Tensor, torch.Tensor]:
    """Router: the top-k experts of every token and their weights, (topk_idx
    [T, K] int64, topk_weights [T, K] float32), from logits [T, E] (float32 or
    bfloat16).  score: "softmax" or "sigmoid"; bias [E] steers the choice and
    stays out of the weights; num_groups / topk_groups restrict it to the best
    groups of consecutive experts.  Ties go to the lowest index; experts at
    -inf or NaN are never chosen.  Enqueued on the current stream."""
    stride = _need_logits(logits)
    T, E = logits.shape
    K = int(num_topk)
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,))
    if out is None:
        out = (torch.empty((T, K), dtype=torch.int64, device=logits.device),
               torch.empty((T, K), dtype=torch.float32, device=logits.device))
    else:
        _need(out[0], "out[0]", torch.int64, (T, K))
        _need(out[1], "out[1]", torch.float32, (T, K))
    _check(lib().ep_route(_ptr(logits), int(logits.dtype == torch.bfloat16), stride, _ptr(bias), T,
                          E, K, _enum(SCORES, score, "score"), int(num_groups), int(topk_groups),
                          int(renormalize), float(scale), _ptr(out[0]), _ptr(out[1]),
                          _stream(logits.device)), "ep_route")
    _debug_check("route", None, logits.device)
    return out


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor, *,
                   score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                   err: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of route's weights with respect to the logits, [T, E] of the
    logits' type, at the choice topk_idx.  Enqueued on the current stream."""
    stride = _need_logits(logits)
    T, E = logits.shape
    if topk_idx.dim() != 2:
        raise EPError("topk_idx must be [num_tokens, num_topk]")
    K = topk_idx.shape[1]
    _need(topk_idx, "topk_idx", torch.int64, (T, K))
    _need(dweights, "dweights", torch.float32, (T, K))
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    _need(out, "out", logits.dtype, (T, E))
    if err is not None:
        _need(err, "err", torch.int32)
    _check(lib().ep_route_backward(_ptr(dweights), _ptr(logits),
                                   int(logits.dtype == torch.bfloat16), stride, _ptr(topk_idx), T,
                                   E, K, _enum(SCORES, score, "score"), int(renormalize),
                                   float(scale), _ptr(out), _ptr(err), _stream(logits.device)),
           "ep_route_backward")
    _debug_check("route_backward", err, logits.device)
    return out


# --------------------------------------------------------------------------
# the gradient of the combine
# --------------------------------------------------------------------------
def _grad_outputs(dout, y, T, K, out):
    _need(dout, "dout", torch.bfloat16)
    _need(y, "y", torch.bfloat16)
    if dout.dim() != 2 or y.dim() != 2 or y.shape[1] != dout.shape[1]:
        raise EPError("dout must be [num_tokens, hidden] and y [rows, hidden]")
    if dout.shape[0] != T:
        raise EPError(f"dout must have {T} rows, got {dout.shape[0]}")
    if out is None:  # rows that no slot names get no gradient
        out = torch.zeros_like(y)
    _need(out, "out", torch.bfloat16, y.shape)
    return out, torch.empty((T, K), dtype=torch.float32, device=y.device)


def combine_backward(dout: torch.Tensor, y: torch.Tensor, topk_idx: torch.Tensor,
                     topk_weights: torch.Tensor, layout: Layout, *,
                     err: torch.Tensor | None = None, out: torch.Tensor | None = None
                     ) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of combine(y, topk_idx, topk_weights, layout) for the gradient
    dout [T, H] of its output: (dy like y, dweights [T, K] float32).  Rows of
    dy that no slot names keep what `out` holds (zeros without `out`, at the
    cost of writing all of dy first).
    Enqueued on the current stream."""
    if topk_idx.dim() != 2:
        raise EPError("topk_idx must be [num_tokens, num_topk]")
    T, K = topk_idx.shape
    dy, dw = _grad_outputs(dout, y, T, K, out)
    _need(topk_idx, "topk_idx", torch.int64, (T, K))
    _need(topk_weights, "topk_weights", torch.float32, (T, K))
    R, E = layout.num_ranks, layout.num_experts
    _need(layout.slot, "slot", torch.int32, (T, R))
    if err is not None:
        _need(err, "err", torch.int32)
    _check(lib().ep_combine_backward(_ptr(dout), _ptr(y), y.shape[1], y.shape[0], _ptr(topk_idx),
                                     _ptr(topk_weights), T, K, E, R, _ptr(layout.slot), _ptr(dy),
                                     _ptr(dw), _ptr(err), _stream(y.device)),
           "ep_combine_backward")
    _debug_check("combine_backward", err, y.device)
    return dy, dw


def ll_combine_backward(dout: torch.Tensor, y: torch.Tensor, topk_weights: torch.Tensor,
                        layout: LLLayout, *, err: torch.Tensor | None = None,
                        out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of ll_combine(y, topk_weights, layout): (dy like y, dweights
    [T, K] float32), as combine_backward.  Enqueued on the current stream."""
    T, K = layout.ll_slot.shape
    dy, dw = _grad_outputs(dout, y, T, K, out)
    _need(layout.ll_slot, "ll_slot", torch.int32, (T, K))
    _need(topk_weights, "topk_weights", torch.float32, (T, K))
    if err is not None:
        _need(err, "err", torch.int32)
    _check(lib().ep_ll_combine_backward(_ptr(dout), _ptr(y), y.shape[1], y.shape[0],
                                        _ptr(topk_weights), T, K, _ptr(layout.ll_slot), _ptr(dy),
                                        _ptr(dw), _ptr(err), _stream(y.device)),
           "ep_ll_combine_backward")
    _debug_check("ll_combine_backward", err, y.device)
    return dy, dw


# --------------------------------------------------------------------------
# the experts' products with 4-bit weights
# --------------------------------------------------------------------------
@dataclass
class W4Weights:
    """4-bit weights of E experts: W[e][n][i] = (q - zero) * scale, one scale
    and zero point per group of consecutive input channels."""
    q: torch.Tensor             # [E, N', I / 2] uint8, channel 2j low half, 2j + 1 high half of byte j
    scales: torch.Tensor        # [E, N', I / group] bfloat16
    zeros: torch.Tensor | None = None  # [E, N', I / group] uint8, the low four bits; None: 8 everywhere


def quantize_w4(weight: torch.Tensor, group_size: int = 128, *,
                zero_points: bool = False) -> W4Weights:
    """Rounds weights [E, N', I] to W4Weights, on the weights' device (set-up
    work in torch, once per model).  Without zero points the scale maps a
    group's largest magnitude to 7; with them, its range to [0, 15]."""
    if group_size not in (32, 64, 128) or weight.dim() != 3 or weight.shape[2] % group_size:
        raise EPError("weight must be [E, N, I] with I a multiple of group_size (32, 64 or 128)")
    E, N, I = weight.shape
    w = weight.float().reshape(E, N, I // group_size, group_size)
    if zero_points:
        lo, hi = w.amin(-1).clamp(max=0.0), w.amax(-1).clamp(min=0.0)
        scales = ((hi - lo) / 15.0).clamp(min=1e-8).to(torch.bfloat16)
        zero = torch.round(-lo / scales.float()).clamp(0, 15)
    else:
        scales = (w.abs().amax(-1) / 7.0).clamp(min=1e-8).to(torch.bfloat16)
        zero = torch.full_like(scales, 8.0, dtype=torch.float32)
    q = (torch.round(w / scales.float()[..., None]) + zero[..., None]).clamp(0, 15)
    q = q.to(torch.uint8).reshape(E, N, I // 2, 2)
    return W4Weights((q[..., 0] | (q[..., 1] << 4)).contiguous(), scales,
                     zero.to(torch.uint8) if zero_points else None)


def ll_experts_w4(x: torch.Tensor, weights: W4Weights, layout: LLLayout, *,
                  x_scales: torch.Tensor | None = None, act: str = "none",
                  err: torch.Tensor | None = None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Every expert's product with its rows of the expert-major layout: x
    [E * cap, I] bfloat16, or E4M3 codes (uint8) with x_scales [E * cap, I /
    128] as ll_dispatch leaves them; returns [E * cap, N] bfloat16.  act
    "swiglu": the weights' first N rows are the gate's, the next N the up
    projection's.  Rows beyond an expert's count keep what `out` holds
    (nothing defined without `out`).  Enqueued on the current stream."""
    E, cap = layout.num_experts, layout.expert_capacity
    fp8 = x_scales is not None
    a = _enum(ACTS, act, "act")
    _need(weights.q, "weights.q", torch.uint8)
    _need(weights.scales, "weights.scales", torch.bfloat16)
    if weights.q.dim() != 3 or weights.scales.dim() != 3 or weights.q.shape[0] != E:
        raise EPError(f"weights.q must be [{E}, N, I / 2] and weights.scales [{E}, N, I / group]")
    rows, I = weights.q.shape[1], 2 * weights.q.shape[2]
    groups = weights.scales.shape[2]
    if tuple(weights.scales.shape[:2]) != (E, rows) or groups == 0 or I % groups:
        raise EPError("weights.scales must have one value per group of input channels")
    if weights.zeros is not None:
        _need(weights.zeros, "weights.zeros", torch.uint8, weights.scales.shape)
    if a and rows % 2:
        raise EPError("swiglu weights have 2 N rows")
    N = rows // 2 if a else rows
    _need(x, "x", torch.uint8 if fp8 else torch.bfloat16, (E * cap, I))
    if fp8:
        _need(x_scales, "x_scales", torch.float32, (E * cap, I // 128))
    _need(layout.ll_count, "ll_count", torch.int32, (E,))
    if out is None:
        out = torch.empty((E * cap, N), dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, (E * cap, N))
    if err is not None:
        _need(err, "err", torch.int32)
    _check(lib().ep_ll_experts_w4(_ptr(x), int(fp8), _ptr(x_scales), I, _ptr(layout.ll_count), E,
                                  cap, _ptr(weights.q), _ptr(weights.scales), _ptr(weights.zeros),
                                  I // groups, N, a, _ptr(out), _ptr(err), _stream(x.device)),
           "ep_ll_experts_w4")
    _debug_check("ll_experts_w4", err, x.device)
    return out


# --------------------------------------------------------------------------
# a whole layer for a few tokens
# --------------------------------------------------------------------------
# The current device's index without torch's check that CUDA is initialised (which
# a CUDA tensor shows), where torch offers it.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _same_device(first: torch.Tensor, *others: torch.Tensor | None) -> torch.device:
    """The tensors' device, which has to be the current one: a kernel launched on another
    device's stream would run where its buffers are not."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise EPError(f"tensors are on different devices ({first.device} and {t.device})")
    if index >= 0 and _current_device() != index:
        raise EPError(f"tensors are on {first.device}, but the current device is "
                      f"cuda:{_current_device()}")
    return first.device


def _need_rows(t: torch.Tensor, name: str, layout: LLLayout):
    if t.shape[0] < layout.num_rows:
        raise EPError(f"{name} must have the layout's {layout.num_rows} rows (E * capacity), "
                      f"got {t.shape[0]}")


def _w4_shape(w: W4Weights, name: str, experts: int) -> tuple[int, int, int]:
    """Checks 4-bit weights; returns their rows, input channels and group size."""
    _need(w.q, f"{name}.q", torch.uint8)
    _need(w.scales, f"{name}.scales", torch.bfloat16)
    if w.q.dim() != 3 or w.scales.dim() != 3 or w.q.shape[0] != experts:
        raise EPError(f"{name}.q must be [{experts}, N, I / 2] and {name}.scales "
                      f"[{experts}, N, I / group]")
    rows, inner, groups = w.q.shape[1], 2 * w.q.shape[2], w.scales.shape[2]
    if tuple(w.scales.shape[:2]) != (experts, rows) or groups == 0 or inner % groups:
        raise EPError(f"{name}.scales must have one value per group of input channels")
    if w.zeros is not None:
        _need(w.zeros, f"{name}.zeros", torch.uint8, w.scales.shape)
    return rows, inner, inner // groups


def layer_w4(x: torch.Tensor, logits: torch.Tensor, gate_up: W4Weights, down: W4Weights,
             num_topk: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
             num_groups: int = 1, topk_groups: int = 1, renormalize: bool = True,
             scale: float = 1.0, out: torch.Tensor | None = None
             ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """A whole mixture-of-experts layer for a few tokens (at most
    EP_LAYER_MAX_TOKENS), in two launches: the choice of route(logits, ...), both
    products of the chosen experts (gate_up [E, 2 N, H], down [E, H, N]) with SwiGLU
    between them, and the weighted sum over the experts.  x [T, H] bfloat16;
    returns (out [T, H] bfloat16, topk_idx [T, K] int64, topk_weights [T, K]
    float32).  `out` may be x.  Enqueued on the current stream."""
    _need(x, "x", torch.bfloat16)
    stride = _need_logits(logits)
    T, E = logits.shape
    if x.dim() != 2 or x.shape[0] != T:
        raise EPError(f"x must be [{T}, hidden], a row for each row of logits")
    H, K = x.shape[1], int(num_topk)
    if T > EP_LAYER_MAX_TOKENS or E > EP_LAYER_MAX_EXPERTS:
        raise EPError(f"layer_w4 takes at most {EP_LAYER_MAX_TOKENS} tokens and "
                      f"{EP_LAYER_MAX_EXPERTS} experts, got {T} and {E}")
    rows, inner, group = _w4_shape(gate_up, "gate_up", E)
    rows2, N, group2 = _w4_shape(down, "down", E)
    if inner != H or rows2 != H or rows != 2 * N:
        raise EPError(f"gate_up must be weights of [{E}, 2 N, {H}] and down of [{E}, {H}, N], got "
                      f"{(E, rows, inner)} and {(E, rows2, N)}")
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,))
    dev = _same_device(x, logits, gate_up.q, gate_up.scales, gate_up.zeros, down.q, down.scales,
                       down.zeros, bias, out)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, (T, H))
    idx = torch.empty((T, K), dtype=torch.int64, device=dev)
    w = torch.empty((T, K), dtype=torch.float32, device=dev)
    n = lib().ep_layer_w4_workspace_bytes(T, N, K)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _check(lib().ep_layer_w4(
        x.data_ptr(), H, N, T, logits.data_ptr(), int(logits.dtype == torch.bfloat16), stride,
        _ptr(bias), E, K, _enum(SCORES, score, "score"), int(num_groups), int(topk_groups),
        int(renormalize), float(scale), gate_up.q.data_ptr(), gate_up.scales.data_ptr(),
        _ptr(gate_up.zeros), group, down.q.data_ptr(), down.scales.data_ptr(), _ptr(down.zeros),
        group2, idx.data_ptr(), w.data_ptr(), out.data_ptr(), ws.data_ptr(), n, _stream(dev)),
        "ep_layer_w4")
    _debug_check("layer_w4", None, dev)
    return out, idx, w


# --------------------------------------------------------------------------
# between two blocks: norms, gate, residual scale
# --------------------------------------------------------------------------
@dataclass
class BlockNorm:
    """Outputs of block_norm and ll_combine_norm."""
    z: torch.Tensor | None         # [T, H] of the stream's type: the stream after the block
    h: torch.Tensor | None         # [T, H] bfloat16: the next block's input
    y: torch.Tensor | None = None  # [T, H] bfloat16: the combined rows (ll_combine_norm, save=True)


@dataclass
class BlockNormGrad:
    """Outputs of block_norm_backward (None: nothing to differentiate)."""
    dx: torch.Tensor                    # [T, H] of the stream's type
    dy: torch.Tensor                    # [T, H] bfloat16
    dgate: torch.Tensor | None          # the gate's shape; float32, or a [T, H] gate's own type
    dpost_weight: torch.Tensor | None   # [H] float32
    dpre_weight: torch.Tensor | None    # [H] float32


_STREAMS = (torch.bfloat16, torch.float32)


def _norm_arguments(x, gate, post_weight, pre_weight):
    """Checks what both directions take; returns T, H, the gate's kind and whether
    gate and weights are bfloat16."""
    if x.dtype not in _STREAMS:
        raise EPError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    _need(x, "x", x.dtype)
    if x.dim() != 2:
        raise EPError("x must be [num_tokens, hidden]")
    T, H = x.shape
    if H % 8 or not 8 <= H <= EP_NORM_MAX_HIDDEN:
        raise EPError(f"hidden must be a multiple of 8 and at most {EP_NORM_MAX_HIDDEN}, got {H}")
    kind, dtype = GATE_NONE, None
    if post_weight is not None:
        dtype = post_weight.dtype
        _need(post_weight, "post_weight", dtype, (H,))
    if pre_weight is not None:
        dtype = dtype or pre_weight.dtype
        _need(pre_weight, "pre_weight", dtype, (H,))
    if gate is not None:
        dtype = dtype or gate.dtype
        _need(gate, "gate", dtype)
        shape = gate.shape
        if shape == (H,):
            kind = GATE_CHANNEL
        elif shape == (T, 1):
            kind = GATE_TOKEN
        elif shape == (T, H):
            kind = GATE_FULL
        else:
            raise EPError(f"gate must be [{H}], [{T}, 1] or [{T}, {H}], got {list(shape)}")
    if dtype is not None and dtype not in _STREAMS:
        raise EPError("gate and weights must be torch.bfloat16 or torch.float32, got "
                      f"{dtype}")
    return T, H, kind, int(dtype == torch.bfloat16)


def _block_norm(x, y, rows, topk_weights, slot, gate, post_weight, pre_weight, scale, eps, save,
                err, out):
    T, H, kind, bf16 = _norm_arguments(x, gate, post_weight, pre_weight)
    if err is not None:
        _need(err, "err", torch.int32)
    dev = _same_device(x, y, topk_weights, slot, gate, post_weight, pre_weight, err, out)
    z = None
    if y is not None:
        z = torch.empty_like(x) if out is None else out
        _need(z, "out", x.dtype, (T, H))
    elif out is not None:
        raise EPError("without y there is no new stream to write")
    h = c = None
    if pre_weight is not None:
        h = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if save:
        c = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _check(lib().ep_block_norm(
        x.data_ptr(), int(x.dtype == torch.float32), _ptr(y), rows, _ptr(topk_weights),
        0 if slot is None else slot.shape[1], _ptr(slot), T, H, _ptr(gate), kind,
        _ptr(post_weight), _ptr(pre_weight), bf16, float(scale), float(eps), _ptr(z), _ptr(h),
        _ptr(c), _ptr(err), _stream(dev)), "ep_block_norm")
    return BlockNorm(z, h, c)


def block_norm(x: torch.Tensor, y: torch.Tensor | None = None, *,
               gate: torch.Tensor | None = None, post_weight: torch.Tensor | None = None,
               pre_weight: torch.Tensor | None = None, scale: float = 1.0, eps: float = 1e-6,
               out: torch.Tensor | None = None) -> BlockNorm:
    """Between two blocks: z = x + scale * gate * norm(y) and h = norm(z), in one
    pass.  x [T, H] is the residual stream (bfloat16 or float32), y [T, H] bfloat16 the
    block's output (None: only h = norm(x)); norm(y) is y / rms(y) *
    post_weight, or y without a post_weight; h = z / rms(z) * pre_weight, None without a
    pre_weight.  gate: [H], [T, 1] or [T, H]; gate and weights are all
    float32 or all bfloat16.  `out` takes z and may be x.  Enqueued on the current stream."""
    if y is None and (gate is not None or post_weight is not None):
        raise EPError("gate and post_weight belong to a block's output y")
    if y is None and pre_weight is None:
        raise EPError("nothing to compute without y and without pre_weight")
    if y is not None:
        _need(y, "y", torch.bfloat16, x.shape)
    r = _block_norm(x, y, 0, None, None, gate, post_weight, pre_weight, scale, eps, False,
                    None, out)
    _debug_check("block_norm", None, x.device)
    return r


def ll_combine_norm(y: torch.Tensor, topk_weights: torch.Tensor | None, layout: LLLayout,
                    x: torch.Tensor, *, gate: torch.Tensor | None = None,
                    post_weight: torch.Tensor | None = None,
                    pre_weight: torch.Tensor | None = None, scale: float = 1.0, eps: float = 1e-6,
                    save: bool = False, err: torch.Tensor | None = None,
                    out: torch.Tensor | None = None) -> BlockNorm:
    """block_norm(x, ll_combine(y, topk_weights, layout), ...) in one pass over the
    experts' rows y [E * cap, H].  save: the combined rows are returned too, as
    block_norm_backward and ll_combine_backward need them.  Enqueued on the current stream."""
    _need(y, "y", torch.bfloat16)
    T, K = layout.ll_slot.shape
    _need(layout.ll_slot, "ll_slot", torch.int32, (T, K))
    if x.dim() != 2 or y.dim() != 2 or x.shape[0] != T or x.shape[1] != y.shape[1]:
        raise EPError(f"x must be [{T}, hidden] and y [rows, hidden]")
    _need_rows(y, "y", layout)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, (T, K))
    r = _block_norm(x, y, y.shape[0], topk_weights, layout.ll_slot, gate, post_weight, pre_weight,
                    scale, eps, save, err, out)
    _debug_check("ll_combine_norm", err, y.device)
    return r


def block_norm_backward(dz: torch.Tensor | None, dh: torch.Tensor | None, z: torch.Tensor,
                        y: torch.Tensor | None = None, *, gate: torch.Tensor | None = None,
                        post_weight: torch.Tensor | None = None,
                        pre_weight: torch.Tensor | None = None, scale: float = 1.0,
                        eps: float = 1e-6) -> BlockNormGrad:
    """Gradient of block_norm for the gradients dz of z (the stream's type) and dh
    of h (bfloat16), at the stored z and y.  Either gradient may be None (zero); dh goes
    with pre_weight, and y is needed with a post_weight or a gate.
    Enqueued on the current stream."""
    T, H, kind, bf16 = _norm_arguments(z, gate, post_weight, pre_weight)
    if dz is None and dh is None:
        raise EPError("one of dz and dh is needed")
    if (dh is None) != (pre_weight is None):
        raise EPError("dh is the gradient of the norm with pre_weight: both or neither")
    if dz is not None:
        _need(dz, "dz", z.dtype, (T, H))
    if dh is not None:
        _need(dh, "dh", torch.bfloat16, (T, H))
    if y is not None:
        _need(y, "y", torch.bfloat16, (T, H))
    elif post_weight is not None or gate is not None:
        raise EPError("the gradients of gate and post_weight need y")
    dev = _same_device(z, dz, dh, y, gate, post_weight, pre_weight)
    f32 = dict(dtype=torch.float32, device=dev)
    dx = torch.empty((T, H), dtype=z.dtype, device=dev)
    dy = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    dpost = None if post_weight is None else torch.empty(H, **f32)
    dpre = None if pre_weight is None else torch.empty(H, **f32)
    dgate = None
    if gate is not None:
        dgate = torch.empty_like(gate) if kind == GATE_FULL else torch.empty(gate.shape, **f32)
    ws, n = None, 0
    if dpost is not None or dpre is not None or kind == GATE_CHANNEL:
        n = lib().ep_block_norm_backward_workspace_bytes(T, H)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _check(lib().ep_block_norm_backward(
        _ptr(dz), _ptr(dh), z.data_ptr(), int(z.dtype == torch.float32), _ptr(y), T, H, _ptr(gate),
        kind, _ptr(post_weight), _ptr(pre_weight), bf16, float(scale), float(eps), dx.data_ptr(),
        dy.data_ptr(), _ptr(dgate), _ptr(dpost), _ptr(dpre), _ptr(ws), n, _stream(dev)),
        "ep_block_norm_backward")
    _debug_check("block_norm_backward", None, dev)
    return BlockNormGrad(dx, dy, dgate, dpost, dpre)


# --------------------------------------------------------------------------
# the gated activation with an 8-bit checkpoint, and its gradient
# --------------------------------------------------------------------------
@dataclass
class Checkpoint8:
    """Rows kept in 8 bits for a backward pass: E4M3 codes and one scale per 128 channels."""
    codes: torch.Tensor   # [rows, C] uint8
    scales: torch.Tensor  # [rows, C / 128] float32


def alloc_checkpoint8(rows: int, channels: int, device: torch.device) -> Checkpoint8:
    """Room for a checkpoint of [rows, channels] (channels a multiple of 128)."""
    if channels % 128:
        raise EPError(f"channels must be a multiple of 128, got {channels}")
    return Checkpoint8(torch.empty((rows, channels), dtype=torch.uint8, device=device),
                       torch.empty((rows, channels // 128), dtype=torch.float32, device=device))


def _need_checkpoint(c: Checkpoint8, rows: int, channels: int):
    if channels % 256:
        raise EPError(f"a checkpoint needs N to be a multiple of 128, got {channels // 2}")
    _need(c.codes, "checkpoint.codes", torch.uint8, (rows, channels))
    _need(c.scales, "checkpoint.scales", torch.float32, (rows, channels // 128))


def ll_swiglu(gate_up: torch.Tensor, layout: LLLayout, topk_weights: torch.Tensor | None = None, *,
              checkpoint: Checkpoint8 | None = None, err: torch.Tensor | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """Gated activation on the rows of the expert-major layout: h = w * silu(g) *
    u for the rows [g | u] of gate_up [rows, 2 N] bfloat16 that the layout's slots
    name, w the slot's top-k weight (1 without topk_weights; with them the
    combine takes none).  checkpoint (alloc_checkpoint8(rows, 2 N)) receives
    gate_up in 8 bits, for ll_swiglu_backward.  Rows that no slot names keep what `out`
    and the checkpoint hold (nothing defined without `out`).  Enqueued on the current
    stream."""
    _need(gate_up, "gate_up", torch.bfloat16)
    T, K = layout.ll_slot.shape
    _need(layout.ll_slot, "ll_slot", torch.int32, (T, K))
    if gate_up.dim() != 2 or gate_up.shape[1] % 16 or gate_up.shape[1] == 0:
        raise EPError("gate_up must be [rows, 2 N] with N a multiple of 8")
    _need_rows(gate_up, "gate_up", layout)
    rows, N = gate_up.shape[0], gate_up.shape[1] // 2
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, (T, K))
    codes = scales = None
    if checkpoint is not None:
        _need_checkpoint(checkpoint, rows, 2 * N)
        codes, scales = checkpoint.codes, checkpoint.scales
    if err is not None:
        _need(err, "err", torch.int32)
    dev = _same_device(gate_up, layout.ll_slot, topk_weights, codes, scales, err, out)
    if out is None:
        out = torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, (rows, N))
    _check(lib().ep_ll_swiglu(gate_up.data_ptr(), N, rows, _ptr(topk_weights), T, K,
                              layout.ll_slot.data_ptr(), out.data_ptr(), _ptr(codes), _ptr(scales),
                              _ptr(err), _stream(dev)), "ep_ll_swiglu")
    _debug_check("ll_swiglu", err, dev)
    return out


def ll_swiglu_backward(dh: torch.Tensor, kept: Checkpoint8 | torch.Tensor, layout: LLLayout,
                       topk_weights: torch.Tensor | None = None, *,
                       err: torch.Tensor | None = None, out: torch.Tensor | None = None
                       ) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Gradient of ll_swiglu for the gradient dh [rows, N] bfloat16 of its output:
    (dgate_up [rows, 2 N] bfloat16, dweights [T, K] float32, or None without
    topk_weights).  kept: the checkpoint, or gate_up itself.  Rows of dgate_up that
    no slot names keep what `out` holds (zeros without `out`, at the cost of writing
    all of it first).  Enqueued on the current stream."""
    _need(dh, "dh", torch.bfloat16)
    T, K = layout.ll_slot.shape
    _need(layout.ll_slot, "ll_slot", torch.int32, (T, K))
    if dh.dim() != 2 or dh.shape[1] % 8 or dh.shape[1] == 0:
        raise EPError("dh must be [rows, N] with N a multiple of 8")
    _need_rows(dh, "dh", layout)
    rows, N = dh.shape
    gate_up = codes = scales = None
    if isinstance(kept, Checkpoint8):
        _need_checkpoint(kept, rows, 2 * N)
        codes, scales = kept.codes, kept.scales
    else:
        gate_up = kept
        _need(gate_up, "gate_up", torch.bfloat16, (rows, 2 * N))
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, (T, K))
    if err is not None:
        _need(err, "err", torch.int32)
    dev = _same_device(dh, gate_up, codes, scales, layout.ll_slot, topk_weights, err, out)
    if out is None:
        out = torch.zeros((rows, 2 * N), dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, (rows, 2 * N))
    dw = None
    if topk_weights is not None:
        dw = torch.empty((T, K), dtype=torch.float32, device=dev)
    _check(lib().ep_ll_swiglu_backward(dh.data_ptr(), _ptr(gate_up), _ptr(codes), _ptr(scales), N,
                                       rows, _ptr(topk_weights), T, K, layout.ll_slot.data_ptr(),
                                       out.data_ptr(), _ptr(dw), _ptr(err), _stream(dev)),
           "ep_ll_swiglu_backward")
    _debug_check("ll_swiglu_backward", err, dev)
    return out, dw
