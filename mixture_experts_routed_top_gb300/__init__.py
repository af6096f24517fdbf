"""Routed top-k Mixture-of-Experts experts forward for GB300 (sm_103a).

Thin ctypes binding over the C ABI declared in include/moe_experts.h.  It
only checks and marshals arguments: every step of the forward runs in the
library's CUDA kernels.  PyTorch provides device memory and the current
stream.  There is no CPU or eager fallback: if the library is missing or no
CUDA device is present the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional, Tuple

import torch

from . import build as _build

__all__ = [
    "MoEError", "lib", "route", "dispatch", "dispatch_workspace_size", "workspace_size",
    "experts_forward", "quantize_fp8_blocks", "quantize_fp4_blocks", "workspace_status", "set_decode_rows",
    "get_decode_rows", "set_swap_rows", "get_swap_rows", "profile_begin", "profile_end", "profile_read",
    "selftest_wait_timeout", "launch_count", "accumulator", "set_block_scaled_mma",
    "get_block_scaled_mma", "set_fp4_gemv_rows", "get_fp4_gemv_rows", "set_decode_single",
    "get_decode_single", "set_tile_group", "get_tile_group", "set_pair_gemm", "get_pair_gemm", "set_down_l2_hints", "get_down_l2_hints", "set_down_phases",
    "get_down_phases",
    "route_scored", "route_scored_backward", "block_norm", "block_norm_backward", "linear", "linear_backward",
    "gated_linear", "gated_linear_backward", "quantize_fp8_rows", "linear_fp8",
    "layer_norm", "layer_norm_backward",
    "Workspace", "STATUS", "STAGES", "W_BF16", "W_FP8_E4M3", "W_FP4_E2M1", "SCALE_NONE", "SCALE_F32",
    "SCALE_UE8M0", "ACTIVATIONS",
]

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_CUDA",
          4: "MOE_ERR_TIMEOUT", 5: "MOE_ERR_WORKSPACE"}
STAGES = ("dispatch", "gemm1", "gemm2", "finish")
W_BF16, W_FP8_E4M3, W_FP4_E2M1 = 0, 1, 2
SCALE_NONE, SCALE_F32, SCALE_UE8M0 = 0, 1, 2
_SCALE_BY_NAME = {None: SCALE_NONE, "none": SCALE_NONE, "f32": SCALE_F32, "float": SCALE_F32,
                  "ue8m0": SCALE_UE8M0}


class MoEError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


_LIB = None
_P, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_L, _F = ctypes.c_int64, ctypes.c_float
_SIGS = {
    "moe_version": ([], _I),
    "moe_last_error": ([], ctypes.c_char_p),
    "moe_route": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "moe_dispatch_workspace_size": ([_I, _I, _I], _SZ),
    "moe_dispatch": ([_P, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "moe_workspace_size": ([_I, _I, _I, _I, _I, _I], _SZ),
    "moe_experts_forward": ([_P, _I, _I, _P, _P, _I, _I, _I, _P, _P, _I, _P, _P, _I, _P, _P,
                             _SZ, _P], _I),
    "moe_experts_forward_act": ([_P, _I, _I, _P, _P, _I, _I, _I, _P, _P, _I, _P, _P, _I, _I, _P,
                                 _P, _SZ, _P], _I),
    "moe_quantize_fp8_blocks": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "moe_quantize_fp4_blocks": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "moe_workspace_status": ([_P, _P], _I),
    "moe_set_decode_rows": ([_I], None),
    "moe_get_decode_rows": ([], _I),
    "moe_set_swap_rows": ([_I], None),
    "moe_get_swap_rows": ([], _I),
    "moe_profile_begin": ([], _I),
    "moe_profile_end": ([ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int), _I], _I),
    "moe_profile_read": ([ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int), _I], _I),
    "moe_selftest_wait_timeout": ([_P, _SZ, _I, _P], _I),
    "moe_launch_count": ([], ctypes.c_longlong),
    "moe_workspace_accumulator_offset": ([_I, _I, _I, _I, _I, _I], _SZ),
    "moe_set_block_scaled_mma": ([_I], None),
    "moe_get_block_scaled_mma": ([], _I),
    "moe_set_down_l2_hints": ([_I], None),
    "moe_get_down_l2_hints": ([], _I),
    "moe_set_pair_gemm": ([_I], None),
    "moe_get_pair_gemm": ([], _I),
    "moe_set_down_phases": ([_I], None),
    "moe_get_down_phases": ([], _I),
    "moe_set_tile_group": ([_I], None),
    "moe_get_tile_group": ([], _I),
    "moe_set_decode_single": ([_I], None),
    "moe_get_decode_single": ([], _I),
    "moe_set_fp4_gemv_rows": ([_I], None),
    "moe_get_fp4_gemv_rows": ([], _I),
    "moe_route_scored": ([_P, _I, _L, _I, _I, _I, _I, _P, _I, _I, _I, _I, _F, _P, _P, _P], _I),
    "moe_route_scored_backward": ([_P, _I, _L, _I, _I, _I, _I, _P, _I, _F, _P, _P, _P, _P, _L, _P], _I),
    "moe_block_norm": ([_P, _I, _L, _P, _L, _P, _I, _I, _L, _F, _I, _P, _I, _P, _I, _F, _I, _I, _P,
                        _P, _P], _I),
    "moe_block_norm_backward_workspace_size": ([_I], _SZ),
    "moe_block_norm_backward": ([_P, _L, _P, _L, _P, _I, _L, _P, _L, _P, _I, _I, _L, _F, _I, _P, _P,
                                 _I, _F, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "moe_call_packed": ([_I, ctypes.c_char_p], _I),
    "moe_linear_workspace_size": ([], _SZ),
    "moe_linear": ([_P, _L, _P, _L, _P, _I, _I, _P, _L, _I, _I, _I, _P, _I, _L, _P, _P, _SZ, _P], _I),
    "moe_linear_backward_workspace_size": ([_I, _I], _SZ),
    "moe_gated_linear": ([_P, _L, _P, _L, _P, _I, _I, _I, _I, _I, _P, _L, _P, _P, _SZ, _P], _I),
    "moe_gated_linear_backward_workspace_size": ([_I, _I], _SZ),
    "moe_gated_linear_backward": ([_P, _L, _P, _L, _P, _L, _I, _P, _L, _I, _I, _I, _P, _P, _P, _P, _SZ,
                                   _P], _I),
    "moe_quantize_fp8_rows": ([_P, _L, _I, _I, _I, _P, _P, _L, _L, _P], _I),
    "moe_linear_fp8_workspace_size": ([_I, _I], _SZ),
    "moe_linear_fp8": ([_P, _L, _P, _L, _L, _P, _L, _P, _I, _P, _I, _I, _P, _L, _I, _I, _I, _P, _I, _L, _P,
                        _SZ, _P], _I),
    "moe_layer_norm": ([_P, _I, _L, _P, _L, _P, _P, _I, _F, _I, _I, _P, _P, _P], _I),
    "moe_layer_norm_backward_workspace_size": ([_I], _SZ),
    "moe_layer_norm_backward": ([_P, _L, _P, _L, _P, _I, _L, _P, _I, _F, _I, _I, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "moe_linear_backward": ([_P, _I, _L, _P, _L, _P, _L, _I, _P, _L, _I, _I, _I, _P, _P, _P, _P, _SZ,
                             _P], _I),
}


def lib_path() -> str:
    return _build.LIB_PATH


def lib(build_if_missing: bool = True):
    """Load libmoe_gb300.so (building it in-tree first if it is absent)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.isfile(path):
        if not build_if_missing:
            raise RuntimeError(f"CUDA library {path} is not built")
        _build.build()
    L = ctypes.CDLL(path)
    for name, (args, res) in _SIGS.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _LIB = L
    return L


def _check(status: int):
    if status != 0:
        raise MoEError(status, lib().moe_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without the Python object around it, which
# costs 3 of the 12 microseconds of a small call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)
if _raw_stream is None or _raw_device is None:
    _raw_device = torch.cuda.current_device

    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _stream(stream=None):
    return _raw_stream(_raw_device()) if stream is None else stream.cuda_stream


def _tensors(values):
    for v in values:
        if isinstance(v, torch.Tensor):
            yield v
        elif isinstance(v, (tuple, list)):
            yield from _tensors(v)


def _on_stream(call, args: dict):
    """call(**args) on args["stream"], as under torch.cuda.stream(): results and
    workspaces are allocated, and workspaces zeroed, in that stream's order.
    Tensors are marked as used by the stream that is not their own, so that
    letting go of one gives its memory to nobody while either still works on it.
    Waiting for what the arguments come from is the caller's, as ever."""
    stream = args.pop("stream")
    given = list(_tensors(args.values()))
    for t in given:
        if t.is_cuda and t.device != stream.device:
            raise ValueError(f"stream on {stream.device}, a tensor on {t.device}")
    before = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        result = call(**args)
    if stream != before:
        for t in given:
            if t.is_cuda:
                t.record_stream(stream)
        for t in _tensors((result,)):
            t.record_stream(before)
    return result


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


# ------------------------------------------------------------------ router
def route(logits: torch.Tensor, k: int, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Top-k routing of fp32 logits [T, E] -> (topk_idx int32 [T,k], topk_w fp32 [T,k])."""
    if stream is not None:
        return _on_stream(route, locals())
    _need_cuda(logits)
    if logits.dtype != torch.float32 or logits.dim() != 2:
        raise ValueError("logits must be fp32 [T, E]")
    T, E = logits.shape
    idx = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    _check(lib().moe_route(_ptr(logits), T, E, k, _ptr(idx), _ptr(w), _stream()))
    return idx, w


# ------------------------------------------------------------------ dispatch
def dispatch_workspace_size(T: int, E: int, k: int) -> int:
    return int(lib().moe_dispatch_workspace_size(T, E, k))


def dispatch(topk_idx: torch.Tensor, E: int, stream=None):
    """Expert-contiguous ordering -> (counts [E], offsets [E+1], sorted_f [T*k], row_of [T*k])."""
    if stream is not None:
        return _on_stream(dispatch, locals())
    _need_cuda(topk_idx)
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be int32 [T, k]")
    T, k = topk_idx.shape
    dev = topk_idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_f = torch.empty(T * k, dtype=torch.int32, device=dev)
    row_of = torch.empty(T * k, dtype=torch.int32, device=dev)
    nbytes = dispatch_workspace_size(T, E, k)
    ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
    _check(lib().moe_dispatch(_ptr(topk_idx), T, E, k, _ptr(counts), _ptr(offsets),
                              _ptr(sorted_f), _ptr(row_of), _ptr(ws), nbytes, _stream()))
    _check(lib().moe_workspace_status(_ptr(ws), _stream()))
    return counts, offsets, sorted_f, row_of


# ------------------------------------------------------------------ forward
def workspace_size(T: int, H: int, I: int, E: int, k: int, wdtype: int = W_BF16) -> int:
    """Bytes of workspace experts_forward needs for these sizes and weight
    type (W_BF16, W_FP8_E4M3 or W_FP4_E2M1)."""
    return int(lib().moe_workspace_size(T, H, I, E, k, wdtype))


def _capturing() -> bool:
    """Whether the current stream is being captured; the default stream (handle 0) cannot be
    and is not asked."""
    return torch.cuda.is_current_stream_capturing()


class Workspace:
    """Caller-owned device scratch, grown on demand.  The first 256 bytes of a
    buffer hold the device error word; they start zeroed.

    buf is the buffer of calls that run at once.  A buffer that a call under
    CUDA-graph capture was given stays allocated as long as the workspace,
    whatever later calls need, since the graph goes on writing to it.  A
    buffer that a capture had to allocate belongs to its graph, which zeroes
    it in each replay: make the call once before, as capturing asks for."""

    def __init__(self, device="cuda"):
        self.device = torch.device(device)
        self.buf = None
        self.home = None        # the stream in whose order buf's memory is given back
        self.captured = []      # buffers that graphs use

    def buffers(self):
        """Every buffer whose error word may be set."""
        own = [] if self.buf is None or any(b is self.buf for b in self.captured) else [self.buf]
        return own + self.captured

    def get(self, nbytes: int, now: Optional[int] = None) -> torch.Tensor:
        """A buffer of at least nbytes for a call on the current stream (its handle: now)."""
        if now is None:
            now = _stream()
        old = self.buf
        if now and _capturing():
            return self._for_graph(nbytes)
        if self.home != now and old is not None:
            old.record_stream(torch.cuda.current_stream(self.device))
        if old is None or old.numel() < nbytes:
            self.buf, self.home = self._new(nbytes), now
            if old is not None and not any(b is old for b in self.captured):
                self.buf[:4].copy_(old[:4])     # errors that nobody has read yet
        return self.buf

    def _new(self, nbytes: int) -> torch.Tensor:
        return torch.zeros(max(nbytes, 1024), dtype=torch.uint8, device=self.device)

    def _for_graph(self, nbytes: int) -> torch.Tensor:
        buf = next((b for b in self.buffers() if b.numel() >= nbytes), None)
        if buf is None:
            buf = self._new(nbytes)
        if not any(b is buf for b in self.captured):
            self.captured.append(buf)
        return buf


# Workspaces of the calls that are given none: one per device and stream, since
# calls on different streams run at the same time.
_DEFAULT_WS = {}


def _default_ws(dev: int) -> Workspace:
    """The default workspace of the device's current stream."""
    key = (dev, _raw_stream(dev))
    ws = _DEFAULT_WS.get(key)
    if ws is not None:
        return ws
    if key[1] and _capturing():
        # a stream that only captures has none; the calls were tried on another one, and what
        # was allocated now would be zeroed, error word and all, in every replay
        for (d, _), other in list(_DEFAULT_WS.items()):
            if d == dev:
                return other
    return _DEFAULT_WS.setdefault(key, Workspace(torch.device("cuda", dev)))


# moe_activation values
ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}


def experts_forward(hidden: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                    w_gate_up: torch.Tensor, w_down: torch.Tensor,
                    scale_gate_up: Optional[torch.Tensor] = None,
                    scale_down: Optional[torch.Tensor] = None, scale_fmt=None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None,
                    stream=None, activation: str = "silu") -> torch.Tensor:
    """Routed experts forward -> bf16 [T, H].

    hidden bf16 [T,H]; topk_idx int32 [T,k]; topk_w fp32 [T,k];
    w_gate_up [E,2I,H] and w_down [E,H,I], bf16 or e4m3 bytes (uint8 or
    float8_e4m3fn) with 128x128 block scales (scale_fmt 'f32' or 'ue8m0'),
    or packed e2m1 bytes (uint8 or int8) [E,2I,H/2] and [E,H,I/2] with 1x32
    UE8M0 scales from quantize_fp4_blocks; activation: the gate activation,
    'silu' (SwiGLU), 'gelu' (GeGLU, exact erf GELU) or 'relu' (ReGLU)."""
    if stream is not None:
        return _on_stream(experts_forward, locals())
    _need_cuda(hidden, topk_idx, topk_w, w_gate_up, w_down, scale_gate_up, scale_down, out)
    T, H = hidden.shape
    k = topk_idx.shape[1]
    E, twoI, H2 = w_gate_up.shape
    I = twoI // 2
    fp4 = w_gate_up.dtype in (torch.uint8, torch.int8) and 2 * H2 == H
    if fp4:
        if tuple(w_down.shape) != (E, H, I // 2):
            raise ValueError("packed FP4 weight shapes must be [E, 2I, H/2] and [E, H, I/2]")
        if scale_fmt is None:
            scale_fmt = "ue8m0"
    elif H2 != H or tuple(w_down.shape) != (E, H, I):
        raise ValueError("weight shapes must be [E, 2I, H] and [E, H, I]")
    if hidden.dtype != torch.bfloat16 or topk_idx.dtype != torch.int32 or topk_w.dtype != torch.float32:
        raise ValueError("hidden bf16, topk_idx int32, topk_w fp32 expected")
    fp8 = not fp4 and w_gate_up.dtype in (torch.uint8, torch.float8_e4m3fn)
    wdtype = W_FP4_E2M1 if fp4 else W_FP8_E4M3 if fp8 else W_BF16
    if not (fp4 or fp8) and w_gate_up.dtype != torch.bfloat16:
        raise ValueError("weights must be bf16, e4m3 bytes or packed e2m1 bytes")
    sf = _SCALE_BY_NAME[scale_fmt] if not isinstance(scale_fmt, int) else scale_fmt
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=hidden.device)
    nbytes = workspace_size(T, H, I, E, k, wdtype)
    ws = _workspace(workspace, hidden.get_device(), nbytes)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    _check(lib().moe_experts_forward_act(
        _ptr(hidden), T, H, _ptr(topk_idx), _ptr(topk_w), E, k, I, _ptr(w_gate_up),
        _ptr(w_down), wdtype, _ptr(scale_gate_up), _ptr(scale_down), sf, ACTIVATIONS[activation],
        _ptr(out), _ptr(ws), ws.numel(), _stream()))
    return out


def workspace_status(workspace=None, stream=None):
    """Synchronise and raise MoEError if a kernel flagged an error in ws (a
    Workspace: in any of its buffers, those of captured graphs among them;
    None: in a default workspace of any stream of the device, which is
    synchronised)."""
    if workspace is None:
        torch.cuda.synchronize()
        dev = torch.cuda.current_device()
        bufs = [b for (d, _), ws in list(_DEFAULT_WS.items()) if d == dev for b in ws.buffers()]
    else:
        bufs = (workspace.buffers() or [None]) if isinstance(workspace, Workspace) else [workspace]
    for ws in bufs:
        _check(lib().moe_workspace_status(_ptr(ws), _stream(stream)))


def accumulator(workspace, T: int, H: int, I: int, E: int, k: int,
                wdtype: int = W_BF16) -> torch.Tensor:
    """fp32 [T, H] view of the workspace's output accumulator: after a
    grouped-path forward with these sizes it holds the un-rounded output
    (see moe_workspace_accumulator_offset)."""
    off = int(lib().moe_workspace_accumulator_offset(T, H, I, E, k, wdtype))
    bufs = workspace.buffers() if isinstance(workspace, Workspace) else [workspace]
    ws = next((b for b in bufs if off + T * H * 4 <= b.numel()), None)
    if off == 0 or ws is None:
        raise ValueError("workspace too small for these sizes")
    return ws[off:off + T * H * 4].view(torch.float32).view(T, H)


def default_workspace(device="cuda", stream=None) -> Workspace:
    """The workspace of calls on the device's current stream (or stream) that are given none.
    A graph captured without a workspace uses the one of the stream that it was
    captured on, or if that has none the device's first: replays and the calls
    that share it have to be ordered."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return default_workspace(stream.device)
    d = torch.device(device)
    return _default_ws(torch.cuda.current_device() if d.index is None else d.index)


# ------------------------------------------------------------------ around the experts
# Activations, logits and their gradients may have rows further apart than
# they are long (a slice of columns of a larger matrix); everything else is
# contiguous.  Each call is asynchronous on the current stream; with stream= it
# runs as under torch.cuda.stream(stream).
_BF16, _F32 = torch.bfloat16, torch.float32
_DT = {_BF16: 0, _F32: 1}
_SCORES = {"softmax": 0, "sigmoid": 1}
_ONLY_F32, _ONLY_BF16, _ONLY_I32 = (_F32,), (_BF16,), (torch.int32,)
_ACT_NONE = -1
_LINEAR_WS = 0  # the library's constant, once it is loaded


# Calls of moe_call_packed and the slots of their argument blocks (q integer or
# pointer, d float); the stream is the last.
_ROUTE = (0, struct.Struct("=12qd3q").pack)
_ROUTE_BWD = (1, struct.Struct("=9qd6q").pack)
_NORM = (2, struct.Struct("=9qd5qd5q").pack)
_NORM_BWD = (3, struct.Struct("=13qd4qd10q").pack)
_LINEAR = (4, struct.Struct("=19q").pack)
_LINEAR_BWD = (5, struct.Struct("=19q").pack)
_GATED = (7, struct.Struct("=16q").pack)
_GATED_BWD = (8, struct.Struct("=18q").pack)
_FP8_ROWS = (9, struct.Struct("=10q").pack)
_LINEAR_FP8 = (10, struct.Struct("=23q").pack)
_LAYER_NORM = (11, struct.Struct("=8qd5q").pack)
_LAYER_NORM_BWD = (12, struct.Struct("=9qd9q").pack)


def _bad(name: str, what: str):
    raise ValueError(f"{name} must be {what}")


def _names(dtypes) -> str:
    return " or ".join(str(d)[6:] for d in dtypes)


def _mat(name: str, t: torch.Tensor, dtypes, shape, dev: int) -> int:
    """Checks a matrix of this shape on device dev, its rows contiguous; -> its row stride."""
    if t.shape != shape or t.dtype not in dtypes or t.get_device() != dev:
        _bad(name, f"a tensor {list(shape)} of {_names(dtypes)} on CUDA device {dev}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        _bad(name, "contiguous along its rows")
    return ld if shape[0] > 1 else shape[1]


def _dense(name: str, t: torch.Tensor, dtypes, shape, dev: int) -> int:
    """Checks a contiguous tensor of this shape; -> its address."""
    if t.shape != shape or t.dtype not in dtypes or t.get_device() != dev or not t.is_contiguous():
        _bad(name, f"a contiguous tensor {list(shape)} of {_names(dtypes)} on CUDA device {dev}")
    return t.data_ptr()


def _call(call, dev: int, *args):
    """One of the packed calls on device `dev`: its current stream appended, the device made current."""
    L = _LIB or lib()
    if _raw_device() == dev:
        status = L.moe_call_packed(call[0], call[1](*args, _raw_stream(dev)))
    else:
        with torch.cuda.device(dev):
            status = L.moe_call_packed(call[0], call[1](*args, _raw_stream(dev)))
    if status:
        _check(status)


def _workspace(workspace: Optional[Workspace], dev: int, nbytes: int) -> torch.Tensor:
    now = _raw_stream(dev)
    if workspace is None:
        workspace = _DEFAULT_WS.get((dev, now)) or _default_ws(dev)
    return workspace.get(nbytes, now)


def _matrix_of(name: str, t: torch.Tensor):
    """-> the device index and shape of a CUDA matrix."""
    dev, shape = t.get_device(), t.shape
    if dev < 0 or len(shape) != 2:
        _bad(name, "a 2-D CUDA tensor")
    return dev, shape


def _score_of(score: str) -> int:
    sc = _SCORES.get(score)
    if sc is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    return sc


def route_scored(logits: torch.Tensor, k: int, *, score: str = "sigmoid",
                 bias: Optional[torch.Tensor] = None, n_group: int = 1, topk_group: int = 1,
                 group_top: int = 2, renormalise: bool = True, scale: float = 1.0,
                 out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Top-k routing by scores -> (topk_idx int32 [T,k], topk_w fp32 [T,k]).

    logits fp32 or bf16 [T,E]; score 'sigmoid' or 'softmax'; bias fp32 [E],
    added to the scores for the choice only; n_group > 1: only the topk_group
    best groups are eligible, a group's score being the sum of its group_top
    (1 or 2) best; the chosen scores are divided by their sum if renormalise,
    then multiplied by scale.  Experts with a logit of -inf or NaN are masked.
    out: (topk_idx, topk_w) to write into."""
    if stream is not None:
        return _on_stream(route_scored, locals())
    dev, shape = _matrix_of("logits", logits)
    ld = _mat("logits", logits, _DT, shape, dev)
    T, E = shape
    if out is None:
        idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
        w = torch.empty((T, k), dtype=_F32, device=logits.device)
        pi, pw = idx.data_ptr(), w.data_ptr()
    else:
        idx, w = out
        pi = _dense("topk_idx", idx, _ONLY_I32, (T, k), dev)
        pw = _dense("topk_w", w, _ONLY_F32, (T, k), dev)
    _call(_ROUTE, dev, logits.data_ptr(), _DT[logits.dtype], ld, T, E, k, _score_of(score),
          0 if bias is None else _dense("bias", bias, _ONLY_F32, (E,), dev), n_group, topk_group, group_top,
          renormalise, scale, pi, pw)
    return idx, w


def route_scored_backward(logits: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                          grad_w: torch.Tensor, *, score: str = "sigmoid",
                          bias: Optional[torch.Tensor] = None, renormalise: bool = True,
                          scale: float = 1.0, out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Gradient of route_scored's weights -> grad_logits [T,E] of the logits' type.

    logits, score, bias, renormalise, scale as route_scored was called with;
    topk_idx, topk_w what it returned; grad_w fp32 [T,k].  out: a tensor to
    write into, its rows contiguous."""
    if stream is not None:
        return _on_stream(route_scored_backward, locals())
    dev, shape = _matrix_of("logits", logits)
    ld = _mat("logits", logits, _DT, shape, dev)
    T, E = shape
    _, slots = _matrix_of("topk_idx", topk_idx)
    if slots[0] != T:
        _bad("topk_idx", "[T, k]")
    if out is None:
        out = torch.empty(shape, dtype=logits.dtype, device=logits.device)
        ldo = E
    else:
        ldo = _mat("out", out, (logits.dtype,), shape, dev)
    _call(_ROUTE_BWD, dev, logits.data_ptr(), _DT[logits.dtype], ld, T, E, slots[1], _score_of(score),
          0 if bias is None else _dense("bias", bias, _ONLY_F32, (E,), dev), renormalise, scale,
          _dense("topk_idx", topk_idx, _ONLY_I32, slots, dev), _dense("topk_w", topk_w, _ONLY_F32, slots, dev),
          _dense("grad_w", grad_w, _ONLY_F32, slots, dev), out.data_ptr(), ldo)
    return out


def _gate_of(gate: torch.Tensor, shape, dev: int):
    """-> (address, moe_gate kind, dtype, row stride): [H] per channel, [T] or
    [T,1] per token, [T,H] per element.  A 1-D gate where T = H is per channel."""
    dt = _DT.get(gate.dtype)
    if dt is None or gate.get_device() != dev:
        _bad("gate", f"a tensor of {_names(_DT)} on CUDA device {dev}")
    T, H = shape
    if gate.shape == shape and H != 1:
        return gate.data_ptr(), 3, dt, _mat("gate", gate, _DT, shape, dev)
    if not gate.is_contiguous():
        _bad("gate", "contiguous")
    if gate.shape == (H,):
        return gate.data_ptr(), 1, dt, 0
    if gate.shape == (T,) or gate.shape == (T, 1):
        return gate.data_ptr(), 2, dt, 0
    return _bad("gate", "[H] (per channel), [T] or [T, 1] (per token), or [T, H]")


def _norm_weights(post_weight, pre_weight, H: int, dev: int):
    """-> the addresses of the norms' weights (0: none), their dtype."""
    post = pre = dt = 0
    if post_weight is not None:
        post, dt = _dense("post_weight", post_weight, _DT, (H,), dev), _DT[post_weight.dtype]
    if pre_weight is not None:
        pre = _dense("pre_weight", pre_weight, _DT, (H,), dev)
        if post and _DT[pre_weight.dtype] != dt:
            raise ValueError("post_weight and pre_weight must have one dtype")
        dt = _DT[pre_weight.dtype]
    return post, pre, dt


def block_norm(residual: torch.Tensor, y: Optional[torch.Tensor] = None, *,
               gate: Optional[torch.Tensor] = None, scale: float = 1.0, post_norm: bool = False,
               post_weight: Optional[torch.Tensor] = None, pre_norm: bool = True,
               pre_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
               out: Optional[Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]] = None,
               stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The norms after and before a block in one pass -> (residual_out, normed).

    z = y / rms(y) * post_weight if post_norm else y;
    residual_out = residual + scale * gate * z;
    normed = residual_out / rms(residual_out) * pre_weight, or None if not pre_norm.

    residual bf16 or fp32 [T,H] (residual_out alike); y bf16 [T,H], or None:
    only the norm, and residual itself is returned; normed bf16; gate [H],
    [T] / [T,1] or [T,H], bf16 or fp32; weights [H], both bf16 or both fp32.
    out: (residual_out, normed) to write into, either of them None for a new
    tensor; residual_out may be residual."""
    if stream is not None:
        return _on_stream(block_norm, locals())
    dev, shape = _matrix_of("residual", residual)
    ld_r = _mat("residual", residual, _DT, shape, dev)
    T, H = shape
    pg, kind, gate_dt, ld_g = (0, 0, 0, 0) if gate is None else _gate_of(gate, shape, dev)
    post, pre, wdt = _norm_weights(post_weight, pre_weight, H, dev)
    res, n = (None, None) if out is None else out
    py = ld_y = pres = pn = 0
    if y is None:
        res = residual
    else:
        py, ld_y = y.data_ptr(), _mat("y", y, _ONLY_BF16, shape, dev)
        if res is None:
            res = torch.empty(shape, dtype=residual.dtype, device=residual.device)
            pres = res.data_ptr()
        else:
            pres = _dense("residual_out", res, (residual.dtype,), shape, dev)
    if not pre_norm:
        n = None
    elif n is None:
        n = torch.empty(shape, dtype=_BF16, device=residual.device)
        pn = n.data_ptr()
    else:
        pn = _dense("normed", n, _ONLY_BF16, shape, dev)
    _call(_NORM, dev, residual.data_ptr(), _DT[residual.dtype], ld_r, py, ld_y, pg, kind, gate_dt, ld_g,
          scale, post_norm, post, pre_norm, pre, wdt, eps, T, H, pres, pn)
    return res, n


def block_norm_backward(grad_residual: Optional[torch.Tensor], grad_normed: Optional[torch.Tensor],
                        residual: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                        gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                        post_norm: bool = False, post_weight: Optional[torch.Tensor] = None,
                        pre_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        workspace: Optional[Workspace] = None, stream=None):
    """Gradients of block_norm -> (d_residual, d_y, d_gate, d_post_weight, d_pre_weight).

    grad_residual: dL/d residual_out [T,H] or None; grad_normed: dL/d normed
    bf16 [T,H], or None where pre_norm was off; residual: the residual_out that
    block_norm returned; the rest as it was called with.  What does not apply
    comes back as None.  d_gate is fp32 for a per-channel gate, else of the
    gate's type; the weights' gradients are fp32 [H].  workspace: as in linear."""
    if stream is not None:
        return _on_stream(block_norm_backward, locals())
    dev, shape = _matrix_of("residual", residual)
    ld_r = _mat("residual", residual, _DT, shape, dev)
    T, H = shape
    device = residual.device
    pgr = ld_gr = pgn = ld_gn = py = ld_y = pdy = pdg = pdpost = pdpre = 0
    d_y = d_gate = d_post = d_pre = None
    if grad_residual is not None:
        pgr, ld_gr = grad_residual.data_ptr(), _mat("grad_residual", grad_residual, (residual.dtype,), shape, dev)
    if grad_normed is not None:
        pgn, ld_gn = grad_normed.data_ptr(), _mat("grad_normed", grad_normed, _ONLY_BF16, shape, dev)
    if y is not None:
        py, ld_y = y.data_ptr(), _mat("y", y, _ONLY_BF16, shape, dev)
        d_y = torch.empty(shape, dtype=_BF16, device=device)
        pdy = d_y.data_ptr()
    pg, kind, gate_dt, ld_g = (0, 0, 0, 0) if gate is None else _gate_of(gate, shape, dev)
    post, pre, wdt = _norm_weights(post_weight, pre_weight, H, dev)
    d_res = torch.empty(shape, dtype=residual.dtype, device=device)
    if kind:
        d_gate = torch.empty(gate.shape, dtype=_F32 if kind == 1 else gate.dtype, device=device)
        pdg = d_gate.data_ptr()
    if post:
        d_post = torch.empty(H, dtype=_F32, device=device)
        pdpost = d_post.data_ptr()
    if pre:
        d_pre = torch.empty(H, dtype=_F32, device=device)
        pdpre = d_pre.data_ptr()
    ws = _workspace(workspace, dev, (_LIB or lib()).moe_block_norm_backward_workspace_size(H))
    _call(_NORM_BWD, dev, pgr, ld_gr, pgn, ld_gn, residual.data_ptr() if pgn else 0, _DT[residual.dtype],
          ld_r, py, ld_y, pg, kind, gate_dt, ld_g, scale, post_norm, post, pre, wdt, eps, T, H, d_res.data_ptr(),
          pdy, pdg, pdpost, pdpre, ws.data_ptr(), ws.numel())
    return d_res, d_y, d_gate, d_post, d_pre


def layer_norm(residual: torch.Tensor, y: Optional[torch.Tensor] = None, *,
               weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
               out: Optional[Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The residual sum and the layer norm after it in one pass -> (residual_out, normed).

    residual_out = residual + y;
    normed = (residual_out - mean) / sqrt(var + eps) * weight + bias over a row.

    residual bf16 or fp32 [T,H] (residual_out alike); y bf16 [T,H], or None:
    only the norm, and residual itself is returned; normed bf16; weight and
    bias [H] or None, both bf16 or both fp32.  out: (residual_out, normed) to
    write into, either of them None for a new tensor; residual_out may be
    residual, and without y is None or residual."""
    if stream is not None:
        return _on_stream(layer_norm, locals())
    dev, shape = _matrix_of("residual", residual)
    ld_r = _mat("residual", residual, _DT, shape, dev)
    T, H = shape
    pw, pb, wdt = _weight_and_bias(weight, bias, H, dev)
    res, n = (None, None) if out is None else out
    py = ld_y = pres = 0
    if y is None:
        if res is not None and res.data_ptr() != residual.data_ptr():
            raise ValueError("a residual_out to write into needs y: without it residual itself is returned")
        res = residual
    else:
        py, ld_y = y.data_ptr(), _mat("y", y, _ONLY_BF16, shape, dev)
        if res is None:
            res = torch.empty(shape, dtype=residual.dtype, device=residual.device)
            pres = res.data_ptr()
        else:
            pres = _dense("residual_out", res, (residual.dtype,), shape, dev)
    if n is None:
        n = torch.empty(shape, dtype=_BF16, device=residual.device)
        pn = n.data_ptr()
    else:
        pn = _dense("normed", n, _ONLY_BF16, shape, dev)
    _call(_LAYER_NORM, dev, residual.data_ptr(), _DT[residual.dtype], ld_r, py, ld_y, pw, pb, wdt, eps, T, H, pres, pn)
    return res, n


def _weight_and_bias(weight, bias, H: int, dev: int):
    """-> the addresses of a layer norm's weight and bias (0: none), their dtype."""
    pw = pb = dt = 0
    if weight is not None:
        pw, dt = _dense("weight", weight, _DT, (H,), dev), _DT[weight.dtype]
    if bias is not None:
        pb = _dense("bias", bias, _DT, (H,), dev)
        if pw and _DT[bias.dtype] != dt:
            raise ValueError("weight and bias must have one dtype")
        dt = _DT[bias.dtype]
    return pw, pb, dt


def layer_norm_backward(grad_residual: Optional[torch.Tensor], grad_normed: torch.Tensor, residual: torch.Tensor, *,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        eps: float = 1e-5, need_y: bool = False, workspace: Optional[Workspace] = None, stream=None):
    """Gradients of layer_norm -> (d_residual, d_y, d_weight, d_bias).

    grad_residual: dL/d residual_out [T,H] or None; grad_normed: dL/d normed
    bf16 [T,H]; residual: the residual_out that layer_norm returned; weight,
    bias, eps as it was called with (None: that gradient is None).  need_y:
    also y's gradient, which is d_residual in bf16 (the same tensor where that
    is bf16).  d_weight and d_bias are fp32 [H].  workspace: as in linear."""
    if stream is not None:
        return _on_stream(layer_norm_backward, locals())
    dev, shape = _matrix_of("residual", residual)
    ld_r = _mat("residual", residual, _DT, shape, dev)
    T, H = shape
    device = residual.device
    pgr = ld_gr = pdy = pdw = pdb = 0
    d_y = d_w = d_b = None
    if grad_residual is not None:
        pgr, ld_gr = grad_residual.data_ptr(), _mat("grad_residual", grad_residual, (residual.dtype,), shape, dev)
    ld_gn = _mat("grad_normed", grad_normed, _ONLY_BF16, shape, dev)
    pw, pb, wdt = _weight_and_bias(weight, bias, H, dev)
    d_res = torch.empty(shape, dtype=residual.dtype, device=device)
    if need_y and residual.dtype == _BF16:
        d_y = d_res
    elif need_y:
        d_y = torch.empty(shape, dtype=_BF16, device=device)
        pdy = d_y.data_ptr()
    if pw:
        d_w = torch.empty(H, dtype=_F32, device=device)
        pdw = d_w.data_ptr()
    if pb:
        d_b = torch.empty(H, dtype=_F32, device=device)
        pdb = d_b.data_ptr()
    ws = _workspace(workspace, dev, (_LIB or lib()).moe_layer_norm_backward_workspace_size(H))
    _call(_LAYER_NORM_BWD, dev, pgr, ld_gr, grad_normed.data_ptr(), ld_gn, residual.data_ptr(), _DT[residual.dtype],
          ld_r, pw, wdt, eps, T, H, d_res.data_ptr(), pdy, pdw, pdb, ws.data_ptr(), ws.numel())
    return d_res, d_y, d_w, d_b


def _act(activation: Optional[str]) -> int:
    if activation is None:
        return _ACT_NONE
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be None or one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[activation]


def linear(x: torch.Tensor, w: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
           activation: Optional[str] = None, residual: Optional[torch.Tensor] = None,
           out_dtype: torch.dtype = torch.bfloat16, preact: bool = False,
           out: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None, stream=None):
    """residual + act(x w^T + bias) -> [T,N], or (that, x w^T + bias) if preact.

    x bf16 [T,K]; w bf16 [N,K]; K a multiple of 8; bias [N] bf16 or fp32;
    activation None, 'silu', 'gelu' (exact) or 'relu'; out_dtype bf16 or fp32
    (router logits), which residual and the pre-activation share.  out: the
    tensor to write into (rows contiguous); it may be residual.  Calls that
    share a workspace must be ordered on one stream; without one they use
    their stream's."""
    global _LINEAR_WS
    if stream is not None:
        return _on_stream(linear, locals())
    dev, xs = _matrix_of("x", x)
    T, K = xs
    ld_x = _mat("x", x, _ONLY_BF16, xs, dev)
    N = w.shape[0]
    ld_w = _mat("w", w, _ONLY_BF16, (N, K), dev)
    shape = (T, N)
    if out is None:
        dt = _DT.get(out_dtype)
        if dt is None:
            _bad("out_dtype", _names(_DT))
        out = torch.empty(shape, dtype=out_dtype, device=x.device)
        ld_o = N
    else:
        ld_o = _mat("out", out, _DT, shape, dev)
        out_dtype = out.dtype
        dt = _DT[out_dtype]
    pb = bdt = pr = ld_r = pz = 0
    z = None
    if bias is not None:
        pb, bdt = _dense("bias", bias, _DT, (N,), dev), _DT[bias.dtype]
    if residual is not None:
        pr, ld_r = residual.data_ptr(), _mat("residual", residual, (out_dtype,), shape, dev)
    if preact:  # it has out's row stride
        z = torch.empty_strided(shape, (ld_o, 1), dtype=out_dtype, device=x.device)
        pz = z.data_ptr()
    _LINEAR_WS = _LINEAR_WS or lib().moe_linear_workspace_size()
    ws = _workspace(workspace, dev, _LINEAR_WS)
    _call(_LINEAR, dev, x.data_ptr(), ld_x, w.data_ptr(), ld_w, pb, bdt, _act(activation), pr, ld_r, T, K, N,
          out.data_ptr(), dt, ld_o, pz, ws.data_ptr(), ws.numel())
    return (out, z) if preact else out


def linear_backward(grad_y: torch.Tensor, x: torch.Tensor, w: torch.Tensor, *,
                    bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                    preact: Optional[torch.Tensor] = None, need_x: bool = True, need_w: bool = True,
                    workspace: Optional[Workspace] = None, stream=None):
    """Gradients of linear -> (dx bf16 [T,K], dw bf16 [N,K], dbias fp32 [N]).

    grad_y [T,N] of linear's output type (it is also the residual's gradient);
    preact: what linear(..., preact=True) returned, with an activation; bias:
    as passed to linear (None: dbias is None).  need_x / need_w = False leave
    that gradient out (None).  workspace: as in linear."""
    if stream is not None:
        return _on_stream(linear_backward, locals())
    dev, xs = _matrix_of("x", x)
    T, K = xs
    ld_x = _mat("x", x, _ONLY_BF16, xs, dev)
    N = w.shape[0]
    ld_w = _mat("w", w, _ONLY_BF16, (N, K), dev)
    shape = (T, N)
    ld_g = _mat("grad_y", grad_y, _DT, shape, dev)
    act = _act(activation)
    if (preact is None) != (act == _ACT_NONE):
        raise ValueError("an activation and its preact go together")
    pz = ld_z = pdx = pdw = pdb = 0
    dx = dw = db = None
    if preact is not None:
        pz, ld_z = preact.data_ptr(), _mat("preact", preact, (grad_y.dtype,), shape, dev)
    if bias is not None:
        _dense("bias", bias, _DT, (N,), dev)
        db = torch.empty(N, dtype=_F32, device=x.device)
        pdb = db.data_ptr()
    if need_x:
        dx = torch.empty(xs, dtype=_BF16, device=x.device)
        pdx = dx.data_ptr()
    if need_w:
        dw = torch.empty((N, K), dtype=_BF16, device=x.device)
        pdw = dw.data_ptr()
    ws = _workspace(workspace, dev, (_LIB or lib()).moe_linear_backward_workspace_size(T, N))
    _call(_LINEAR_BWD, dev, grad_y.data_ptr(), _DT[grad_y.dtype], ld_g, x.data_ptr(), ld_x, w.data_ptr(),
          ld_w, act, pz, ld_z, T, K, N, pdx, pdw, pdb, ws.data_ptr(), ws.numel())
    return dx, dw, db


def _gate_act(activation: str) -> int:
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[activation]


def _halves(w: torch.Tensor) -> int:
    """-> the rows of each half of gate and up weights."""
    if w.dim() != 2 or w.shape[0] % 2:
        _bad("w", "[2 I, K]: gate rows, then as many up rows")
    return w.shape[0] // 2


def gated_linear(x: torch.Tensor, w: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
                 activation: str = "silu", preact: bool = False, out: Optional[torch.Tensor] = None,
                 workspace: Optional[Workspace] = None, stream=None):
    """act(z[:, :I]) * z[:, I:] with z = x w^T + bias -> bf16 [T,I], or (that, z) if preact.

    Both projections of a gated feed-forward, its activation and product in one
    kernel.  x bf16 [T,K]; w bf16 [2I,K]: I gate rows, then I up rows (an
    expert's w_gate_up); K a multiple of 8; bias [2I] bf16 or fp32; activation
    'silu', 'gelu' (exact) or 'relu'; z bf16 [T,2I], for the backward pass.
    out: the tensor to write into (rows contiguous).  workspace: as in linear."""
    global _LINEAR_WS
    if stream is not None:
        return _on_stream(gated_linear, locals())
    dev, xs = _matrix_of("x", x)
    T, K = xs
    ld_x = _mat("x", x, _ONLY_BF16, xs, dev)
    I = _halves(w)
    ld_w = _mat("w", w, _ONLY_BF16, (2 * I, K), dev)
    act = _gate_act(activation)
    pb = bdt = pz = 0
    z = None
    if bias is not None:
        pb, bdt = _dense("bias", bias, _DT, (2 * I,), dev), _DT[bias.dtype]
    if out is None:
        out = torch.empty((T, I), dtype=_BF16, device=x.device)
        ld_o = I
    else:
        ld_o = _mat("out", out, _ONLY_BF16, (T, I), dev)
    if preact:
        z = torch.empty((T, 2 * I), dtype=_BF16, device=x.device)
        pz = z.data_ptr()
    _LINEAR_WS = _LINEAR_WS or lib().moe_linear_workspace_size()
    ws = _workspace(workspace, dev, _LINEAR_WS)
    _call(_GATED, dev, x.data_ptr(), ld_x, w.data_ptr(), ld_w, pb, bdt, act, T, K, I, out.data_ptr(), ld_o, pz,
          ws.data_ptr(), ws.numel())
    return (out, z) if preact else out


def gated_linear_backward(grad_h: torch.Tensor, x: torch.Tensor, w: torch.Tensor, preact: torch.Tensor, *,
                          bias: Optional[torch.Tensor] = None, activation: str = "silu", need_x: bool = True,
                          need_w: bool = True, workspace: Optional[Workspace] = None, stream=None):
    """Gradients of gated_linear -> (dx bf16 [T,K], dw bf16 [2I,K], dbias fp32 [2I]).

    grad_h bf16 [T,I]; preact: the z that gated_linear(..., preact=True)
    returned; bias: as passed to gated_linear (None: dbias is None).  need_x /
    need_w = False leave that gradient out (None).  workspace: as in linear."""
    if stream is not None:
        return _on_stream(gated_linear_backward, locals())
    dev, xs = _matrix_of("x", x)
    T, K = xs
    ld_x = _mat("x", x, _ONLY_BF16, xs, dev)
    I = _halves(w)
    ld_w = _mat("w", w, _ONLY_BF16, (2 * I, K), dev)
    ld_g = _mat("grad_h", grad_h, _ONLY_BF16, (T, I), dev)
    ld_z = _mat("preact", preact, _ONLY_BF16, (T, 2 * I), dev)
    act = _gate_act(activation)
    pdx = pdw = pdb = 0
    dx = dw = db = None
    if bias is not None:
        _dense("bias", bias, _DT, (2 * I,), dev)
        db = torch.empty(2 * I, dtype=_F32, device=x.device)
        pdb = db.data_ptr()
    if need_x:
        dx = torch.empty(xs, dtype=_BF16, device=x.device)
        pdx = dx.data_ptr()
    if need_w:
        dw = torch.empty((2 * I, K), dtype=_BF16, device=x.device)
        pdw = dw.data_ptr()
    ws = _workspace(workspace, dev, (_LIB or lib()).moe_gated_linear_backward_workspace_size(T, I))
    _call(_GATED_BWD, dev, grad_h.data_ptr(), ld_g, x.data_ptr(), ld_x, w.data_ptr(), ld_w, act, preact.data_ptr(),
          ld_z, T, K, I, pdx, pdw, pdb, ws.data_ptr(), ws.numel())
    return dx, dw, db


_E4M3 = (torch.uint8, torch.float8_e4m3fn)


@functools.lru_cache(maxsize=256)
def _fp8_workspace(T: int, K: int) -> int:
    return lib().moe_linear_fp8_workspace_size(T, K)


_SCALE_DT = {_F32: SCALE_F32, torch.uint8: SCALE_UE8M0}


def quantize_fp8_rows(x: torch.Tensor, scale_fmt: str = "f32", *,
                      out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, stream=None):
    """bf16 [T,K] -> (e4m3 codes uint8 [T,K], scales [T,K/128] of its 1x128 blocks as
    fp32 ('f32') or uint8 exponent bytes ('ue8m0')), for linear_fp8.

    K a multiple of 128.  out: (codes, scales) to write into, codes contiguous,
    scales with any positive strides."""
    if stream is not None:
        return _on_stream(quantize_fp8_rows, locals())
    dev, xs = _matrix_of("x", x)
    T, K = xs
    ld_x = _mat("x", x, _ONLY_BF16, xs, dev)
    sf = _SCALE_BY_NAME.get(scale_fmt, SCALE_NONE)
    if sf == SCALE_NONE:
        raise ValueError("scale_fmt must be 'f32' or 'ue8m0'")
    if out is None:
        q = torch.empty(xs, dtype=torch.uint8, device=x.device)
        pq = q.data_ptr()
        s = torch.empty((T, K // 128), dtype=_F32 if sf == SCALE_F32 else torch.uint8, device=x.device)
    else:
        q, s = out
        pq = _dense("codes", q, _E4M3, xs, dev)
    ps, s_row, s_kb = _row_scales("scales", s, sf, xs, dev)
    _call(_FP8_ROWS, dev, x.data_ptr(), ld_x, T, K, sf, pq, ps, s_row, s_kb)
    return q, s


def _row_scales(name: str, s: torch.Tensor, sf: int, xs, dev: int):
    """Checks the scales of a matrix's 1x128 blocks; -> (address, strides of row and block)."""
    shape = (xs[0], xs[1] // 128)
    if s.shape != shape or _SCALE_DT.get(s.dtype) != sf or s.get_device() != dev:
        _bad(name, f"a tensor {list(shape)} of {'float32' if sf == SCALE_F32 else 'uint8'} on CUDA device {dev}")
    a, b = s.stride()
    return s.data_ptr(), max(a, 1) if shape[0] == 1 else a, max(b, 1) if shape[1] == 1 else b


def linear_fp8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *,
               x_scale: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               activation: Optional[str] = None, residual: Optional[torch.Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               workspace: Optional[Workspace] = None, stream=None) -> torch.Tensor:
    """residual + act(x w^T + bias) -> [T,N] of 8-bit operands with block scales.

    w e4m3 [N,K] (uint8 or float8_e4m3fn), K a multiple of 128, N any; w_scale
    [ceil(N/128), K/128] of its 128x128 blocks: fp32, or uint8 UE8M0 exponent
    bytes.  quantize_fp8_blocks makes both of whole blocks: where N is no multiple of
    128, of w with rows of zeros up to the next one, whose codes [:N] are w.  x bf16 [T,K], quantised in 1x128 blocks with
    scales of w_scale's format on the way; or e4m3 with x_scale [T,K/128] of
    that format (quantize_fp8_rows), any strides; a row's side by side are
    read best.  bias, activation, residual,
    out_dtype, out, workspace: as in linear."""
    global _LINEAR_WS
    if stream is not None:
        return _on_stream(linear_fp8, locals())
    dev, xs = _matrix_of("x", x)
    T, K = xs
    ld_x = _mat("x", x, _ONLY_BF16 if x_scale is None else _E4M3, xs, dev)
    N = w.shape[0]
    ld_w = _mat("w", w, _E4M3, (N, K), dev)
    sf = _SCALE_DT.get(w_scale.dtype)
    pws = _dense("w_scale", w_scale, _SCALE_DT, ((N + 127) // 128, K // 128), dev)
    px, s_row, s_kb = (0, 0, 0) if x_scale is None else _row_scales("x_scale", x_scale, sf, xs, dev)
    shape = (T, N)
    if out is None:
        dt = _DT.get(out_dtype)
        if dt is None:
            _bad("out_dtype", _names(_DT))
        out = torch.empty(shape, dtype=out_dtype, device=x.device)
        ld_o = N
    else:
        ld_o = _mat("out", out, _DT, shape, dev)
        out_dtype = out.dtype
        dt = _DT[out_dtype]
    pb = bdt = pr = ld_r = 0
    if bias is not None:
        pb, bdt = _dense("bias", bias, _DT, (N,), dev), _DT[bias.dtype]
    if residual is not None:
        pr, ld_r = residual.data_ptr(), _mat("residual", residual, (out_dtype,), shape, dev)
    if x_scale is None:
        need = _fp8_workspace(T, K)
    else:
        need = _LINEAR_WS = _LINEAR_WS or lib().moe_linear_workspace_size()
    ws = _workspace(workspace, dev, need)
    _call(_LINEAR_FP8, dev, x.data_ptr(), ld_x, px, s_row, s_kb, w.data_ptr(), ld_w, pws, sf, pb, bdt,
          _act(activation), pr, ld_r, T, K, N, out.data_ptr(), dt, ld_o, ws.data_ptr(), ws.numel())
    return out


# ------------------------------------------------------------------ FP8
def quantize_fp8_blocks(w: torch.Tensor, scale_fmt: str = "f32", stream=None):
    """bf16 [..., R, C] -> (e4m3 codes uint8 [..., R, C], scales [..., R/128, C/128]
    as fp32 ('f32') or uint8 exponent bytes ('ue8m0')).  R and C multiples of 128."""
    if stream is not None:
        return _on_stream(quantize_fp8_blocks, locals())
    _need_cuda(w)
    if w.dtype != torch.bfloat16:
        raise ValueError("w must be bf16")
    *lead, R, C = w.shape
    nmat = 1
    for d in lead:
        nmat *= d
    q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    sf = _SCALE_BY_NAME[scale_fmt]
    sdt = torch.uint8 if sf == SCALE_UE8M0 else torch.float32
    s = torch.empty(*lead, R // 128 if R % 128 == 0 else 0, C // 128 if C % 128 == 0 else 0,
                    dtype=sdt, device=w.device)
    _check(lib().moe_quantize_fp8_blocks(_ptr(w), nmat, R, C, sf, _ptr(q), _ptr(s),
                                         _stream()))
    return q, s


def quantize_fp4_blocks(w: torch.Tensor, stream=None):
    """bf16 [..., R, C] -> (packed e2m1 codes uint8 [..., R, C/2], two per
    byte with the even element in the low nibble; UE8M0 exponent bytes
    uint8 [..., R, C/32], one per 1x32 block)."""
    if stream is not None:
        return _on_stream(quantize_fp4_blocks, locals())
    _need_cuda(w)
    if w.dtype != torch.bfloat16:
        raise ValueError("w must be bf16")
    *lead, R, C = w.shape
    nmat = 1
    for d in lead:
        nmat *= d
    q = torch.empty(*lead, R, C // 2, dtype=torch.uint8, device=w.device)
    s = torch.empty(*lead, R, C // 32, dtype=torch.uint8, device=w.device)
    _check(lib().moe_quantize_fp4_blocks(_ptr(w), nmat, R, C, _ptr(q), _ptr(s), _stream()))
    return q, s


# ------------------------------------------------------------------ control
def set_decode_rows(rows: int):
    lib().moe_set_decode_rows(int(rows))


def get_decode_rows() -> int:
    return int(lib().moe_get_decode_rows())


def set_swap_rows(rows_per_expert: int):
    """Mean rows per expert at or below which the bf16 GEMMs use the swap-AB
    orientation (< 0: default, 0: never)."""
    lib().moe_set_swap_rows(int(rows_per_expert))


def get_swap_rows() -> int:
    return int(lib().moe_get_swap_rows())


def set_block_scaled_mma(on: bool):
    """UE8M0 FP8 experts on the tensor core's block scaling (True, default)
    or on the software-promotion kernel (False)."""
    lib().moe_set_block_scaled_mma(1 if on else 0)


def get_block_scaled_mma() -> bool:
    return bool(lib().moe_get_block_scaled_mma())


def set_down_l2_hints(bits: int):
    """L2 policies of the down GEMMs: bit 0 accumulator evict_last, bit 1
    W_down loads evict_first (< 0: the default, 1)."""
    lib().moe_set_down_l2_hints(int(bits))


def get_down_l2_hints() -> int:
    return int(lib().moe_get_down_l2_hints())


def set_pair_gemm(mask: int):
    """bf16 grouped GEMMs on CTA pairs: bit 0 gate/up, bit 1 down (< 0: the
    default, gate/up on pairs where H >= 4096)."""
    lib().moe_set_pair_gemm(int(mask))


def get_pair_gemm() -> int:
    return int(lib().moe_get_pair_gemm())


def set_down_phases(phases: int):
    """Output-column slices of the down GEMMs run one after the other (< 0:
    automatic, the default; 0 or 1: one)."""
    lib().moe_set_down_phases(int(phases))


def get_down_phases() -> int:
    return int(lib().moe_get_down_phases())


def set_tile_group(m_tiles: int):
    """m-tiles per tile group of the token-row gate/up GEMM (0: all)."""
    lib().moe_set_tile_group(int(m_tiles))


def get_tile_group() -> int:
    return int(lib().moe_get_tile_group())


def set_decode_single(on: bool):
    """Small bf16 decode batches (<= 64 routed rows) as one cooperative
    kernel (True) or as two kernels (False, default)."""
    lib().moe_set_decode_single(1 if on else 0)


def get_decode_single() -> bool:
    return bool(lib().moe_get_decode_single())


def set_fp4_gemv_rows(rows: int):
    """FP4 forwards with T*k <= rows use the CUDA-core GEMVs, larger ones the
    block-scaled tensor-core GEMMs (< 0: the default, 0 = GEMMs always; at
    most 64)."""
    lib().moe_set_fp4_gemv_rows(int(rows))


def get_fp4_gemv_rows() -> int:
    return int(lib().moe_get_fp4_gemv_rows())


def profile_begin():
    _check(lib().moe_profile_begin())


def profile_end():
    """-> {stage: (total_ms, launches)} for the forwards since profile_begin()."""
    n = len(STAGES)
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int * n)()
    lib().moe_profile_end(ms, cnt, n)
    return {STAGES[i]: (float(ms[i]), int(cnt[i])) for i in range(n)}


def profile_read():
    """-> {stage: (total_ms, launches)} of the forwards recorded so far, without
    ending the session (after a CUDA-graph replay: that replay's times)."""
    n = len(STAGES)
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int * n)()
    lib().moe_profile_read(ms, cnt, n)
    return {STAGES[i]: (float(ms[i]), int(cnt[i])) for i in range(n)}


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(lib().moe_launch_count())


def selftest_wait_timeout(limit_us: int = 2000, stream=None) -> int:
    """Run the bounded-wait self-test; returns the status that
    moe_workspace_status reports afterwards (expected MOE_ERR_TIMEOUT)."""
    if stream is not None:
        return _on_stream(selftest_wait_timeout, locals())
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    _check(lib().moe_selftest_wait_timeout(_ptr(ws), ws.numel(), int(limit_us), _stream()))
    return int(lib().moe_workspace_status(_ptr(ws), _stream()))
