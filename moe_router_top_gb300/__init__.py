"""GB300-native MoE routing front-end: route (gate GEMM, bf16 logits, top-k,
renormalised softmax, shared slot), moe_align_block_size and, behind it, the
experts' feed-forward in bf16 or MXFP4.

Python names mirror the C ABI of include/smr.h; this layer only turns torch
tensors into pointers, allocates outputs with torch when the caller does not
pass them, and raises on a non-OK status. The work runs in libsmr.so's CUDA
kernels on the caller's current stream. Without a workspace route, align,
route_align and expert_gemm share one per device, so such calls must not
overlap on the GPU; expert_up and expert_down keep one per stream.
``SMR_DISABLE=1`` makes every call raise :class:`SmrUnsupported`, so a caller
can take its own fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional, Tuple

from . import _lib
from ._lib import AlignArgs, ExpertDownArgs, ExpertGemmArgs, ExpertUpArgs, RouteArgs

__all__ = [
    "SmrError", "SmrUnsupported", "Workspace", "route", "align", "route_align",
    "route_align_static", "expert_gemm", "expert_up", "expert_down", "quantize_mxfp4",
    "dequantize_mxfp4", "tile_mxfp4_scales",
    "select_block_size", "align_capacity", "route_workspace_size", "align_workspace_size",
    "route_align_workspace_size", "get_device_error", "clear_device_error",
    "get_static_device_error", "clear_static_device_error", "release_workspaces", "test_force_wait_timeout",
    "last_launch_count", "version",
]

ERR_BAD_ID = 1
ERR_WAIT_TIMEOUT = 2
ERR_BAD_SLOT = 4


class SmrError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_name(status)}: {message}")
        self.status = status


class SmrUnsupported(SmrError):
    """The request is outside the implemented contract; fall back."""


def _status_name(status: int) -> str:
    try:
        return _lib.load().smr_status_string(status).decode()
    except Exception:  # library missing while formatting an error
        return f"status {status}"


def _check(status: int) -> None:
    if status == _lib.SMR_OK:
        return
    msg = _lib.load().smr_last_error().decode()
    if status == _lib.SMR_ERR_UNSUPPORTED:
        raise SmrUnsupported(status, msg)
    raise SmrError(status, msg)


def _disabled() -> None:
    if os.environ.get("SMR_DISABLE", "0") not in ("", "0"):
        raise SmrUnsupported(_lib.SMR_ERR_UNSUPPORTED, "disabled by SMR_DISABLE")


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _raw_stream(dev: int) -> int:
    """The current stream of a device, as the pointer that the library takes."""
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_ptr(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _stream_context(stream, device):
    """The context of a call's stream (a torch stream or a pointer; None: the current one)."""
    torch = _torch()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


_ERROR_WORD = slice(4, 8)  # bytes of a workspace's header


class Workspace:
    """A zero-initialised device buffer that grows on demand.

    The library leaves a workspace ready for its next call (counters back at
    zero, a call tag that only advances), so a workspace is zeroed once (on
    allocation) and can be reused by later calls and CUDA graph replays.
    Calls sharing one workspace must not overlap on the GPU. Threads may call
    with it on one stream: the launches of a call stay together.

    It does not grow while its stream is being captured (the zeroing would
    only be recorded, and repeated by every replay): a call that needs more is
    refused then, so make it once, or call ensure, before the capture. Memory
    that a capture has used stays with the workspace when it grows later.
    """

    def __init__(self, nbytes: int = 0, device=None):
        torch = _torch()
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self._on_cuda = self.device.type == "cuda"
        self.buf = None
        self.lock = threading.RLock()  # held from reading buf until the launches are made
        self._captured = False  # whether a capture has used buf
        self._kept = []         # what captures used before
        if nbytes:
            self.ensure(nbytes)

    def __getstate__(self):  # (locks cannot be copied, and graphs know the original's memory only)
        return {"device": self.device, "buf": self.buf}

    def __setstate__(self, state):
        self.__init__(0, state["device"])
        self.buf = state["buf"]

    def ensure(self, nbytes: int):
        """Grows to nbytes, in order on the current stream; the sticky error
        bits go over to the new memory."""
        torch = _torch()
        buf = self.buf
        capturing = self._on_cuda and torch._C._cuda_isCurrentStreamCapturing()
        if buf is None or buf.numel() < nbytes:
            if capturing:
                raise SmrError(_lib.SMR_ERR_WORKSPACE, f"a workspace cannot grow (to {nbytes} bytes) while its stream "
                               "is being captured: make the call once, or call ensure, before the capture")
            error = None
            if buf is not None:
                error = buf[_ERROR_WORD].clone()
                if self._captured:
                    self._kept.append(buf)
                    self._captured = False
                elif buf.is_cuda:  # (calls so far may have run on another stream than its own)
                    buf.record_stream(torch.cuda.current_stream(self.device))
                buf = self.buf = None
            self.buf = buf = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=self.device)
            if error is not None:
                buf[_ERROR_WORD].copy_(error)
        elif capturing:
            self._captured = True
        return buf

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


_default_ws = {}


def _launch(fn, args, ws, nbytes: int, device, stream) -> int:
    """Calls fn(*args, memory, its size, stream) with nbytes of the caller's
    workspace, or of the one that such calls share on the device. The memory
    stays the workspace's until the launches are made."""
    if ws is None:
        key = (device.type, device.index)
        ws = _default_ws.get(key) or _default_ws.setdefault(key, Workspace(0, device))
        if (ws.buf is None or ws.nbytes < nbytes) and ws._on_cuda and _torch()._C._cuda_isCurrentStreamCapturing():
            # memory of the graph's own, which it zeroes at every replay
            ws = _torch().zeros(nbytes, dtype=_torch().uint8, device=device)
    if not isinstance(ws, Workspace):
        return fn(*args, ws.data_ptr(), ws.numel() * ws.element_size(), _stream_ptr(stream))
    with ws.lock:
        if stream is None or (ws.buf is not None and ws.nbytes >= nbytes):
            buf = ws.ensure(nbytes)
        else:
            with _stream_context(stream, device):
                buf = ws.ensure(nbytes)
        return fn(*args, buf.data_ptr(), buf.numel(), _stream_ptr(stream))


def _route_args(hidden, gate_w, shared_w, bias, topk, shared_scale, renormalize, ids, wts,
                logits_out, shared_logit_bf16=False, hidden_fp8=None, hidden_scales=None) -> RouteArgs:
    torch = _torch()
    if hidden.dtype != torch.bfloat16 or gate_w.dtype != torch.bfloat16:
        raise TypeError("hidden and gate_w must be bfloat16")
    if hidden.dim() != 2 or hidden.stride(1) != 1:
        raise ValueError("hidden must be 2-D [M, H] with unit stride along H")
    if gate_w.dim() != 2 or not gate_w.is_contiguous():
        raise ValueError("gate_w must be a contiguous [E, H] tensor")
    if shared_w is not None and (shared_w.dtype != torch.bfloat16 or not shared_w.is_contiguous()):
        raise ValueError("shared_w must be a contiguous bfloat16 [1, H] tensor")
    if bias is not None and (bias.dtype != torch.float32 or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float32 [E] tensor")
    a = RouteArgs()
    a.M, a.H = hidden.shape
    a.E = gate_w.shape[0]
    if gate_w.shape[1] != a.H:
        raise ValueError("gate_w must be [E, H] with the hidden size of `hidden`")
    a.topk = int(topk)
    a.has_shared = 1 if shared_w is not None else 0
    a.shared_scale = float(shared_scale)
    a.renormalize = 1 if renormalize else 0
    a.hidden = _ptr(hidden)
    a.ld_hidden = hidden.stride(0) if a.M > 1 else a.H
    a.gate_w = _ptr(gate_w)
    a.shared_w = _ptr(shared_w)
    a.bias = _ptr(bias)
    a.topk_ids = _ptr(ids)
    a.topk_weights = _ptr(wts)
    a.logits_out = _ptr(logits_out)
    a.shared_logit_bf16 = 1 if shared_logit_bf16 else 0
    if hidden_fp8 is not None:
        M, H = hidden.shape
        if (hidden_fp8.dtype != torch.uint8 or tuple(hidden_fp8.shape) != (M, H)
                or not hidden_fp8.is_contiguous()):
            raise ValueError("hidden_fp8 must be a contiguous uint8 [M, H] tensor (e4m3 codes)")
        if (hidden_scales is None or hidden_scales.dtype != torch.float32
                or tuple(hidden_scales.shape) != (M, H // 128) or not hidden_scales.is_contiguous()):
            raise ValueError("hidden_scales must be a contiguous float32 [M, H // 128] tensor")
        a.hidden_fp8 = _ptr(hidden_fp8)
        a.hidden_scales = _ptr(hidden_scales)
    return a


def _route_outputs(hidden, topk, has_shared, ids, wts):
    torch = _torch()
    M = hidden.shape[0]
    width = topk + (1 if has_shared else 0)
    if ids is None:
        ids = torch.empty((M, width), dtype=torch.int32, device=hidden.device)
    if wts is None:
        wts = torch.empty((M, width), dtype=torch.float32, device=hidden.device)
    return ids, wts


def route(hidden, gate_w, shared_w=None, bias=None, *, topk: int, shared_scale: float = 1.0,
          renormalize: bool = True, shared_logit_bf16: bool = False, topk_ids=None,
          topk_weights=None, logits_out=None, hidden_fp8=None, hidden_scales=None,
          workspace=None, stream=None) -> Tuple:
    """Route M tokens: returns (topk_ids int32 [M, k+S], topk_weights fp32 [M, k+S]).
    hidden_fp8 (uint8 [M, H]) and hidden_scales (float32 [M, H/128]), when
    given, receive the hidden states as e4m3 codes with one scale per 128
    values, written by the same launch."""
    _disabled()
    lib = _lib.load()
    topk_ids, topk_weights = _route_outputs(hidden, topk, shared_w is not None, topk_ids, topk_weights)
    a = _route_args(hidden, gate_w, shared_w, bias, topk, shared_scale, renormalize, topk_ids,
                    topk_weights, logits_out, shared_logit_bf16, hidden_fp8, hidden_scales)
    need = lib.smr_route_workspace_size(ctypes.byref(a))
    _check(_launch(lib.smr_route, (ctypes.byref(a),), workspace, need, hidden.device, stream))
    return topk_ids, topk_weights


def _align_args(topk_ids, num_tokens, width, num_experts, block_size, routed_topk,
                routed_experts, sorted_ids, expert_ids, npp, eplb=None) -> AlignArgs:
    a = AlignArgs()
    a.topk_ids = _ptr(topk_ids)
    a.num_tokens = int(num_tokens)
    a.width = int(width)
    a.num_experts = int(num_experts)
    a.routed_topk = int(routed_topk)
    a.routed_experts = int(routed_experts)
    a.block_size = int(block_size)
    a.sorted_token_ids = _ptr(sorted_ids)
    a.sorted_cap = 0 if sorted_ids is None else sorted_ids.numel()
    a.expert_ids = _ptr(expert_ids)
    a.expert_cap = 0 if expert_ids is None else expert_ids.numel()
    a.num_tokens_post_padded = _ptr(npp)
    if eplb is not None:
        emap, ecount, nphys = eplb
        a.eplb_map = _ptr(emap)
        a.eplb_count = _ptr(ecount)
        a.eplb_max_replicas = int(emap.shape[1]) if emap.dim() == 2 else 1
        a.num_physical = int(nphys)
    return a


def _eplb(eplb_map, eplb_count, num_physical):
    """(map, count, num_physical) of an EPLB remap, or None."""
    if eplb_map is None:
        return None
    torch = _torch()
    for t in (eplb_map, eplb_count):
        if t is None or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError("eplb_map [E_al, R] and eplb_count [E_al] must be contiguous int32 tensors")
    return eplb_map, eplb_count, int(num_physical)


def _align_outputs(device, numel, num_experts, A, sorted_ids, expert_ids, npp):
    torch = _torch()
    cap = align_capacity(numel, num_experts, A)
    if sorted_ids is None:
        sorted_ids = torch.empty(max(cap, 1), dtype=torch.int32, device=device)
    if expert_ids is None:
        expert_ids = torch.empty(max((cap + A - 1) // A, 1), dtype=torch.int32, device=device)
    if npp is None:
        npp = torch.empty(1, dtype=torch.int32, device=device)
    return sorted_ids, expert_ids, npp


def align(topk_ids, num_experts: int, block_size: int = 0, *, routed_topk: int = 0,
          routed_experts: int = 0, sorted_token_ids=None, expert_ids=None,
          num_tokens_post_padded=None, eplb_map=None, eplb_count=None, num_physical: int = 0,
          workspace=None, stream=None) -> Tuple:
    """moe_align_block_size of an int32 [num_tokens, width] id matrix,
    optionally behind an EPLB logical->physical remap (eplb_map [E, R],
    eplb_count [E], num_physical; see smr_align_args in include/smr.h).

    Returns (sorted_token_ids, expert_ids, num_tokens_post_padded); only the
    first npp / npp // A entries of the first two are defined."""
    _disabled()
    torch = _torch()
    lib = _lib.load()
    if topk_ids.dtype != torch.int32 or topk_ids.dim() != 2 or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be a contiguous int32 [num_tokens, width] tensor")
    T, W = topk_ids.shape
    A = block_size if block_size > 0 else select_block_size(T, routed_topk, routed_experts)
    eplb = _eplb(eplb_map, eplb_count, num_physical)
    outs = _align_outputs(topk_ids.device, T * W, num_physical if eplb else num_experts, A,
                          sorted_token_ids, expert_ids, num_tokens_post_padded)
    a = _align_args(topk_ids, T, W, num_experts, block_size, routed_topk, routed_experts, *outs,
                    eplb=eplb)
    need = lib.smr_align_workspace_size(ctypes.byref(a))
    _check(_launch(lib.smr_align, (ctypes.byref(a),), workspace, need, topk_ids.device, stream))
    return outs


def route_align(hidden, gate_w, shared_w=None, bias=None, *, topk: int, block_size: int = 0,
                shared_scale: float = 1.0, renormalize: bool = True,
                shared_logit_bf16: bool = False, topk_ids=None, topk_weights=None,
                logits_out=None, sorted_token_ids=None, expert_ids=None,
                num_tokens_post_padded=None, eplb_map=None, eplb_count=None,
                num_physical: int = 0, hidden_fp8=None, hidden_scales=None, workspace=None,
                stream=None) -> Tuple:
    """Route then align (one launch for M <= 16 without an EPLB remap).
    Returns (topk_ids, topk_weights, sorted_token_ids, expert_ids,
    num_tokens_post_padded)."""
    _disabled()
    lib = _lib.load()
    S = 1 if shared_w is not None else 0
    topk_ids, topk_weights = _route_outputs(hidden, topk, S, topk_ids, topk_weights)
    ra = _route_args(hidden, gate_w, shared_w, bias, topk, shared_scale, renormalize, topk_ids,
                     topk_weights, logits_out, shared_logit_bf16, hidden_fp8, hidden_scales)
    M, E = ra.M, ra.E
    A = block_size if block_size > 0 else select_block_size(M, topk, E)
    eplb = _eplb(eplb_map, eplb_count, num_physical)
    outs = _align_outputs(hidden.device, M * (topk + S), num_physical if eplb else E + S, A,
                          sorted_token_ids, expert_ids, num_tokens_post_padded)
    aa = _align_args(topk_ids, M, topk + S, E + S, block_size, topk, E, *outs, eplb=eplb)
    need = lib.smr_route_align_workspace_size(ctypes.byref(ra), ctypes.byref(aa))
    _check(_launch(lib.smr_route_align, (ctypes.byref(ra), ctypes.byref(aa)), workspace, need, hidden.device, stream))
    return (topk_ids, topk_weights) + tuple(outs)


def route_align_static(hidden, gate_w, shared_w=None, bias=None, *, topk: int,
                       block_size: int = 0, shared_scale: float = 1.0, renormalize: bool = True,
                       shared_logit_bf16: bool = False, topk_ids=None, topk_weights=None,
                       logits_out=None, sorted_token_ids=None, expert_ids=None,
                       num_tokens_post_padded=None, stream=None) -> Tuple:
    """route_align for 1 <= M <= 16 without a workspace: the library's fixed
    device scratch array is used instead, for callers that cannot allocate
    device memory. Calls must not overlap on the GPU; the first call on a
    device must come before any stream capture. Same outputs as route_align.
    (Passing the outputs in avoids the allocations this wrapper otherwise
    makes with torch for convenience.)"""
    _disabled()
    lib = _lib.load()
    S = 1 if shared_w is not None else 0
    topk_ids, topk_weights = _route_outputs(hidden, topk, S, topk_ids, topk_weights)
    ra = _route_args(hidden, gate_w, shared_w, bias, topk, shared_scale, renormalize, topk_ids,
                     topk_weights, logits_out, shared_logit_bf16)
    M, E = ra.M, ra.E
    A = block_size if block_size > 0 else select_block_size(M, topk, E)
    outs = _align_outputs(hidden.device, M * (topk + S), E + S, A, sorted_token_ids, expert_ids,
                          num_tokens_post_padded)
    aa = _align_args(topk_ids, M, topk + S, E + S, block_size, topk, E, *outs)
    _check(lib.smr_route_align_static(ctypes.byref(ra), ctypes.byref(aa), _stream_ptr(stream)))
    return (topk_ids, topk_weights) + tuple(outs)


def expert_gemm(hidden, expert_w, sorted_token_ids, expert_ids, num_tokens_post_padded, *,
                width: int, block_size: int, out=None, workspace=None, stream=None):
    """The consumer expert GEMM over the align's outputs: returns out fp32
    [num_tokens * width, N], row t * width + s = hidden[t] . W[e]^T for the
    slot's expert e (expert_w bf16 [num_experts, N, H]); blocks at or past
    num_tokens_post_padded do no work."""
    _disabled()
    torch = _torch()
    lib = _lib.load()
    if hidden.dtype != torch.bfloat16 or hidden.dim() != 2 or hidden.stride(1) != 1:
        raise ValueError("hidden must be a bfloat16 [T, H] tensor with unit stride along H")
    if expert_w.dtype != torch.bfloat16 or expert_w.dim() != 3 or not expert_w.is_contiguous():
        raise ValueError("expert_w must be a contiguous bfloat16 [num_experts, N, H] tensor")
    T, H = hidden.shape
    E, N, H2 = expert_w.shape
    if H2 != H:
        raise ValueError("expert_w's last dimension must be H")
    if out is None:
        out = torch.empty((T * width, N), dtype=torch.float32, device=hidden.device)
    a = ExpertGemmArgs()
    a.hidden, a.ld_hidden = _ptr(hidden), (hidden.stride(0) if T > 1 else H)
    a.num_tokens, a.width, a.H = T, int(width), H
    a.expert_w, a.num_experts, a.N = _ptr(expert_w), E, N
    a.block_size = int(block_size)
    a.sorted_token_ids, a.sorted_cap = _ptr(sorted_token_ids), sorted_token_ids.numel()
    a.expert_ids, a.num_tokens_post_padded = _ptr(expert_ids), _ptr(num_tokens_post_padded)
    a.out = _ptr(out)
    _check(_launch(lib.smr_expert_gemm, (ctypes.byref(a),), workspace, 256, hidden.device, stream))
    return out


def _check_cuda(*tensors) -> int:
    """Index of the CUDA device that every tensor (None is left out) is on."""
    devices = {t.get_device() for t in tensors if t is not None}
    dev = devices.pop()
    if devices:
        raise ValueError("tensors must be on one device (got "
                         + ", ".join(sorted({str(t.device) for t in tensors if t is not None})) + ")")
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    return dev


def _elsewhere(dev: int, stream):
    """The context to allocate and launch in, or None for the current stream
    of the current device."""
    torch = _torch()
    if stream is None:
        return None if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream must be on the operands' device, cuda:{dev} (got {stream.device})")
    return torch.cuda.stream(stream)


_stream_ws = {}
_PER_THREAD_STREAM = 2  # the handle by which every thread names a default stream of its own


def _stream_workspace(dev: int, s: int) -> Workspace:
    """The workspace of calls on a stream that were given none."""
    key = (dev, s) if s != _PER_THREAD_STREAM else (dev, s, threading.get_ident())
    return _stream_ws.get(key) or _stream_ws.setdefault(key, Workspace(0, _torch().device("cuda", dev)))


def release_workspaces() -> None:
    """Gives back the memory that expert_up and expert_down keep, per stream,
    for calls without a workspace (as much as the largest such call took; work
    that is queued on it is not disturbed). Later calls take new memory. To be
    called, too, before a stream that torch did not make is destroyed and once
    its work is done: another one may get its handle."""
    _stream_ws.clear()


def _check_sizes(bits: int) -> None:
    """Refuses sizes that the library's 32-bit arguments would cut off (bits:
    the sizes or-ed together)."""
    if bits & ~0x7FFFFFFF:
        raise ValueError("sizes must be at least 0 and below 2^31")


def _check_buffer(ws, dev: int) -> None:
    """Refuses a workspace that kernels on device `dev` could not write to."""
    if ws.get_device() != dev:
        raise ValueError(f"workspace must be on the operands' device, cuda:{dev} (got {ws.device})")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _call_product(fn, size_fn, ref, ws, dev: int, s: int, capturing: bool) -> int:
    """One call on a Workspace. One that is too small is refused before any
    launch; it grows and the call is made again."""
    with ws.lock:
        buf = ws.buf
        status = _lib.SMR_ERR_WORKSPACE
        if buf is not None:
            _check_buffer(buf, dev)
            ws._captured |= capturing
            status = fn(ref, buf.data_ptr(), buf.numel(), s)
        if status == _lib.SMR_ERR_WORKSPACE:
            buf = ws.ensure(size_fn(ref))
            _check_buffer(buf, dev)
            status = fn(ref, buf.data_ptr(), buf.numel(), s)
    return status


def _run_product(fn, size_fn, args, ws, dev: int) -> None:
    """Calls a product with the caller's workspace, or with one per device and
    stream (calls on two streams may overlap). A call that is being captured
    gets a workspace of its own, which its graph keeps and zeroes itself."""
    torch = _torch()
    ref = ctypes.byref(args)
    s, capturing = torch._C._cuda_getCurrentRawStream(dev), torch._C._cuda_isCurrentStreamCapturing()
    if isinstance(ws, Workspace):
        status = _call_product(fn, size_fn, ref, ws, dev, s, capturing)
    elif ws is None and not capturing:
        status = _call_product(fn, size_fn, ref, _stream_workspace(dev, s), dev, s, False)
    else:
        if ws is None:
            ws = torch.empty(size_fn(ref), dtype=torch.uint8, device=torch.device("cuda", dev))
            ws[:256].zero_()
        else:
            _check_buffer(ws, dev)
        status = fn(ref, ws.data_ptr(), ws.nbytes, s)
    if status:
        _check(status)


def _product_inputs(x, w, x_scales, w_scales, rows, K, w_rows, gated, sorted_token_ids, expert_ids, npp, block_size,
                    extra):
    """Checks of a product's operands in either format and of the align's outputs
    (extra: one more size)."""
    torch = _torch()
    _check_sizes(rows | K | w_rows | w.shape[0] | block_size | extra)
    mx = x_scales is not None
    if mx != (w_scales is not None):
        raise ValueError("x_scales and w_scales must both be given (MXFP4) or both be None (bfloat16)")
    dtype, kdim = (torch.uint8, K // 2) if mx else (torch.bfloat16, K)
    if x.dtype is not dtype or x.shape != (rows, kdim) or (x.stride(1) != 1 and kdim > 1):
        raise ValueError(f"x must be a {dtype} [{rows}, {kdim}] tensor with unit stride along its rows")
    if w.dtype is not dtype or w.shape[1:] != (w_rows, kdim) or not w.is_contiguous():
        raise ValueError(f"w must be a contiguous {dtype} [num_experts, {w_rows}, {kdim}] tensor")
    if mx:
        if not x.is_contiguous():
            raise ValueError("MXFP4 codes x must be contiguous")
        if x_scales.dtype is not torch.uint8 or x_scales.shape != (rows, K // 32) or not x_scales.is_contiguous():
            raise ValueError(f"x_scales must be a contiguous uint8 [{rows}, {K // 32}] tensor")
        need = _lib.load().smr_mxfp4_tiled_scale_bytes(w.shape[0], w_rows, K, 1 if gated else 0)
        if w_scales.dtype is not torch.uint8 or w_scales.numel() != need or not w_scales.is_contiguous():
            raise ValueError(f"w_scales must be the {need} bytes that tile_mxfp4_scales gives for this weight")
    int32 = torch.int32
    if (sorted_token_ids.dtype is not int32 or expert_ids.dtype is not int32 or npp.dtype is not int32
            or not sorted_token_ids.is_contiguous() or not expert_ids.is_contiguous()):
        raise ValueError("sorted_token_ids, expert_ids and num_tokens_post_padded must be contiguous int32 tensors")
    if block_size > 0 and expert_ids.numel() * block_size < sorted_token_ids.numel():
        raise ValueError("expert_ids must hold an entry for every block of sorted_token_ids")
    if npp.numel() < 1:
        raise ValueError("num_tokens_post_padded must hold one entry")


def _output(out, lead, n, dtype, like, name="out"):
    """The caller's output of shape [*lead, n], checked, or a new one on like's device."""
    if out is None:
        return _torch().empty((*lead, n), dtype=dtype, device=like.device)
    if out.dtype != dtype or out.shape != (*lead, n) or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {(*lead, n)}")
    return out


def expert_up(x, w, sorted_token_ids, expert_ids, num_tokens_post_padded, *, width: int, block_size: int,
              x_scales=None, w_scales=None, out=None, workspace=None, stream=None):
    """The experts' gated product behind the align: returns act bf16
    [num_tokens * width, I], row t * width + s = silu(g) * u with g and u the
    products of x[t] (bf16 [num_tokens, H]) with the gate rows w[e, :I] and the
    up rows w[e, I:] (bf16 [num_experts, 2 I, H]) of the slot's expert e.
    With x_scales and w_scales, x and w are MXFP4 codes (quantize_mxfp4;
    w_scales laid out by tile_mxfp4_scales(..., gated=True)). Rows of slots
    that the align skipped are left as they are in `out`."""
    _disabled()
    torch = _torch()
    lib = _lib.load()
    if w.dim() != 3 or w.shape[1] % 2 or x.dim() != 2:
        raise ValueError("x must be [num_tokens, H] and w [num_experts, 2 I, H]")
    width, block_size = int(width), int(block_size)
    if width < 1:
        raise ValueError(f"width must be >= 1 (got {width})")
    T, H = x.shape
    E, I = w.shape[0], w.shape[1] // 2
    if x_scales is not None:
        H *= 2
    _product_inputs(x, w, x_scales, w_scales, T, H, 2 * I, True, sorted_token_ids, expert_ids,
                    num_tokens_post_padded, block_size, width)
    dev = _check_cuda(x, w, x_scales, w_scales, sorted_token_ids, expert_ids, num_tokens_post_padded, out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return expert_up(x, w, sorted_token_ids, expert_ids, num_tokens_post_padded, width=width,
                             block_size=block_size, x_scales=x_scales, w_scales=w_scales, out=out,
                             workspace=workspace)
    out = _output(out, (T * width,), I, torch.bfloat16, x)
    a = ExpertUpArgs(T, width, H, I, E, block_size, x.data_ptr(), x.stride(0) if T > 1 else H, _ptr(x_scales),
                     w.data_ptr(), _ptr(w_scales), sorted_token_ids.data_ptr(), sorted_token_ids.numel(),
                     expert_ids.data_ptr(), num_tokens_post_padded.data_ptr(), out.data_ptr())
    _run_product(lib.smr_expert_up, lib.smr_expert_up_workspace_size, a, workspace, dev)
    return out


def expert_down(x, w, topk_ids, topk_weights, sorted_token_ids, expert_ids, num_tokens_post_padded, *,
                block_size: int, num_logical: int = 0, fp32_rows: bool = False, x_scales=None,
                w_scales=None, out=None, workspace=None, stream=None):
    """The experts' second product, summed per token: returns out bf16
    [num_tokens, H], out[t] = sum over s of topk_weights[t, s] * (x[t * width +
    s] . w[e]^T) for the slots' experts e; x bf16 [num_tokens * width, I] (the
    rows of expert_up), w bf16 [num_experts, H, I], topk_ids and topk_weights
    [num_tokens, width] as routed. With x_scales and w_scales, x and w are
    MXFP4 codes. A slot whose id is outside [0, num_logical) contributes
    nothing (num_logical: the experts that were aligned; num_experts if 0);
    every other slot must have been aligned. The products wait for the sum in
    fp32 while they are few, else in bf16; fp32_rows=True keeps them in fp32
    whatever the batch (smr_expert_down_fp32 in include/smr.h)."""
    _disabled()
    torch = _torch()
    lib = _lib.load()
    if topk_ids.dtype != torch.int32 or topk_ids.dim() != 2 or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be a contiguous int32 [num_tokens, width] tensor")
    if topk_weights.dtype != torch.float32 or topk_weights.shape != topk_ids.shape or not topk_weights.is_contiguous():
        raise ValueError("topk_weights must be a contiguous float32 tensor of topk_ids' shape")
    if w.dim() != 3 or x.dim() != 2:
        raise ValueError("x must be [num_tokens * width, I] and w [num_experts, H, I]")
    block_size, num_logical = int(block_size), int(num_logical)
    T, width = topk_ids.shape
    E, H, I = w.shape
    if x_scales is not None:
        I *= 2
    _product_inputs(x, w, x_scales, w_scales, T * width, I, H, False, sorted_token_ids, expert_ids,
                    num_tokens_post_padded, block_size, num_logical)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    dev = _check_cuda(x, w, topk_ids, topk_weights, x_scales, w_scales, sorted_token_ids, expert_ids,
                      num_tokens_post_padded, out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return expert_down(x, w, topk_ids, topk_weights, sorted_token_ids, expert_ids, num_tokens_post_padded,
                               block_size=block_size, num_logical=num_logical, fp32_rows=fp32_rows,
                               x_scales=x_scales, w_scales=w_scales, out=out, workspace=workspace)
    out = _output(out, (T,), H, torch.bfloat16, x)
    a = ExpertDownArgs(T, width, H, I, E, block_size, x.data_ptr(), _ptr(x_scales), w.data_ptr(), _ptr(w_scales),
                       topk_ids.data_ptr(), topk_weights.data_ptr(), num_logical if num_logical else E,
                       sorted_token_ids.data_ptr(), sorted_token_ids.numel(), expert_ids.data_ptr(),
                       num_tokens_post_padded.data_ptr(), out.data_ptr())
    if fp32_rows:
        _run_product(lib.smr_expert_down_fp32, lib.smr_expert_down_fp32_workspace_size, a, workspace, dev)
    else:
        _run_product(lib.smr_expert_down, lib.smr_expert_down_workspace_size, a, workspace, dev)
    return out


def quantize_mxfp4(x, *, codes=None, scales=None, stream=None) -> Tuple:
    """bf16 x [..., K] to MXFP4: returns (codes uint8 [..., K / 2], scales
    uint8 [..., K / 32]); see smr_quantize_mxfp4 in include/smr.h. x is
    contiguous, or 2-D with unit stride along K."""
    _disabled()
    torch = _torch()
    lib = _lib.load()
    shape = x.shape
    dense = x.is_contiguous()
    if x.dtype != torch.bfloat16 or len(shape) < 1 or not (dense or (len(shape) == 2 and x.stride(1) == 1)):
        raise ValueError("x must be a bfloat16 tensor, contiguous or 2-D with unit stride along its rows")
    K = shape[-1]
    if K < 32 or K % 32:
        raise ValueError(f"x's last dimension must be a positive multiple of 32 (got {K})")
    _check_sizes(K)
    dev = _check_cuda(x, codes, scales)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return quantize_mxfp4(x, codes=codes, scales=scales)
    lead = shape[:-1]
    codes = _output(codes, lead, K // 2, torch.uint8, x, "codes")
    scales = _output(scales, lead, K // 32, torch.uint8, x, "scales")
    rows = x.numel() // K
    _check(lib.smr_quantize_mxfp4(x.data_ptr(), rows, K, K if dense or rows < 2 else x.stride(0), codes.data_ptr(),
                                  scales.data_ptr(), _raw_stream(dev)))
    return codes, scales


def dequantize_mxfp4(codes, scales, *, out=None, stream=None):
    """The bf16 values [..., K] of MXFP4 codes [..., K / 2] and row-major
    scales [..., K / 32] (exact; NaN where the scale byte is 255)."""
    _disabled()
    torch = _torch()
    lib = _lib.load()
    shape = codes.shape
    if codes.dtype != torch.uint8 or len(shape) < 1 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous uint8 tensor")
    lead, K = shape[:-1], 2 * shape[-1]
    if K < 32 or K % 32:
        raise ValueError(f"codes' last dimension must be a positive multiple of 16 (got {K // 2})")
    _check_sizes(K)
    if scales.dtype != torch.uint8 or scales.shape != lead + (K // 32,) or not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous uint8 tensor of shape {tuple(lead) + (K // 32,)}")
    dev = _check_cuda(codes, scales, out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return dequantize_mxfp4(codes, scales, out=out)
    out = _output(out, lead, K, torch.bfloat16, codes)
    _check(lib.smr_dequantize_mxfp4(codes.data_ptr(), scales.data_ptr(), codes.numel() * 2 // K, K, out.data_ptr(),
                                    _raw_stream(dev)))
    return out


def tile_mxfp4_scales(scales, *, gated: bool = False, out=None, stream=None):
    """A weight's row-major scales uint8 [num_experts, N, K / 32] laid out once
    for expert_up (gated=True: N = 2 I) or expert_down: uint8 [num_experts,
    tiles, K / 128, 512]."""
    _disabled()
    torch = _torch()
    lib = _lib.load()
    if scales.dtype != torch.uint8 or scales.dim() != 3 or not scales.is_contiguous():
        raise ValueError("scales must be a contiguous uint8 [num_experts, N, K / 32] tensor")
    E, N, K = scales.shape[0], scales.shape[1], 32 * scales.shape[2]
    _check_sizes(E | N | K)
    dev = _check_cuda(scales, out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return tile_mxfp4_scales(scales, gated=gated, out=out)
    tiles = -(-(N // 2) // 64) if gated else -(-N // 128)
    out = _output(out, (E, tiles, K // 128), 512, torch.uint8, scales)
    _check(lib.smr_tile_mxfp4_scales(scales.data_ptr(), E, N, K, 1 if gated else 0, out.data_ptr(),
                                     _raw_stream(dev)))
    return out


def select_block_size(num_tokens: int, topk: int, num_experts: int) -> int:
    return int(_lib.load().smr_select_block_size(num_tokens, topk, num_experts))


def align_capacity(numel: int, num_experts: int, block_size: int) -> int:
    return int(_lib.load().smr_align_capacity(numel, num_experts, block_size))


def route_workspace_size(args: RouteArgs) -> int:
    return int(_lib.load().smr_route_workspace_size(ctypes.byref(args)))


def align_workspace_size(args: AlignArgs) -> int:
    return int(_lib.load().smr_align_workspace_size(ctypes.byref(args)))


def route_align_workspace_size(route_args: RouteArgs, align_args: AlignArgs) -> int:
    return int(_lib.load().smr_route_align_workspace_size(ctypes.byref(route_args),
                                                          ctypes.byref(align_args)))


def _shared_default_ws():
    """The workspace that route, align and expert_gemm share on the current device, None if there is none yet."""
    ws = _default_ws.get(("cuda", _torch().cuda.current_device()))
    return None if ws is None or ws.buf is None else ws


def get_device_error(workspace=None, stream=None) -> int:
    """Sticky error bits of a workspace (synchronises the stream). Without one:
    those of the calls on the current device that were given none, and of every
    expert_up and expert_down there, replayed ones included. (A route or align
    captured without a workspace before any such eager call keeps its bits in
    its graph's memory.)"""
    lib = _lib.load()
    code = ctypes.c_int32(0)
    bits = 0
    if workspace is None:
        _check(lib.smr_get_expert_error(_stream_ptr(stream), ctypes.byref(code)))
        bits, workspace = code.value, _shared_default_ws()
        if workspace is None:
            return bits
    buf = workspace.buf if isinstance(workspace, Workspace) else workspace
    _check(lib.smr_get_device_error(buf.data_ptr(), _stream_ptr(stream), ctypes.byref(code)))
    return bits | code.value


def clear_device_error(workspace=None, stream=None) -> None:
    """Clears what get_device_error reads with the same arguments."""
    lib = _lib.load()
    if workspace is None:
        _check(lib.smr_clear_expert_error(_stream_ptr(stream)))
        workspace = _shared_default_ws()
        if workspace is None:
            return
    buf = workspace.buf if isinstance(workspace, Workspace) else workspace
    _check(lib.smr_clear_device_error(buf.data_ptr(), _stream_ptr(stream)))


def get_static_device_error(stream=None) -> int:
    """Sticky error bits of route_align_static's fixed scratch array on the
    current device (synchronises the stream)."""
    code = ctypes.c_int32(0)
    _check(_lib.load().smr_get_static_device_error(_stream_ptr(stream), ctypes.byref(code)))
    return code.value


def clear_static_device_error(stream=None) -> None:
    _check(_lib.load().smr_clear_static_device_error(_stream_ptr(stream)))


STALL_NONE = _lib.SMR_STALL_NONE
STALL_SMALL_TAIL = _lib.SMR_STALL_SMALL_TAIL
STALL_TC_MERGE = _lib.SMR_STALL_TC_MERGE


def test_force_wait_timeout(site: int, limit: int = 1) -> None:
    """Test hook: make one bounded wait of later launches run out (see
    smr_test_force_wait_timeout in include/smr.h); STALL_NONE switches it off."""
    _check(_lib.load().smr_test_force_wait_timeout(int(site), int(limit)))


def last_launch_count() -> int:
    return int(_lib.load().smr_last_launch_count())


def version() -> int:
    return int(_lib.load().smr_version())
