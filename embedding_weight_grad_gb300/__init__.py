"""Sparse embedding weight-gradient accumulation on GB300 (sm_103a).

``accumulate_embedding_wgrad(ids, grad, main_grad)`` performs
``main_grad += embedding_dense_backward(grad, ids)`` touching only the rows of the ids
that occur, with the values of PyTorch's sort-based embedding backward followed by
``main_grad.add_`` (Megatron Core API docs, ``core.fusions.fused_embedding_wgrad``:
module docstring, ``accumulate_embedding_wgrad`` and ``can_accumulate_embedding_wgrad``).

Beside it, the other operators of a training step that deal with the vocabulary and with
main_grads: ``token_logprobs`` and ``token_logprobs_backward`` (log probabilities of given
tokens, entropies and the most likely alternatives from logits, and their gradient),
``orthogonalize_update`` (the Newton-Schulz orthogonalisation of the Muon optimiser),
``layer_norm`` and ``layer_norm_backward`` (whose weights' gradients go into main_grads) and
``adamw_plan`` / ``adamw_step`` (AdamW over many tensors at once, with states in 32 bits or in 8).

This module only marshals arguments into the C ABI of ``libewg.so`` (declared in
``include/ewg.h``); every step of the computation runs in that library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no CPU
fallback: without the compiled library every entry point raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple, Optional

import torch

__all__ = [
    "MIN_TOKENS", "MAX_TOKENS", "NROWS", "EwgError", "can_accumulate_embedding_wgrad",
    "accumulate_embedding_wgrad", "workspace_bytes", "plan", "apply", "read_status",
    "library_path", "lib", "accumulate_embedding_wgrad_shard", "MAX_TOP", "TokenLogprobs",
    "token_logprobs", "token_logprobs_backward", "status_workspace",
    "orthogonalize_update", "orthogonalize_workspace", "LayerNorm", "layer_norm",
    "layer_norm_backward", "layer_norm_workspace", "ADAMW_BLOCK", "AdamWPlan", "adamw_plan",
    "adamw_step",
]

MIN_TOKENS = 3073
MAX_TOKENS = 1 << 28
NROWS = 10
MAX_TOP = 32
ADAMW_BLOCK = 256

_INT32, _INT64, _BF16, _FP32 = 0, 1, 2, 3
OK, ERR_UNSUPPORTED, ERR_INVALID, ERR_CUDA, ERR_ID_OUT_OF_RANGE, ERR_TIMEOUT, ERR_BOUNDS = \
    0, 1, 2, 3, 4, 5, 6

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libewg.so")
# The same library built with every kernel index checked (EWG_ERR_BOUNDS on a failure).
_DEBUG_LIB_PATH = os.path.join(_HERE, "libewg_debug.so")
_lib = None
_debug_lib = None
_lock = threading.Lock()
# Pinned host tensors handed to the host-input call, each kept alive until an event
# recorded after the call has completed: the library copies from their raw pointers, so
# torch's pinned-memory allocator does not know the copies are still pending.
_pending_host = []
_pending_lock = threading.Lock()


class EwgError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(msg)
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded C library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            _lib = _load(_LIB_PATH)
    return _lib


def debug_lib():
    """The bounds-checking build of the same library (libewg_debug.so), for tests."""
    global _debug_lib
    if _debug_lib is not None:
        return _debug_lib
    with _lock:
        if _debug_lib is None:
            _debug_lib = _load(_DEBUG_LIB_PATH)
    return _debug_lib


def _load(path):
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m embedding_weight_grad_gb300.build` (needs nvcc)")
    L = ctypes.CDLL(path)
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    L.ewg_can_accumulate.argtypes = [vp, i32, i64, vp, i32, i64, vp, i32, i64, i64, i64]
    L.ewg_can_accumulate.restype = i32
    L.ewg_workspace_bytes.argtypes = [i64, i64]
    L.ewg_workspace_bytes.restype = sz
    L.ewg_accumulate.argtypes = [vp, i32, i64, vp, i32, i64, vp, i32, i64, i64, i64, vp,
                                 sz, vp]
    L.ewg_accumulate.restype = i32
    L.ewg_plan.argtypes = [vp, i32, i64, i64, i64, vp, sz, vp]
    L.ewg_plan.restype = i32
    L.ewg_apply.argtypes = [vp, i32, i64, vp, i32, i64, i64, i64, i64, vp, sz, vp]
    L.ewg_apply.restype = i32
    L.ewg_accumulate_shard.argtypes = [vp, i32, i64, vp, i32, i64, vp, i32, i64, i64, i64,
                                       i64, i64, vp, sz, vp]
    L.ewg_accumulate_shard.restype = i32
    L.ewg_plan_shard.argtypes = [vp, i32, i64, i64, i64, i64, i64, vp, sz, vp]
    L.ewg_plan_shard.restype = i32
    L.ewg_host_workspace_bytes.argtypes = [i64, i64, i32, i32]
    L.ewg_host_workspace_bytes.restype = sz
    L.ewg_accumulate_host.argtypes = [vp, i32, i64, vp, i32, vp, i32, i64, i64, i64, vp,
                                      sz, vp]
    L.ewg_accumulate_host.restype = i32
    f32 = ctypes.c_float
    L.ewg_token_logprobs.argtypes = [vp, i32, i64, vp, i32, i64, i64, f32, i32, vp, vp, vp, vp,
                                     vp, vp, vp, sz, vp]
    L.ewg_token_logprobs.restype = i32
    L.ewg_token_logprobs_backward.argtypes = [vp, i32, i64, vp, i32, i64, i64, f32, vp, vp, vp,
                                              vp, vp, vp, i64, vp, sz, vp]
    L.ewg_token_logprobs_backward.restype = i32
    L.ewg_orthogonalize_workspace_bytes.argtypes = [i64, i64, i64]
    L.ewg_orthogonalize_workspace_bytes.restype = sz
    for f in (L.ewg_orthogonalize, L.ewg_orthogonalize_transposed):
        f.argtypes = [vp, i32, i64, i64, i64, i64, i64, vp, i64, i64, i32, f32, f32, f32, vp, sz, vp]
        f.restype = i32
    f64 = ctypes.c_double
    L.ewg_layer_norm.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, f64, vp, i64, vp, vp, vp]
    L.ewg_layer_norm.restype = i32
    L.ewg_layer_norm_workspace_bytes.argtypes = [i64, i64]
    L.ewg_layer_norm_workspace_bytes.restype = sz
    L.ewg_layer_norm_backward.argtypes = [vp, i64, vp, i64, i32, i64, i64, vp, vp, vp, i32, vp, i64,
                                          vp, vp, i32, vp, sz, vp]
    L.ewg_layer_norm_backward.restype = i32
    L.ewg_adamw_plan_bytes.argtypes = [i64]
    L.ewg_adamw_plan_bytes.restype = sz
    L.ewg_adamw_plan.argtypes = [vp, i64, i32, vp, sz]
    L.ewg_adamw_plan.restype = i32
    L.ewg_adamw_step.argtypes = [vp, sz, i64, vp, f64, vp, f64, f64, f64, f64, vp, vp]
    L.ewg_adamw_step.restype = i32
    L.ewg_read_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
    L.ewg_read_status.restype = i32
    L.ewg_status_string.argtypes = [i32]
    L.ewg_status_string.restype = ctypes.c_char_p
    L.ewg_last_error.argtypes = []
    L.ewg_last_error.restype = ctypes.c_char_p
    L.ewg_version.argtypes = []
    L.ewg_version.restype = i32
    return L


def _raise_on(code: int):
    if code != OK:
        L = lib()
        raise EwgError(code, f"{L.ewg_status_string(code).decode()}: {L.ewg_last_error().decode()}")


_FLOAT_CODES = {torch.bfloat16: _BF16, torch.float32: _FP32}
_ID_CODES = {torch.int32: _INT32, torch.int64: _INT64}


def _stream_ptr(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


class _Args:
    """The C-ABI view of (ids, grad, main_grad), or the reason there is none."""

    def __init__(self, ids: torch.Tensor, grad: torch.Tensor, main_grad: torch.Tensor):
        self.reason = None
        if not (ids.is_cuda and grad.is_cuda and main_grad.is_cuda):
            self.reason = "tensors must be on a CUDA device"
            return
        if ids.dtype not in _ID_CODES or grad.dtype not in _FLOAT_CODES \
                or main_grad.dtype not in _FLOAT_CODES:
            self.reason = "ids must be int32/int64; grad and main_grad bf16/fp32"
            return
        if main_grad.dim() != 2 or main_grad.stride(1) != 1:
            self.reason = "main_grad must be [num_embeddings, hidden] with unit inner stride"
            return
        if not ids.is_contiguous():
            self.reason = "ids must be contiguous"
            return
        V, H = main_grad.shape
        n = ids.numel()
        if tuple(grad.shape) != tuple(ids.shape) + (H,):
            self.reason = "grad must be [*ids.shape, hidden]"
            return
        try:
            g2 = grad.view(n, H)
        except RuntimeError:
            self.reason = "grad rows must share one row stride"
            return
        if H > 0 and n > 0 and g2.stride(1) != 1:
            self.reason = "grad must have unit inner stride"
            return
        self.ids, self.grad, self.main_grad = ids.reshape(n), g2, main_grad
        self.n, self.V, self.H = n, V, H
        self.grad_stride = g2.stride(0) if n > 1 else H
        self.mg_stride = main_grad.stride(0) if V > 1 else H
        self.device = main_grad.device

    def c_args(self):
        return (self.ids.data_ptr(), _ID_CODES[self.ids.dtype], self.n,
                self.grad.data_ptr(), _FLOAT_CODES[self.grad.dtype], self.grad_stride,
                self.main_grad.data_ptr(), _FLOAT_CODES[self.main_grad.dtype], self.V, self.H,
                self.mg_stride)


def can_accumulate_embedding_wgrad(ids: torch.Tensor, grad: torch.Tensor,
                                   main_grad: torch.Tensor) -> bool:
    """Whether accumulate_embedding_wgrad supports these tensors (see include/ewg.h)."""
    a = _Args(ids, grad, main_grad)
    if a.reason is not None:
        return False
    with torch.cuda.device(a.device):
        return bool(lib().ewg_can_accumulate(*a.c_args()))


def workspace_bytes(num_tokens: int, hidden: int) -> int:
    return int(lib().ewg_workspace_bytes(num_tokens, hidden))


def new_workspace(num_tokens: int, hidden: int, device=None) -> torch.Tensor:
    """A device buffer large enough for any call with these sizes (no init needed)."""
    nbytes = workspace_bytes(num_tokens, hidden)
    if nbytes == 0:
        raise EwgError(ERR_UNSUPPORTED, "unsupported num_tokens / hidden")
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def accumulate_embedding_wgrad(ids: torch.Tensor, grad: torch.Tensor, main_grad: torch.Tensor,
                               *, workspace: torch.Tensor | None = None,
                               check: bool = False) -> None:
    """main_grad += embedding_dense_backward(grad, ids), touching only the rows of ids.

    ids: token ids, any shape, num_tokens elements; grad: [*ids.shape, hidden];
    main_grad: [num_embeddings, hidden], updated in place.  Requires
    can_accumulate_embedding_wgrad(ids, grad, main_grad) (raises ValueError otherwise).
    The work is enqueued on the current stream.  With check=True the call waits for it
    and raises EwgError if the device found an id outside [0, num_embeddings), in which
    case main_grad was left untouched.
    """
    a = _Args(ids, grad, main_grad)
    if a.reason is not None:
        raise ValueError(f"accumulate_embedding_wgrad does not support these tensors: {a.reason}")
    with torch.cuda.device(a.device):
        L = lib()
        if not L.ewg_can_accumulate(*a.c_args()):
            raise ValueError("accumulate_embedding_wgrad does not support these tensors: "
                             + L.ewg_last_error().decode())
        ws = workspace if workspace is not None else new_workspace(a.n, a.H, a.device)
        stream = _stream_ptr(a.device)
        _raise_on(L.ewg_accumulate(*a.c_args(), ws.data_ptr(), ws.numel(), stream))
        if check:
            raise_on_device_status(ws)


def new_host_workspace(num_tokens: int, hidden: int, ids_dtype: torch.dtype,
                       grad_dtype: torch.dtype, device=None) -> torch.Tensor:
    """A device buffer for accumulate_embedding_wgrad_from_host with these sizes and dtypes."""
    nbytes = int(lib().ewg_host_workspace_bytes(num_tokens, hidden, _ID_CODES.get(ids_dtype, -1),
                                                _FLOAT_CODES.get(grad_dtype, -1)))
    if nbytes == 0:
        raise EwgError(ERR_UNSUPPORTED, "unsupported num_tokens / hidden / dtypes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def _keep_until_passed(stream, tensors) -> None:
    """Holds `tensors` until `stream` has passed the work enqueued so far; entries whose
    event has completed are dropped on every call."""
    ev = torch.cuda.Event()
    ev.record(stream)
    with _pending_lock:
        _pending_host[:] = [(e, t) for (e, t) in _pending_host if not e.query()]
        _pending_host.append((ev, tensors))


def accumulate_embedding_wgrad_from_host(ids: torch.Tensor, grad: torch.Tensor,
                                         main_grad: torch.Tensor, *,
                                         workspace: torch.Tensor | None = None,
                                         check: bool = False) -> None:
    """accumulate_embedding_wgrad with ids and grad in pinned host memory: the library
    copies them to the device (the grad copy overlapping the plan) and accumulates into
    main_grad on its device, all enqueued on the current stream.  ids: contiguous CPU
    int32/int64 tensor, grad: contiguous CPU bf16/fp32 tensor [*ids.shape, hidden], both
    pinned; main_grad: CUDA [num_embeddings, hidden].  check=True as in
    accumulate_embedding_wgrad.

    The copies run after the call returns.  This function keeps ids and grad alive until
    the stream has passed the call, so dropping them (or a temporary ``x.pin_memory()``)
    right away is safe; writing new values into them before the stream has passed the
    call is not (synchronize the stream, or wait on an event recorded after the call)."""
    if ids.is_cuda or grad.is_cuda or not main_grad.is_cuda:
        raise ValueError("ids and grad must be host tensors, main_grad a CUDA tensor")
    if not (ids.is_contiguous() and grad.is_contiguous() and ids.is_pinned() and grad.is_pinned()):
        raise ValueError("ids and grad must be contiguous pinned host tensors")
    if ids.dtype not in _ID_CODES or grad.dtype not in _FLOAT_CODES \
            or main_grad.dtype not in _FLOAT_CODES or main_grad.dim() != 2 or main_grad.stride(1) != 1:
        raise ValueError("unsupported dtypes or main_grad layout")
    V, H = main_grad.shape
    n = ids.numel()
    if tuple(grad.shape) != tuple(ids.shape) + (H,):
        raise ValueError("grad must be [*ids.shape, hidden]")
    with torch.cuda.device(main_grad.device):
        L = lib()
        ws = workspace if workspace is not None else new_host_workspace(n, H, ids.dtype, grad.dtype,
                                                                        main_grad.device)
        _raise_on(L.ewg_accumulate_host(
            ids.data_ptr(), _ID_CODES[ids.dtype], n, grad.data_ptr(), _FLOAT_CODES[grad.dtype],
            main_grad.data_ptr(), _FLOAT_CODES[main_grad.dtype], V, H,
            main_grad.stride(0) if V > 1 else H, ws.data_ptr(), ws.numel(),
            _stream_ptr(main_grad.device)))
        _keep_until_passed(torch.cuda.current_stream(main_grad.device), (ids, grad))
        if check:
            raise_on_device_status(ws)


def accumulate_embedding_wgrad_shard(ids: torch.Tensor, grad: torch.Tensor,
                                     main_grad_shard: torch.Tensor, row_begin: int,
                                     num_embeddings: int, *,
                                     workspace: torch.Tensor | None = None,
                                     check: bool = False) -> None:
    """accumulate_embedding_wgrad restricted to the table rows
    [row_begin, row_begin + main_grad_shard.shape[0]) of a num_embeddings-row table.

    main_grad_shard holds those rows (its row 0 is table row row_begin) and ends with
    the bits the whole-table call would give them; ids of other rows are skipped, ids
    outside [0, num_embeddings) are errors.  One GPU per row range needs no exchange.
    """
    a = _Args(ids, grad, main_grad_shard)
    if a.reason is not None:
        raise ValueError(f"accumulate_embedding_wgrad_shard does not support these tensors: {a.reason}")
    rows = a.V
    with torch.cuda.device(a.device):
        L = lib()
        ws = workspace if workspace is not None else new_workspace(a.n, a.H, a.device)
        args = list(a.c_args())
        args[8:9] = [num_embeddings, row_begin, rows]   # V -> (num_embeddings, row_begin, rows)
        _raise_on(L.ewg_accumulate_shard(*args, ws.data_ptr(), ws.numel(), _stream_ptr(a.device)))
        if check:
            raise_on_device_status(ws)


def read_status(workspace: torch.Tensor) -> int:
    """Waits for the current stream and returns the device status of the last call."""
    status = ctypes.c_int(-1)
    with torch.cuda.device(workspace.device):
        _raise_on(lib().ewg_read_status(workspace.data_ptr(), _stream_ptr(workspace.device),
                                        ctypes.byref(status)))
    return status.value


def raise_on_device_status(workspace: torch.Tensor) -> None:
    s = read_status(workspace)
    if s != OK:
        raise EwgError(s, f"device reported {lib().ewg_status_string(s).decode()}")


def plan(ids: torch.Tensor, num_embeddings: int, hidden: int, workspace: torch.Tensor) -> None:
    """Sort + run listing of ids into `workspace` (first half of the accumulation)."""
    ids_flat = ids.reshape(-1)
    if ids.dtype not in _ID_CODES or not ids.is_contiguous():
        raise ValueError("ids must be contiguous int32/int64")
    with torch.cuda.device(ids.device):
        _raise_on(lib().ewg_plan(ids_flat.data_ptr(), _ID_CODES[ids.dtype], ids_flat.numel(),
                                 num_embeddings, hidden, workspace.data_ptr(), workspace.numel(),
                                 _stream_ptr(ids.device)))


def apply(grad: torch.Tensor, main_grad: torch.Tensor, num_tokens: int,
          workspace: torch.Tensor) -> None:
    """Partial sums and the add into main_grad, using the plan in `workspace`."""
    V, H = main_grad.shape
    g2 = grad.view(num_tokens, H)
    with torch.cuda.device(main_grad.device):
        _raise_on(lib().ewg_apply(g2.data_ptr(), _FLOAT_CODES[grad.dtype],
                                  g2.stride(0) if num_tokens > 1 else H, main_grad.data_ptr(),
                                  _FLOAT_CODES[main_grad.dtype], num_tokens, V, H,
                                  main_grad.stride(0) if V > 1 else H, workspace.data_ptr(),
                                  workspace.numel(), _stream_ptr(main_grad.device)))


class TokenLogprobs(NamedTuple):
    """What token_logprobs returns: fp32 tensors of the targets' shape, and with `top` the
    alternatives ([*targets.shape, top] fp32 and int64, best first)."""
    logprobs: torch.Tensor
    entropy: torch.Tensor
    row_max: torch.Tensor          # largest logit of the row
    log_sum: torch.Tensor          # log of the sum of exp(scale * (logit - row_max))
    top_logprobs: Optional[torch.Tensor]
    top_ids: Optional[torch.Tensor]


def status_workspace(device=None) -> torch.Tensor:
    """The 256 device bytes in which token_logprobs and its backward leave their status."""
    return torch.empty(256, dtype=torch.uint8, device=device or "cuda")


# The current stream's handle without a Stream object around it (torch keeps this function
# for generated code; the ordinary way is the fallback).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


# The current device's index, asked for a tensor of some device (so that there is one).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _enqueue(index, call, *args):
    """call(*args, current stream) with device `index` current; raises on an error code."""
    if index == _current_device():
        code = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            code = call(*args, _raw_stream(index))
    if code != OK:
        _raise_on(code)


def _logits_args(name, logits, targets):
    """(device index, num_tokens, vocab, row stride) of logits [*targets.shape, vocab]."""
    index = logits.get_device()
    shape = logits.shape
    if index < 0 or targets.get_device() != index:
        reason = "logits and targets must be on one CUDA device"
    elif logits.dtype not in _FLOAT_CODES or targets.dtype not in _ID_CODES:
        reason = "logits must be bf16/fp32, targets int32/int64"
    elif len(shape) == 0 or shape[:-1] != targets.shape:
        reason = "logits must be [*targets.shape, vocab]"
    elif not targets.is_contiguous():
        reason = "targets must be contiguous"
    else:
        n, V = targets.numel(), shape[-1]
        return index, n, V, _row_stride(name, "logits", logits, n, V)
    raise ValueError(f"{name} does not support these tensors: {reason}")


def _row_stride(name, what, x, n, V):
    """The stride between the n rows of x [..., V], whose elements are neighbours."""
    if x.is_contiguous():
        return V
    if x.dim() != 2:
        try:
            x = x.view(n, V)
        except RuntimeError:
            x = None
    if x is None or (x.stride(1) != 1 and V > 1 and n > 0):
        raise ValueError(f"{name} does not support these tensors: {what} must have rows of unit "
                         "inner stride that share one row stride")
    return x.stride(0) if n > 1 else V


def _written(out):
    """Tells autograd that the library has written a caller's tensor (or several), so that a graph
    that saved what was there raises instead of using it."""
    torch.autograd.graph.increment_version(out)


def _status_ws(workspace, check, device):
    """(workspace, its pointer, its bytes); without one and without check there is none."""
    if workspace is None:
        if not check:
            return None, None, 0
        workspace = status_workspace(device)
    return workspace, workspace.data_ptr(), workspace.numel()


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, *, scale: float = 1.0,
                   top: int = 0, workspace: torch.Tensor | None = None,
                   check: bool = False) -> TokenLogprobs:
    """Log probabilities of `targets` under softmax(scale * logits), with entropies and the
    `top` most likely tokens of each row (see ewg_token_logprobs in include/ewg.h).

    logits: [*targets.shape, vocab], bf16 or fp32, rows of unit inner stride; targets:
    contiguous int32/int64.  A negative target marks a row without a token: its logprob,
    entropy, row_max and log_sum are 0 and its alternatives missing (id -1, -inf).  Logits
    of -inf are tokens that cannot occur.  The work is enqueued on the current stream; with
    check=True the call waits for it and raises EwgError if a target was vocab or more
    (whose logprob is NaN).  workspace: status_workspace(), to read the status later with
    read_status.

    The results carry no autograd graph, whether or not logits requires gradients: their
    gradient is token_logprobs_backward, for the caller's own torch.autograd.Function or
    training step.
    """
    index, n, V, stride = _logits_args("token_logprobs", logits, targets)
    if not 0 <= top <= min(V, MAX_TOP):
        raise ValueError(f"top must be in [0, min(vocab, {MAX_TOP})]")
    device, shape = logits.device, targets.shape
    # (separate allocations: views of one take longer to make)
    first = torch.empty(shape, dtype=torch.float32, device=device)
    stats = (first, torch.empty_like(first), torch.empty_like(first), torch.empty_like(first))
    top_logprobs = top_ids = None
    if top:
        top_logprobs = torch.empty((*shape, top), dtype=torch.float32, device=device)
        top_ids = torch.empty((*shape, top), dtype=torch.int64, device=device)
    ws, ws_ptr, ws_bytes = _status_ws(workspace, check, device)
    _enqueue(index, lib().ewg_token_logprobs, logits.data_ptr(), _FLOAT_CODES[logits.dtype], stride,
             targets.data_ptr(), _ID_CODES[targets.dtype], n, V, scale, top,
             *[s.data_ptr() for s in stats], top_logprobs.data_ptr() if top else None,
             top_ids.data_ptr() if top else None, ws_ptr, ws_bytes)
    if check and n:
        raise_on_device_status(ws)
    return TokenLogprobs(*stats, top_logprobs, top_ids)


def token_logprobs_backward(logits: torch.Tensor, targets: torch.Tensor, row_max: torch.Tensor,
                            log_sum: torch.Tensor, grad_logprobs: torch.Tensor, *,
                            entropy: torch.Tensor | None = None,
                            grad_entropy: torch.Tensor | None = None, scale: float = 1.0,
                            out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None,
                            check: bool = False) -> torch.Tensor:
    """The gradient of token_logprobs' logprobs (and, with grad_entropy, entropies) with
    respect to the logits, in the logits' dtype (see ewg_token_logprobs_backward in
    include/ewg.h).

    row_max, log_sum and entropy are what token_logprobs returned for these logits, targets
    and scale; grad_logprobs and grad_entropy are fp32 of the targets' shape (entropy is only
    read with grad_entropy).  out: where to write; out=logits replaces the logits.  Without
    it the gradient is allocated, with the logits' row padding where that is less than an
    eighth of a row.  Padding rows get zeros.  (Autograd is told that out was written: a graph
    that saved the logits replaced by it raises in its backward pass.)
    """
    index, n, V, stride = _logits_args("token_logprobs_backward", logits, targets)
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs the forward call's entropy")
    shape = targets.shape
    for t in (row_max, log_sum, grad_logprobs) if grad_entropy is None else \
            (row_max, log_sum, grad_logprobs, entropy, grad_entropy):
        if t.shape != shape or t.dtype != torch.float32 or t.get_device() != index \
                or not t.is_contiguous():
            raise ValueError("row_max, log_sum, entropy and the incoming gradients must be contiguous "
                             "fp32 tensors of the targets' shape on the logits' device")
    given = out is not None
    if not given:
        if stride == V or stride > V + V // 8:
            out, out_stride = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device), V
        else:
            # rows placed like the logits' rows, so that both are read and written in whole vectors
            out = torch.empty((*shape, stride), dtype=logits.dtype, device=logits.device)[..., :V]
            out_stride = stride
    else:
        if out.shape != logits.shape or out.dtype != logits.dtype or out.get_device() != index:
            raise ValueError("out must have the logits' shape, dtype and device")
        out_stride = _row_stride("token_logprobs_backward", "out", out, n, V)
    ws, ws_ptr, ws_bytes = _status_ws(workspace, check, logits.device)
    both = grad_entropy is not None
    _enqueue(index, lib().ewg_token_logprobs_backward, logits.data_ptr(), _FLOAT_CODES[logits.dtype],
             stride, targets.data_ptr(), _ID_CODES[targets.dtype], n, V, scale, row_max.data_ptr(),
             log_sum.data_ptr(), entropy.data_ptr() if both else None, grad_logprobs.data_ptr(),
             grad_entropy.data_ptr() if both else None, out.data_ptr(), out_stride, ws_ptr, ws_bytes)
    if given:
        _written(out)
    if check and n:
        raise_on_device_status(ws)
    return out


def orthogonalize_workspace(shape, device=None) -> torch.Tensor:
    """A device buffer for orthogonalize_update of a tensor of this shape (no init needed)."""
    *lead, rows, cols = shape
    batch = 1
    for d in lead:
        batch *= d
    nbytes = int(lib().ewg_orthogonalize_workspace_bytes(max(batch, 1), rows, cols))
    if nbytes == 0:
        raise EwgError(ERR_UNSUPPORTED, "unsupported sizes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def _matrices(what, x):
    """x [..., rows, cols] as [batch, rows, cols] with unit inner stride; no copy."""
    try:
        x3 = x.view(-1, *x.shape[-2:]) if x.dim() != 2 else x[None]
    except RuntimeError:
        x3 = None
    if x3 is None or (x3.stride(2) != 1 and x3.shape[2] > 1):
        raise ValueError(f"orthogonalize_update does not support these tensors: {what} must have "
                         "unit inner stride and leading dimensions that share one stride")
    return x3


def orthogonalize_update(grad: torch.Tensor, *, steps: int = 5,
                         coefficients: tuple = (3.4445, -4.7750, 2.0315),
                         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         check: bool = False) -> torch.Tensor:
    """Newton-Schulz orthogonalisation of each [rows, cols] matrix of grad, in bf16 (see
    ewg_orthogonalize in include/ewg.h): `steps` times X <- a X + (b A + c A^2) X with
    A = X X^T, from X = grad / |grad|.

    grad: [..., rows, cols] bf16 or fp32 (leading dimensions are a batch of matrices; a
    transposed matrix is taken as such); out: bf16 of the same shape, whose rows or columns are
    contiguous, apart from grad.  The work is enqueued on the current stream.  workspace:
    orthogonalize_workspace(grad.shape), allocated when not given.  check=True waits and raises
    EwgError if a wait on the device gave up.
    """
    if not grad.is_cuda or grad.dtype not in _FLOAT_CODES or grad.dim() < 2:
        raise ValueError("orthogonalize_update does not support these tensors: grad must be "
                         "[..., rows, cols], bf16/fp32, on a CUDA device")
    if out is not None and (out.shape != grad.shape or out.dtype != torch.bfloat16
                            or out.device != grad.device):
        raise ValueError("out must be bf16 of grad's shape on grad's device")
    if grad.stride(-1) != 1 and grad.stride(-2) == 1 and grad.shape[-1] > 1:
        # a transposed matrix: the steps of the transpose give the transpose
        return orthogonalize_update(grad.mT, steps=steps, coefficients=coefficients,
                                    out=None if out is None else out.mT, workspace=workspace,
                                    check=check).mT
    given = out is not None
    if not given:
        out = torch.empty(grad.shape, dtype=torch.bfloat16, device=grad.device)
    if grad.numel() == 0 and 0 not in grad.shape[-2:]:
        return out
    call, o = lib().ewg_orthogonalize, out
    if out.stride(-1) != 1 and out.stride(-2) == 1 and out.shape[-1] > 1:
        call, o = lib().ewg_orthogonalize_transposed, out.mT     # the other way round than grad
    g3, o3 = _matrices("grad", grad), _matrices("out", o)
    batch, rows, cols = g3.shape
    ws = workspace if workspace is not None else orthogonalize_workspace(grad.shape, grad.device)
    _enqueue(grad.get_device(), call, g3.data_ptr(), _FLOAT_CODES[grad.dtype],
             batch, rows, cols, g3.stride(0), g3.stride(1), o3.data_ptr(), o3.stride(0),
             o3.stride(1), steps, *coefficients, ws.data_ptr(), ws.numel())
    if given:
        _written(out)
    if check:
        raise_on_device_status(ws)
    return out


class LayerNorm(NamedTuple):
    """What layer_norm returns: the normalised rows, and fp32 tensors of x.shape[:-1] that
    layer_norm_backward takes (None without stats)."""
    out: torch.Tensor
    mean: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]   # 1 / sqrt(variance + eps)


# (These calls are often bound by the host, so that their checks are few and taken once.)
def _norm_input(name, x):
    """(device index, hidden, rows, row stride, dtype code) of x [..., hidden]."""
    index, code = x.get_device(), _FLOAT_CODES.get(x.dtype)
    H = x.shape[-1] if x.dim() else 0
    if index < 0 or code is None or H == 0:
        raise ValueError(f"{name} does not support these tensors: x must be [..., hidden], bf16/fp32, "
                         "on a CUDA device")
    n = x.numel() // H
    return index, H, n, H if x.is_contiguous() else _row_stride(name, "x", x, n, H), code


def _norm_rows(name, what, y, x, n, H):
    """The row stride of y, which has x's shape, dtype and device."""
    if y.dtype != x.dtype or y.shape != x.shape or y.get_device() != x.get_device():
        raise ValueError(f"{name} does not support these tensors: {what} must have x's shape, dtype "
                         "and device")
    return H if y.is_contiguous() else _row_stride(name, what, y, n, H)


def _norm_vectors(name, what, v, w, H, index):
    """(pointer of v, pointer of w, dtype code) of two vectors [H], each of which may be None."""
    if v is None:
        v, w = w, None
        if v is None:
            return None, None, _FP32
        return (None, *_norm_vectors(name, what, v, None, H, index)[::2])
    dtype = v.dtype
    code = _FLOAT_CODES.get(dtype)
    if code is None or v.shape != (H,) or v.get_device() != index or not v.is_contiguous() or (
            w is not None and (w.dtype != dtype or w.shape != (H,) or w.get_device() != index
                               or not w.is_contiguous())):
        raise ValueError(f"{name} does not support these tensors: {what} must be contiguous [hidden] "
                         "vectors of one dtype, bf16/fp32, on x's device")
    return v.data_ptr(), None if w is None else w.data_ptr(), code


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, *, eps: float = 1e-5, stats: bool = True,
               out: torch.Tensor | None = None) -> LayerNorm:
    """Each row of x [..., hidden] less its mean, over its standard deviation, times weight, plus
    bias (see ewg_layer_norm in include/ewg.h), with the rows' means and 1 / standard deviations.

    x: bf16 or fp32, rows of unit inner stride; weight and bias: contiguous [hidden], both bf16 or
    both fp32, whatever x is (without them ones and zeros); out: where to write, of x's shape and
    dtype; out=x replaces x.  stats=False leaves out the means and standard deviations, where
    nothing goes back through the rows.  The work is enqueued on the current stream.

    The results carry no autograd graph: their gradient is layer_norm_backward.
    """
    index, H, n, stride, x_code = _norm_input("layer_norm", x)
    w, b, code = _norm_vectors("layer_norm", "weight and bias", weight, bias, H, index)
    given = out is not None
    if given:
        out_stride = _norm_rows("layer_norm", "out", out, x, n, H)
    else:
        out_stride = H
        out = torch.empty_like(x) if stride == H else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    mean = rstd = mean_ptr = rstd_ptr = None
    if stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        mean_ptr, rstd_ptr = mean.data_ptr(), rstd.data_ptr()
    _enqueue(index, lib().ewg_layer_norm, x.data_ptr(), x_code, n, H, stride, w, b, code, eps,
             out.data_ptr(), out_stride, mean_ptr, rstd_ptr)
    if given:
        _written(out)
    return LayerNorm(out, mean, rstd)


def layer_norm_workspace(shape, device=None) -> torch.Tensor:
    """A device buffer for layer_norm_backward of rows of this shape (no init needed)."""
    rows = 1
    for d in shape[:-1]:
        rows *= d
    nbytes = int(lib().ewg_layer_norm_workspace_bytes(rows, shape[-1]))
    if nbytes == 0:
        raise EwgError(ERR_UNSUPPORTED, "unsupported sizes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def layer_norm_backward(grad: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, *,
                        weight_main_grad: torch.Tensor | None = None,
                        bias_main_grad: torch.Tensor | None = None,
                        out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of layer_norm with respect to x, in x's dtype; the weight's and the bias's are
    added to weight_main_grad and bias_main_grad where these are given (see
    ewg_layer_norm_backward in include/ewg.h).

    grad: of x's shape and dtype; mean and rstd: what layer_norm returned for x; weight: as given to
    it.  The main_grads are contiguous [hidden], both bf16 or both fp32, whatever the weight
    is.  out: where to write; out=grad or out=x replaces it.  workspace:
    layer_norm_workspace(x.shape), allocated when not given; calls that may run at the same time (two
    streams, two captured graphs) need one each.  The work is enqueued on the current stream; the
    same call gives the same bits.
    """
    name = "layer_norm_backward"
    index, H, n, x_stride, x_code = _norm_input(name, x)
    grad_stride = _norm_rows(name, "grad", grad, x, n, H)
    lead = x.shape[:-1]
    for t in (mean, rstd):
        if t.shape != lead or t.dtype != torch.float32 or t.get_device() != index or not t.is_contiguous():
            raise ValueError("mean and rstd must be contiguous fp32 tensors of x.shape[:-1] on x's device")
    w, _, w_code = _norm_vectors(name, "weight", weight, None, H, index)
    mg_w, mg_b, m_code = _norm_vectors(name, "main_grads", weight_main_grad, bias_main_grad, H, index)
    given = out is not None
    if given:
        out_stride = _norm_rows(name, "out", out, x, n, H)
    else:
        out_stride = H
        out = torch.empty_like(x) if x_stride == H else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if n == 0:
        return out
    L = lib()
    if workspace is None:
        nbytes = L.ewg_layer_norm_workspace_bytes(n, H)
        if nbytes == 0:
            raise EwgError(ERR_UNSUPPORTED, "unsupported sizes")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    _enqueue(index, L.ewg_layer_norm_backward, grad.data_ptr(), grad_stride, x.data_ptr(), x_stride,
             x_code, n, H, mean.data_ptr(), rstd.data_ptr(), w, w_code, out.data_ptr(), out_stride,
             mg_w, mg_b, m_code, workspace.data_ptr(), workspace.numel())
    for t, written in ((out, given), (weight_main_grad, mg_w), (bias_main_grad, mg_b)):
        if written:
            _written(t)
    return out


class _AdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("count", ctypes.c_int64), ("weight_decay", ctypes.c_double),
                ("param_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int)]


_data_ptr = torch.Tensor.data_ptr
_storage_ptr = torch.UntypedStorage.data_ptr


class AdamWPlan:
    """What adamw_plan makes: the tensors of an AdamW step, checked, with their states.

    params, grads, copies: the tensors given; exp_avg, exp_avg_sq, scales: lists of the states, of
    each param's shape (scales: [blocks, 2] fp32, None in 32 bits).  state_bits 32: exp_avg and
    exp_avg_sq are fp32.  state_bits 8: they are float8_e4m3fn, and element i of a flattened
    tensor has the average exp_avg[i] * scales[i // ADAMW_BLOCK, 0] and the second average
    (exp_avg_sq[i] * scales[i // ADAMW_BLOCK, 1]) ** 2.
    """

    def __init__(self, params, grads, copies, exp_avg, exp_avg_sq, scales, state_bits, index):
        self.params, self.grads, self.copies = params, grads, copies
        self.exp_avg, self.exp_avg_sq, self.scales = exp_avg, exp_avg_sq, scales
        self.state_bits = state_bits
        self._index = index
        self._all = [t for group in (params, grads, exp_avg, exp_avg_sq, scales or (), copies or ())
                     for t in group if t is not None]
        # Every step looks whether all tensors are where they were, and whether the memory that they were in is: it is
        # held, but may have been resized, and a tensor that was put elsewhere lie in what became of it.
        storages = {}
        for t in self._all:
            storage = t.untyped_storage()
            storages[storage._cdata] = storage
        self._storages = list(storages.values())
        self._addresses = self._places()
        self._written = [t for group in (params, exp_avg, exp_avg_sq, scales or (), copies or ())
                         for t in group if t is not None]
        self._buffer = None            # of ewg_adamw_plan, and its bytes
        self._bytes = 0

    def _places(self):
        return [*map(_data_ptr, self._all), *map(_storage_ptr, self._storages)]


def _state_list(name, given, params, dtype, shapes):
    if given is None:
        return [torch.zeros(s, dtype=dtype, device=p.device) for s, p in zip(shapes, params)]
    given = list(given)
    if len(given) != len(params) or any(t.shape != torch.Size(s) or t.dtype != dtype for t, s in zip(given, shapes)):
        raise ValueError(f"{name} must hold a {dtype} tensor of the right shape for each param")
    return given


def adamw_plan(params, grads, *, state_bits: int = 32, copies=None, weight_decay=0.01,
               exp_avg=None, exp_avg_sq=None, scales=None) -> AdamWPlan:
    """Prepares AdamW steps of `params` (see ewg_adamw_plan in include/ewg.h) and makes their states.

    params: bf16 or fp32 CUDA tensors of any shape, contiguous, of one device; grads: their
    main_grads, bf16 or fp32, from which every adamw_step reads (the tensors, not only their present
    values: a plan holds addresses); copies: a bf16 tensor (or None) for each param that is fp32,
    which receives the new param rounded; weight_decay: a number, or one for each param.
    state_bits: 32, or 8 (with a scale for every ADAMW_BLOCK elements).  exp_avg, exp_avg_sq and
    scales: states to go on from, shaped as AdamWPlan says; zeros without them.

    The plan holds the tensors; steps update the params, states and copies in place.
    """
    params, grads = list(params), list(grads)
    if state_bits not in (8, 32):
        raise ValueError("state_bits must be 8 or 32")
    if len(grads) != len(params):
        raise ValueError("grads must hold a tensor for each param")
    copies = [None] * len(params) if copies is None else list(copies)
    decays = [float(weight_decay)] * len(params) if isinstance(weight_decay, (int, float)) else list(weight_decay)
    if len(copies) != len(params) or len(decays) != len(params):
        raise ValueError("copies and weight_decay must hold an element for each param")
    index = params[0].get_device() if params else None
    for p, g, c in zip(params, grads, copies):
        if p.get_device() < 0 or p.dtype not in _FLOAT_CODES or g.dtype not in _FLOAT_CODES:
            raise ValueError("adamw_plan does not support these tensors: params and grads must be "
                             "bf16/fp32, on a CUDA device")
        if g.shape != p.shape or (c is not None and (c.shape != p.shape or c.dtype != torch.bfloat16
                                                     or p.dtype != torch.float32)):
            raise ValueError("grads must have the params' shapes; copies too, bf16 beside fp32 params")
    shapes = [p.shape for p in params]
    dtype = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
    exp_avg = _state_list("exp_avg", exp_avg, params, dtype, shapes)
    exp_avg_sq = _state_list("exp_avg_sq", exp_avg_sq, params, dtype, shapes)
    if state_bits == 8:
        blocks = [(-(-p.numel() // ADAMW_BLOCK), 2) for p in params]
        scales = _state_list("scales", scales, params, torch.float32, blocks)
    elif scales is not None:
        raise ValueError("scales belong to states in 8 bits")
    plan = AdamWPlan(params, grads, copies, exp_avg, exp_avg_sq, scales, state_bits, index)
    for t in plan._all:
        if t.get_device() != index or not t.is_contiguous():
            raise ValueError("adamw_plan does not support these tensors: all must be contiguous, on one device")
        if t.is_inference():
            raise ValueError("adamw_plan does not support these tensors: inference tensors cannot be "
                             "updated in place")
    L = lib()
    table = (_AdamWTensor * max(1, len(params)))()
    for k, t in enumerate(table[:len(params)]):
        t.param, t.grad = params[k].data_ptr(), grads[k].data_ptr()
        t.exp_avg, t.exp_avg_sq = exp_avg[k].data_ptr(), exp_avg_sq[k].data_ptr()
        t.scales = scales[k].data_ptr() if scales is not None else None
        t.copy = copies[k].data_ptr() if copies[k] is not None else None
        t.count, t.weight_decay = params[k].numel(), decays[k]
        t.param_dtype, t.grad_dtype = _FLOAT_CODES[params[k].dtype], _FLOAT_CODES[grads[k].dtype]
        table[k] = t
    nbytes = int(L.ewg_adamw_plan_bytes(len(params)))
    plan._buffer, plan._bytes = (ctypes.c_uint64 * (nbytes // 8 + 1))(), nbytes
    if params:
        with torch.cuda.device(index):
            _raise_on(L.ewg_adamw_plan(table, len(params), state_bits, plan._buffer, nbytes))
    return plan


def _scalar(name, value, dtype, index):
    """(value, pointer) of a number or of a device scalar."""
    if not isinstance(value, torch.Tensor):
        return int(value) if dtype == torch.int64 else float(value), None
    if value.numel() != 1 or value.dtype != dtype or value.get_device() != index:
        raise ValueError(f"{name} must be a number, or one {dtype} element on the params' device")
    return 0, value.data_ptr()


def adamw_step(plan: AdamWPlan, step, *, lr, betas: tuple = (0.9, 0.999), eps: float = 1e-8,
               grad_scale=1.0) -> None:
    """One AdamW step of a plan's tensors (see ewg_adamw_step in include/ewg.h), the `step`-th from 1.

    grad_scale multiplies the gradients: a clipping factor, or the inverse of a loss scale.  step
    (int64), lr and grad_scale (fp32) may be CUDA tensors of one element, which the step reads on
    the device: a captured step then follows their values (they may not lie in what the step
    writes).  The work is enqueued on the current stream.  Raises ValueError if a tensor of the plan
    has moved to another address, or the memory that it was in has been given back.
    """
    if not plan.params:
        return
    if plan._places() != plan._addresses:
        raise ValueError("a tensor of the plan has moved to another address: make a new plan")
    index = plan._index
    step, step_ptr = _scalar("step", step, torch.int64, index)
    lr, lr_ptr = _scalar("lr", lr, torch.float32, index)
    grad_scale, scale_ptr = _scalar("grad_scale", grad_scale, torch.float32, index)
    _enqueue(index, lib().ewg_adamw_step, plan._buffer, plan._bytes, step, step_ptr, lr, lr_ptr,
             *betas, eps, grad_scale, scale_ptr)
    _written(plan._written)
