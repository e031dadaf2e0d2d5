"""GB300 (sm_103a) fused cross-entropy -- Python binding of ``libfoak_ce.so``.

The library is the FastCrossEntropyLoss of the fms-acceleration FOAK plugin
(fms-acceleration PR #79, Description item 4) rebuilt as hand-written CUDA for
sm_103a behind a C ABI (``include/foak_ce.h``).  This module only marshals
arguments: it takes torch tensors for device memory and the current stream,
passes their pointers through ctypes, and raises on a non-zero status.  Every
step of the computation runs in the library's kernels; there is no CPU or
PyTorch fallback -- importing fails loudly when the library is missing.

Build it with ``python -c "import __graft_entry__ as g; g.build()"`` (or
``cross_entropy_loss_gb300._build.build()``).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

from . import _build

LIB_PATH = _build.LIB

FOAK_OK = 0
FOAK_ERR_INVALID_ARG = 1
FOAK_ERR_UNSUPPORTED = 2
FOAK_ERR_LABEL_RANGE = 3
FOAK_ERR_WORKSPACE = 4
FOAK_ERR_CUDA = 5
FOAK_ERR_TIMEOUT = 6
FOAK_ERR_PAGE_RANGE = 7
FOAK_F32 = 0
FOAK_BF16 = 1
FOAK_ERRBIT_LABEL_RANGE = 1
FOAK_ERRBIT_TIMEOUT = 2
FOAK_ERRBIT_PAGE_RANGE = 4

# C entry points and their ctypes signatures (restype, argtypes).
_vp, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "foak_status_string": (ctypes.c_char_p, [_i32]),
    "foak_abi_version": (_i32, []),
    "foak_ce_max_vocab": (_i64, [_i32]),
    "foak_ce_workspace_size": (_sz, [_i64]),
    "foak_ce_forward": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                               _vp]),
    "foak_ce_backward": (_i32, [_vp, _vp, _i32, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _f32, _vp, _vp]),
    "foak_rmsnorm_forward": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _f32, _vp, _i64, _vp, _vp]),
    "foak_rmsnorm_workspace_size": (_sz, [_i64]),
    "foak_rmsnorm_backward": (_i32, [_vp, _i64, _vp, _i64, _vp, _vp, _i32, _i64, _i64, _vp, _i64, _vp, _vp, _sz,
                                     _vp]),
    "foak_rmsnorm_linear_ce_workspace_size": (_sz, [_i64, _i64, _i64, _i64]),
    "foak_rmsnorm_linear_ce_chunked": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _f32, _f32, _f32,
                                              _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "foak_rope_cache_size": (_sz, [_i64, _i64]),
    "foak_rope_build_cache": (_i32, [ctypes.c_double, _i64, _i64, _vp, _sz, _vp]),
    "foak_rope_apply": (_i32, [_vp, _i32, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _vp]),
    "foak_rope_apply_qk": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _i64, _i64, _vp, _vp, _i64, _i32, _vp,
                                  _vp]),
    "foak_ce_host_workspace_size": (_sz, [_i64]),
    "foak_ce_fwd_bwd_host": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i64, _f32, _f32, _vp, _vp, _vp, _vp, _vp, _vp,
                                    _sz, _vp]),
    "foak_ce_fwd_bwd": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i64, _f32, _f32, _vp, _vp, _vp, _vp, _vp, _sz,
                               _vp]),
    "foak_ce_count_valid": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "foak_ce_fwd_bwd_devdenom": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _sz, _vp]),
    "foak_ce_fwd_bwd_noalloc": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i64, _f32, _f32, _vp, _vp, _vp, _vp,
                                       _vp]),
    "foak_gemm_bf16": (_i32, [_vp, _i64, _i32, _vp, _i64, _i32, _i64, _i64, _i64, _vp, _i64, _i32, _vp, _vp]),
    "foak_gemm_bf16_group": (_i32, [_vp, _i32, _vp, _vp]),
    "foak_test_gemm_group_schedule": (_i32, [_vp, _i32, _i32, _vp, _vp, _i32]),
    "foak_linear_ce_workspace_size": (_sz, [_i64, _i64, _i64, _i64]),
    "foak_linear_ce_chunked": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _f32, _f32, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _sz, _vp]),
    "foak_logprobs_workspace_size": (_sz, []),
    "foak_logprobs_forward": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i64, _f32, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _vp, _sz, _vp]),
    "foak_logprobs_backward": (_i32, [_vp, _vp, _i32, _i64, _vp, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp,
                                      _vp]),
    "foak_distill_forward": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _i32, _f32, _f32,
                                    _f32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "foak_distill_fwd_bwd": (_i32, [_vp, _vp, _i32, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _i32, _f32,
                                    _f32, _f32, _f32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "foak_distill_backward": (_i32, [_vp, _vp, _i32, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _i32, _f32,
                                     _f32, _f32, _vp, _vp, _f32, _vp, _vp]),
    "foak_residual_norm_forward": (_i32, [_vp, _i64, _vp, _i64, _i32, _i64, _i64, _vp, _i32, _i64, _vp, _vp, _f32, _f32,
                                          _f32, _vp, _i64, _vp, _i64, _vp, _vp, _vp]),
    "foak_residual_norm_workspace_size": (_sz, [_i64, _i64]),
    "foak_residual_norm_backward": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i64, _vp, _i32, _i64,
                                           _vp, _vp, _vp, _vp, _f32, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _sz,
                                           _vp]),
    "foak_rotary_inv_freq": (_i32, [ctypes.c_double, _i64, _i32, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                    ctypes.c_double, _vp]),
    "foak_rotary_turns": (_i32, [_vp, _i64, _vp]),
    "foak_rotary_apply": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _i32,
                                 _i64, _i64, _i64, _i32, _vp, _vp, _f32, _i32, _vp]),
    "foak_kv_slots": (_i32, [_vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "foak_kv_append": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i32, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _i64,
                              _vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i32, _vp,
                              _vp, _f32, _vp, _vp]),
    "foak_test_fail_next_launches": (None, [_i32]),
    "foak_test_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "foak_test_skip_row_load": (None, [_i64]),
    "foak_test_set_row_path": (None, [_i32]),
}


class FoakError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"cross_entropy_loss_gb300: {LIB_PATH} is missing; build it first "
            "(python -c 'import __graft_entry__ as g; g.build()'). There is no fallback path.")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.foak_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != FOAK_OK:
        raise FoakError(status, where)


@functools.lru_cache(maxsize=1024)  # a number of N alone; the foreign call takes as long as a small allocation
def foak_ce_workspace_size(N: int) -> int:
    return int(lib.foak_ce_workspace_size(int(N)))


def foak_ce_max_vocab(dtype: int) -> int:
    return int(lib.foak_ce_max_vocab(int(dtype)))


# --------------------------------------------------------------------- torch glue
import torch  # noqa: E402  (device memory and streams only)

_DT = {torch.bfloat16: FOAK_BF16, torch.float32: FOAK_F32}
_ws_lock = threading.Lock()
_ws_cache: dict = {}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device, stream):
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# The current stream's handle without a Stream object, where torch has it (a call of a few
# microseconds' work spends two of them on the object).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(device, stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _addr(t):
    return None if t is None else t.data_ptr()


def _tensors_of(out):
    if isinstance(out, torch.Tensor):
        return [out]
    values = out.values() if isinstance(out, dict) else out if isinstance(out, (tuple, list)) else ()
    return [t.turns if isinstance(t, RotaryPlan) else t for t in values if isinstance(t, (torch.Tensor, RotaryPlan))]


def _on_stream(call):
    """Run ``call`` with its ``stream`` argument as the current stream.

    What the call allocates (outputs, error word, workspace) is written on that stream, so it
    has to come from memory whose earlier uses that stream has behind it: memory of the
    caller's stream may still be in use there, and an output that the caller drops at once
    would be given out again while the kernel has yet to write it.  The outputs are held until
    the caller's stream has passed its uses of them, too.  (The caller makes one stream wait
    for the other, before the call and before reading its outputs.)
    """
    @functools.wraps(call)
    def run(*args, stream=None, **kwargs):
        return call(*args, **kwargs) if stream is None else _run_on(stream, call, args, kwargs)

    return run


def _run_on(stream, call, args, kwargs):
    """What :func:`_on_stream` does with a stream that was given."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    before = torch.cuda.current_stream(stream.device)
    if before.cuda_stream == stream.cuda_stream:
        return call(*args, **kwargs)
    with torch.cuda.stream(stream):
        out = call(*args, **kwargs)
    for t in _tensors_of(args) + _tensors_of(kwargs):
        if t.is_cuda:
            t.record_stream(stream)
    for t in _tensors_of(out):
        if t.is_cuda:
            t.record_stream(before)
    return out


def _logits_args(logits):
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be a 2-D tensor with unit column stride (N x V, row stride ld)")
    if logits.dtype not in _DT:
        raise TypeError("logits must be bfloat16 or float32")
    if not logits.is_cuda:
        raise ValueError("logits must be on a CUDA device")
    N, V = logits.shape
    ld = logits.stride(0) if N > 1 else max(V, logits.stride(0))
    return N, V, ld, _DT[logits.dtype]


def _labels_arg(labels, N, device):
    if labels.dtype != torch.int64 or labels.dim() != 1 or labels.numel() != N or not labels.is_contiguous():
        raise ValueError("labels must be a contiguous int64 vector of length N")
    if labels.device != device:
        raise ValueError("labels must live on the logits' device")
    return labels


def _cached_workspace(cache: dict, need: int, device, handle, fill=torch.zeros) -> torch.Tensor:
    """A buffer of ``need`` bytes or more, zeros before its first use: the current stream's own in
    ``cache`` (``handle`` is the stream's), or a new one while that stream is captured into a graph.

    The calls of a stream run one after another and leave the buffer zeroed; calls of
    two streams may overlap, and must not count in one header.  A graph's replays overlap with
    anything, and outlive a cached buffer that a larger call replaces: each captured call has a
    buffer of the graph's memory, filled by the graph.
    """
    if handle and torch.cuda.is_current_stream_capturing():  # the legacy stream, 0, cannot be
        return fill(need, dtype=torch.uint8, device=device)
    key = (device, handle)
    ws = cache.get(key)
    if ws is None or ws.numel() < need:
        with _ws_lock:
            ws = cache.get(key)
            if ws is None or ws.numel() < need:
                ws = cache[key] = fill(max(need, 4096), dtype=torch.uint8, device=device)
    return ws


def workspace(N: int, device) -> torch.Tensor:
    """A zero-filled, reusable workspace of at least foak_ce_workspace_size(N) bytes for the
    device's current stream.

    Calls leave it zeroed again, so the cached buffer serves every call on that stream; calls
    on another stream get another one.  While the stream is captured into a graph every call of
    this function gives a new buffer, which the graph fills with zeros: pass ``workspace_tensor``
    to captured calls to be without that step, one buffer for the graph's calls on one stream.
    """
    dev = _device_of(device)
    return _cached_workspace(_ws_cache, foak_ce_workspace_size(N), dev, _stream_handle(dev, None))


def _workspace_arg(ws, device) -> torch.Tensor:
    if ws.device != device:
        raise ValueError("workspace_tensor must live on the logits' device")
    return ws


def _workspace_or_cached(ws, need: int, device, handle) -> torch.Tensor:
    return _cached_workspace(_ws_cache, need, device, handle) if ws is None else _workspace_arg(ws, device)


def _device_of(device) -> torch.device:
    dev = torch.device(device)
    return torch.device(dev.type, torch.cuda.current_device()) if dev.type == "cuda" and dev.index is None else dev


@_on_stream
def foak_ce_forward(logits, labels, *, ignore_index: int = -100, denom: float = 0.0, want_lse: bool = True,
                    want_row_loss: bool = False, workspace_tensor=None, stream=None):
    """Mean CE loss over non-ignored rows.  Returns dict(loss, lse, row_loss, n_valid, err)."""
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_arg(labels, N, dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    n_valid = torch.empty(1, dtype=torch.int32, device=dev)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev) if want_lse else None
    row_loss = torch.empty(N, dtype=torch.float32, device=dev) if want_row_loss else None
    ws = workspace(N, dev) if workspace_tensor is None else workspace_tensor
    st = lib.foak_ce_forward(_ptr(logits), dt, ld, _ptr(labels), N, V, int(ignore_index), float(denom), _ptr(loss),
                             _ptr(lse), _ptr(row_loss), _ptr(n_valid), _ptr(err), _ptr(ws), ws.numel(),
                             _stream(dev, stream))
    _check(st, "foak_ce_forward")
    return dict(loss=loss, lse=lse, row_loss=row_loss, n_valid=n_valid, err=err)


@_on_stream
def foak_ce_backward(logits, labels, lse, grad_out=None, *, dlogits=None, ignore_index: int = -100,
                     denom: float = 0.0, stream=None):
    """dlogits = (softmax - onehot) * g / D.  Pass ``dlogits=logits`` to overwrite in place."""
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_arg(labels, N, dev)
    if dlogits is None:
        # same row stride and the same offset modulo 16 bytes as logits (the kernels share row geometry)
        es = logits.element_size()
        shift = (logits.data_ptr() % 16) // es
        n = ((N - 1) * ld + V + shift) if N > 0 else 1
        base = torch.empty(n, dtype=logits.dtype, device=dev)
        dlogits = base.as_strided((N, V), (ld, 1), storage_offset=shift)
    if dlogits.shape != logits.shape or dlogits.stride() != logits.stride() or dlogits.dtype != logits.dtype:
        raise ValueError("dlogits must match logits in shape, strides and dtype")
    if lse.dtype != torch.float32 or lse.numel() != N or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 vector of length N")
    if grad_out is not None and (grad_out.dtype != torch.float32 or grad_out.numel() != 1):
        raise ValueError("grad_out must be a float32 scalar tensor")
    err = torch.empty(1, dtype=torch.int32, device=dev)
    st = lib.foak_ce_backward(_ptr(dlogits), _ptr(logits), dt, ld, _ptr(labels), N, V, int(ignore_index), _ptr(lse),
                              _ptr(grad_out), float(denom), _ptr(err), _stream(dev, stream))
    _check(st, "foak_ce_backward")
    return dlogits, err


@_on_stream
def foak_ce_fwd_bwd(logits, labels, *, g: float = 1.0, ignore_index: int = -100, denom: float = 0.0,
                    want_lse: bool = False, workspace_tensor=None, stream=None):
    """Fused forward + backward in place: ``logits`` is overwritten by dlogits.

    Returns dict(loss, n_valid, err, lse).
    """
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_arg(labels, N, dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    n_valid = torch.empty(1, dtype=torch.int32, device=dev)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev) if want_lse else None
    ws = workspace(N, dev) if workspace_tensor is None else workspace_tensor
    st = lib.foak_ce_fwd_bwd(_ptr(logits), dt, ld, _ptr(labels), N, V, int(ignore_index), float(g), float(denom),
                             _ptr(loss), _ptr(lse), _ptr(n_valid), _ptr(err), _ptr(ws), ws.numel(),
                             _stream(dev, stream))
    _check(st, "foak_ce_fwd_bwd")
    return dict(loss=loss, n_valid=n_valid, err=err, lse=lse)


@_on_stream
def foak_ce_count_valid(labels, V: int, *, ignore_index: int = -100, out=None, err=None, stream=None):
    """Number of labels in [0, V) (not ignore_index), as an int64 device tensor of one element
    (``out`` if given), e.g. this rank's term of a data-parallel all-reduced denominator."""
    if labels.dtype != torch.int64 or labels.dim() != 1 or not labels.is_contiguous():
        raise ValueError("labels must be a contiguous int64 vector")
    dev = labels.device
    if out is None:
        out = torch.empty(1, dtype=torch.int64, device=dev)
    if out.dtype != torch.int64 or out.numel() != 1:
        raise ValueError("out must be a one-element int64 tensor")
    st = lib.foak_ce_count_valid(_ptr(labels), labels.numel(), int(V), int(ignore_index), _ptr(out), _ptr(err),
                                 _stream(dev, stream))
    _check(st, "foak_ce_count_valid")
    return out


@_on_stream
def foak_ce_fwd_bwd_devdenom(logits, labels, denom_count, *, g: float = 1.0, ignore_index: int = -100,
                             want_lse: bool = False, workspace_tensor=None, stream=None):
    """foak_ce_fwd_bwd dividing by the int64 count in device memory ``denom_count`` (read when the
    kernel runs, e.g. after an all-reduce on the same stream).  ``loss`` is this call's share
    sum(l_i) / D.  Returns dict(loss, n_valid, err, lse)."""
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_arg(labels, N, dev)
    if denom_count.dtype != torch.int64 or denom_count.numel() != 1 or denom_count.device != dev:
        raise ValueError("denom_count must be a one-element int64 tensor on the logits' device")
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    n_valid = torch.empty(1, dtype=torch.int32, device=dev)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev) if want_lse else None
    ws = workspace(N, dev) if workspace_tensor is None else workspace_tensor
    st = lib.foak_ce_fwd_bwd_devdenom(_ptr(logits), dt, ld, _ptr(labels), N, V, int(ignore_index), float(g),
                                      _ptr(denom_count), _ptr(loss), _ptr(lse), _ptr(n_valid), _ptr(err), _ptr(ws),
                                      ws.numel(), _stream(dev, stream))
    _check(st, "foak_ce_fwd_bwd_devdenom")
    return dict(loss=loss, n_valid=n_valid, err=err, lse=lse)


def foak_ce_host_workspace_size(N: int) -> int:
    return int(lib.foak_ce_host_workspace_size(int(N)))


@_on_stream
def foak_ce_fwd_bwd_host(host_logits, host_labels, dev_logits, dev_labels, *, g: float = 1.0,
                         ignore_index: int = -100, denom: float = 0.0, workspace_tensor=None, out=None, stream=None):
    """Fused forward + backward on HOST logits: the call copies labels and logits to
    ``dev_logits`` / ``dev_labels`` in row chunks and sweeps each chunk as it lands;
    ``dev_logits`` ends holding dlogits.

    ``host_logits`` is a CPU bf16/fp32 tensor (pinned for a full-speed copy) with
    the shape and row stride of ``dev_logits``; ``host_labels`` a CPU int64 tensor.
    Returns dict(loss, n_valid, err) of pinned host tensors (pass ``out`` to reuse
    them), valid once the stream has been synchronised.
    """
    N, V, ld, dt = _logits_args(dev_logits)
    dev = dev_logits.device
    if host_logits.is_cuda or host_logits.dtype != dev_logits.dtype or host_logits.dim() != 2:
        raise ValueError("host_logits must be a CPU tensor of the device logits' dtype")
    if tuple(host_logits.shape) != (N, V) or host_logits.stride(1) != 1 or (N > 1 and host_logits.stride(0) != ld):
        raise ValueError("host_logits must have the shape and row stride of dev_logits")
    if host_labels.is_cuda or host_labels.dtype != torch.int64 or host_labels.numel() != N:
        raise ValueError("host_labels must be a CPU int64 tensor of N labels")
    if not host_labels.is_contiguous():
        raise ValueError("host_labels must be contiguous")
    dev_labels = _labels_arg(dev_labels, N, dev)
    if out is None:
        out = dict(loss=torch.empty(1, dtype=torch.float32).pin_memory(),
                   n_valid=torch.empty(1, dtype=torch.int32).pin_memory(),
                   err=torch.empty(1, dtype=torch.int32).pin_memory())
    need = foak_ce_host_workspace_size(N)
    ws = workspace(N + 64, dev) if workspace_tensor is None else workspace_tensor  # + 256 bytes of results
    if ws.numel() < need:
        raise ValueError("workspace_tensor smaller than foak_ce_host_workspace_size(N)")
    st = lib.foak_ce_fwd_bwd_host(_ptr(host_logits), dt, ld, _ptr(host_labels), N, V, int(ignore_index), float(g),
                                  float(denom), _ptr(dev_logits), _ptr(dev_labels), _ptr(out["loss"]),
                                  _ptr(out["n_valid"]), _ptr(out["err"]), _ptr(ws), ws.numel(), _stream(dev, stream))
    _check(st, "foak_ce_fwd_bwd_host")
    return out


FOAK_CE_NOALLOC_MAX_ROWS = 262144


@_on_stream
def foak_ce_fwd_bwd_noalloc(logits, labels, *, g: float = 1.0, ignore_index: int = -100, denom: float = 0.0,
                            want_lse: bool = False, stream=None):
    """Fused forward + backward in place, for callers that may not allocate device memory.

    Same result as :func:`foak_ce_fwd_bwd`, but the library takes its scratch from a
    fixed array in its own device image instead of a workspace, so no workspace
    buffer is needed (this wrapper still allocates its small output tensors with
    torch; a C caller passes its own).  N is limited to FOAK_CE_NOALLOC_MAX_ROWS,
    and calls that overlap on the GPU race on the shared scratch.
    """
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_arg(labels, N, dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    n_valid = torch.empty(1, dtype=torch.int32, device=dev)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev) if want_lse else None
    # the library uses the scratch array of the CURRENT device: make it the logits' device
    with torch.cuda.device(dev):
        st = lib.foak_ce_fwd_bwd_noalloc(_ptr(logits), dt, ld, _ptr(labels), N, V, int(ignore_index), float(g),
                                         float(denom), _ptr(loss), _ptr(lse), _ptr(n_valid), _ptr(err),
                                         _stream(dev, stream))
    _check(st, "foak_ce_fwd_bwd_noalloc")
    return dict(loss=loss, n_valid=n_valid, err=err, lse=lse)


FOAK_GEMM_BF16, FOAK_GEMM_F32, FOAK_GEMM_F32_ACC = 0, 1, 2


def foak_gemm_bf16(a, b, out, *, a_mn_major: bool = False, b_mn_major: bool = False, mode: int = FOAK_GEMM_BF16,
                   M: int | None = None, N: int | None = None, K: int | None = None, err=None, stream=None):
    """out (+)= A @ B^T on the tensor cores.  a, b: 2-D bf16 tensors with unit column stride.

    a is [M][K] (or [K][M] with a_mn_major), b is [N][K] (or [K][N] with b_mn_major);
    out is [M][N] with unit column stride, bf16 for FOAK_GEMM_BF16 else fp32.
    """
    for t in (a, b, out):
        if t.dim() != 2 or t.stride(1) != 1 or not t.is_cuda:
            raise ValueError("operands must be 2-D CUDA tensors with unit column stride")
    if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
        raise TypeError("a and b must be bfloat16")
    M = (a.shape[1] if a_mn_major else a.shape[0]) if M is None else M
    K = (a.shape[0] if a_mn_major else a.shape[1]) if K is None else K
    N = (b.shape[1] if b_mn_major else b.shape[0]) if N is None else N
    st = lib.foak_gemm_bf16(_ptr(a), a.stride(0), int(a_mn_major), _ptr(b), b.stride(0), int(b_mn_major), M, N, K,
                            _ptr(out), out.stride(0), int(mode), _ptr(err), _stream(out.device, stream))
    _check(st, "foak_gemm_bf16")
    return out


class _GemmProblem(ctypes.Structure):
    """foak_gemm_problem of the C header."""
    _fields_ = [("a", ctypes.c_void_p), ("lda", ctypes.c_int64), ("a_mn_major", ctypes.c_int32),
                ("b", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("b_mn_major", ctypes.c_int32),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("ldo", ctypes.c_int64), ("out_mode", ctypes.c_int32)]


FOAK_GEMM_GROUP_MAX = 3


def foak_gemm_bf16_group(problems, *, err=None, stream=None):
    """Several independent products out (+)= A @ B^T in one persistent launch.

    problems: sequence of dicts with keys a, b, out and optionally a_mn_major, b_mn_major,
    mode, M, N, K -- each as for foak_gemm_bf16.  No product may write what another reads.
    """
    if len(problems) > FOAK_GEMM_GROUP_MAX:
        raise ValueError(f"at most {FOAK_GEMM_GROUP_MAX} products")
    arr = (_GemmProblem * max(1, len(problems)))()
    dev = None
    for i, q in enumerate(problems):
        a, b, out = q["a"], q["b"], q["out"]
        for t in (a, b, out):
            if t.dim() != 2 or t.stride(1) != 1 or not t.is_cuda:
                raise ValueError("operands must be 2-D CUDA tensors with unit column stride")
        if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
            raise TypeError("a and b must be bfloat16")
        amn, bmn = bool(q.get("a_mn_major", False)), bool(q.get("b_mn_major", False))
        M = q.get("M", a.shape[1] if amn else a.shape[0])
        K = q.get("K", a.shape[0] if amn else a.shape[1])
        N = q.get("N", b.shape[1] if bmn else b.shape[0])
        arr[i] = _GemmProblem(_ptr(a), a.stride(0), int(amn), _ptr(b), b.stride(0), int(bmn), M, N, K, _ptr(out),
                              out.stride(0), int(q.get("mode", FOAK_GEMM_BF16)))
        dev = out.device
    st = lib.foak_gemm_bf16_group(ctypes.cast(arr, ctypes.c_void_p), len(problems), _ptr(err),
                                  _stream(dev, stream) if dev is not None else None)
    _check(st, "foak_gemm_bf16_group")


def foak_linear_ce_workspace_size(N: int, V: int, D: int, chunk: int) -> int:
    return int(lib.foak_linear_ce_workspace_size(int(N), int(V), int(D), int(chunk)))


_lin_ws: dict = {}


@_on_stream
def foak_linear_ce_chunked(H, W, labels, *, chunk: int = 1024, g: float = 1.0, ignore_index: int = -100,
                           denom: float = 0.0, dH=None, dW=None, workspace_tensor=None, stream=None):
    """Loss, dH and dW of CE(H W^T) in chunks of rows on the tensor cores.

    H: bf16 [N][D], W: bf16 [V][D] (contiguous).  Returns dict(loss, dH, dW, n_valid, err);
    dH is bf16 [N][D], dW fp32 [V][D].
    """
    if H.dtype != torch.bfloat16 or W.dtype != torch.bfloat16 or not H.is_contiguous() or not W.is_contiguous():
        raise ValueError("H and W must be contiguous bfloat16 tensors")
    N, D = H.shape
    V, D2 = W.shape
    if D2 != D:
        raise ValueError("H and W disagree on the hidden size")
    dev = H.device
    labels = _labels_arg(labels, N, dev)
    dH = torch.empty(N, D, dtype=torch.bfloat16, device=dev) if dH is None else dH
    dW = torch.empty(V, D, dtype=torch.float32, device=dev) if dW is None else dW
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    n_valid = torch.empty(1, dtype=torch.int32, device=dev)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    need = foak_linear_ce_workspace_size(N, V, D, chunk)
    ws = workspace_tensor
    if ws is None:
        ws = _cached_workspace(_lin_ws, need, dev, _stream_handle(dev, None))
    st = lib.foak_linear_ce_chunked(_ptr(H), _ptr(W), _ptr(labels), N, V, D, int(ignore_index), int(chunk), float(g),
                                    float(denom), _ptr(loss), _ptr(dH), _ptr(dW), _ptr(n_valid), _ptr(err), _ptr(ws),
                                    ws.numel(), _stream(dev, stream))
    _check(st, "foak_linear_ce_chunked")
    return dict(loss=loss, dH=dH, dW=dW, n_valid=n_valid, err=err)


# --------------------------------------------------------------------- RMSNorm
_norm_ws: dict = {}
_norm_lin_ws: dict = {}


def _rows_arg(t, name):
    if t.dim() != 2 or t.stride(1) != 1 or t.dtype not in _DT or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D bfloat16/float32 CUDA tensor with unit column stride")
    return t.shape[0], t.shape[1], (t.stride(0) if t.shape[0] > 1 else t.shape[1])


@_on_stream
def foak_rmsnorm_forward(X, gamma, *, eps: float = 1e-5, Y=None, want_rstd: bool = True, stream=None):
    """Y = X / sqrt(mean(X^2) + eps) * gamma per row (fp32 arithmetic, one rounding).

    Returns (Y, rstd); rstd (float32 [N]) is None unless ``want_rstd``.
    """
    N, D, ldx = _rows_arg(X, "X")
    if gamma.dtype != X.dtype or gamma.numel() != D or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous vector of D elements in X's dtype")
    Y = torch.empty_like(X) if Y is None else Y
    _, _, ldy = _rows_arg(Y, "Y")
    rstd = torch.empty(N, dtype=torch.float32, device=X.device) if want_rstd else None
    st = lib.foak_rmsnorm_forward(_ptr(X), _DT[X.dtype], ldx, _ptr(gamma), N, D, float(eps), _ptr(Y), ldy, _ptr(rstd),
                                  _stream(X.device, stream))
    _check(st, "foak_rmsnorm_forward")
    return Y, rstd


@_on_stream
def foak_rmsnorm_backward(dY, X, gamma, rstd, *, dX=None, want_dgamma: bool = True, stream=None):
    """dX (X's dtype) and dgamma (float32 [D], or None) of sum(dY * rmsnorm(X))."""
    N, D, lddy = _rows_arg(dY, "dY")
    _, _, ldx = _rows_arg(X, "X")
    dX = torch.empty_like(X) if dX is None else dX
    _, _, lddx = _rows_arg(dX, "dX")
    dev = X.device
    dgamma = torch.empty(D, dtype=torch.float32, device=dev) if want_dgamma else None
    need = int(lib.foak_rmsnorm_workspace_size(D))
    # partial sums only: each is written before it is read
    ws = _cached_workspace(_norm_ws, need, dev, _stream_handle(dev, None), fill=torch.empty)
    st = lib.foak_rmsnorm_backward(_ptr(dY), lddy, _ptr(X), ldx, _ptr(gamma), _ptr(rstd), _DT[X.dtype], N, D, _ptr(dX),
                                   lddx, _ptr(dgamma), _ptr(ws), ws.numel(), _stream(dev, stream))
    _check(st, "foak_rmsnorm_backward")
    return dX, dgamma


@_on_stream
def foak_rmsnorm_linear_ce_chunked(X, gamma, W, labels, *, eps: float = 1e-5, chunk: int = 1024, g: float = 1.0,
                                   ignore_index: int = -100, denom: float = 0.0, dX=None, dW=None,
                                   workspace_tensor=None, stream=None):
    """Final norm -> LM head -> CE: loss, dX, dgamma, dW of CE(rmsnorm(X, gamma) W^T).

    X: bf16 [N][D], gamma: bf16 [D], W: bf16 [V][D] (contiguous).  Returns
    dict(loss, dX, dgamma, dW, n_valid, err); dX bf16, dgamma and dW float32.
    """
    for t, n in ((X, "X"), (gamma, "gamma"), (W, "W")):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous bfloat16 tensor")
    N, D = X.shape
    V = W.shape[0]
    if W.shape[1] != D or gamma.numel() != D:
        raise ValueError("X, gamma and W disagree on the hidden size")
    dev = X.device
    labels = _labels_arg(labels, N, dev)
    dX = torch.empty_like(X) if dX is None else dX
    dW = torch.empty(V, D, dtype=torch.float32, device=dev) if dW is None else dW
    dgamma = torch.empty(D, dtype=torch.float32, device=dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    n_valid = torch.empty(1, dtype=torch.int32, device=dev)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    need = int(lib.foak_rmsnorm_linear_ce_workspace_size(N, V, D, chunk))
    ws = workspace_tensor
    if ws is None:
        ws = _cached_workspace(_norm_lin_ws, need, dev, _stream_handle(dev, None))
    st = lib.foak_rmsnorm_linear_ce_chunked(_ptr(X), _ptr(gamma), _ptr(W), _ptr(labels), N, V, D, int(ignore_index),
                                            int(chunk), float(eps), float(g), float(denom), _ptr(loss), _ptr(dX),
                                            _ptr(dgamma), _ptr(dW), _ptr(n_valid), _ptr(err), _ptr(ws), ws.numel(),
                                            _stream(dev, stream))
    _check(st, "foak_rmsnorm_linear_ce_chunked")
    return dict(loss=loss, dX=dX, dgamma=dgamma, dW=dW, n_valid=n_valid, err=err)


# --------------------------------------------------------------------- RoPE
@_on_stream
def foak_rope_cache(max_pos: int, d: int, base: float = 10000.0, device="cuda", stream=None):
    """The cos/sin table for positions [0, max_pos) and head dimension d (uint8 device tensor)."""
    need = int(lib.foak_rope_cache_size(int(max_pos), int(d)))
    if need == 0:
        raise ValueError("unsupported max_pos / d (d must be a multiple of 16)")
    dev = torch.device(device)
    cache = torch.empty(need, dtype=torch.uint8, device=dev)
    st = lib.foak_rope_build_cache(float(base), int(d), int(max_pos), _ptr(cache), need, _stream(dev, stream))
    _check(st, "foak_rope_build_cache")
    cache.max_pos, cache.head_dim = int(max_pos), int(d)
    return cache


@_on_stream
def foak_rope_apply(x, positions, cache, *, inverse: bool = False, stream=None):
    """Rotate ``x`` (T x H x d bf16/fp32 CUDA view, heads contiguous) in place by the
    angles of ``positions`` (int64 [T]); returns the device error word."""
    if x.dim() != 3 or x.stride(2) != 1 or x.stride(1) != x.shape[2] or x.dtype not in _DT or not x.is_cuda:
        raise ValueError("x must be a T x H x d CUDA view with contiguous heads")
    T, H, d = x.shape
    if d != cache.head_dim:
        raise ValueError("cache built for another head dimension")
    if positions.dtype != torch.int64 or positions.numel() != T or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int64 vector of length T")
    ldt = x.stride(0) if T > 1 else H * d
    err = torch.empty(1, dtype=torch.int32, device=x.device)
    st = lib.foak_rope_apply(_ptr(x), _DT[x.dtype], T, H, ldt, d, _ptr(positions), _ptr(cache), cache.max_pos,
                             1 if inverse else 0, _ptr(err), _stream(x.device, stream))
    _check(st, "foak_rope_apply")
    return err


@_on_stream
def foak_rope_apply_qk(q, k, positions, cache, *, inverse: bool = False, stream=None):
    """Rotate Q (T x Hq x d) and K (T x Hk x d) in place in one launch; returns the error word."""
    views = []
    for x in (q, k):
        if x.dim() != 3 or x.stride(2) != 1 or x.stride(1) != x.shape[2] or x.dtype not in _DT or not x.is_cuda:
            raise ValueError("q and k must be T x H x d CUDA views with contiguous heads")
        T, H, d = x.shape
        views.append((H, x.stride(0) if T > 1 else H * d))
    if q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2] or q.dtype != k.dtype:
        raise ValueError("q and k disagree on tokens, head dimension or dtype")
    T, _, d = q.shape
    if d != cache.head_dim:
        raise ValueError("cache built for another head dimension")
    if positions.dtype != torch.int64 or positions.numel() != T or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int64 vector of length T")
    err = torch.empty(1, dtype=torch.int32, device=q.device)
    (hq, ldq), (hk, ldk) = views
    st = lib.foak_rope_apply_qk(_ptr(q), hq, ldq, _ptr(k), hk, ldk, _DT[q.dtype], T, d, _ptr(positions), _ptr(cache),
                                cache.max_pos, 1 if inverse else 0, _ptr(err), _stream(q.device, stream))
    _check(st, "foak_rope_apply_qk")
    return err


# --------------------------------------------------------------------- log probabilities
FOAK_LOGPROBS_MAX_K = 256
_HEADER_BYTES = int(lib.foak_logprobs_workspace_size())


def _labels_or_none(labels, N, device):
    return None if labels is None else _labels_arg(labels, N, device)


def _row_vector(t, n, device, name):
    if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} elements on the logits' device")
    return t


def _dlogits_arg(dlogits, logits, N, V, ld):
    """``dlogits``, or a new tensor of the logits' strides and offset modulo 16 bytes."""
    if dlogits is None:
        shift = (logits.data_ptr() % 16) // logits.element_size()
        n = ((N - 1) * ld + V + shift) if N > 0 else 1
        base = torch.empty(n, dtype=logits.dtype, device=logits.device)
        return base.as_strided((N, V), (ld, 1), storage_offset=shift)
    if dlogits.shape != logits.shape or dlogits.stride() != logits.stride() or dlogits.dtype != logits.dtype:
        raise ValueError("dlogits must match logits in shape, strides and dtype")
    if dlogits.device != logits.device:
        raise ValueError("dlogits must live on the logits' device")
    return dlogits


@_on_stream
def foak_logprobs_forward(logits, labels=None, *, top_k: int = 0, temperature: float = 1.0, ignore_index: int = -100,
                          want_entropy: bool = True, want_lse: bool = True, want_stats: bool = True,
                          workspace_tensor=None, stream=None):
    """Log probability of each row's token, entropy, log-sum-exp and the top_k most likely tokens.

    ``labels`` (int64 [N]) are the given tokens; None computes every row and leaves logp out.
    Returns dict(logp, entropy, lse, stats, top_logprobs, top_ids, err): float32 [N] each,
    stats [N, 2] for :func:`foak_logprobs_backward`, the tops [N, top_k] (ids int32, in
    descending order, equal logits by the lower id); what was not asked for is None.  Rows
    whose label is ``ignore_index`` are not read: 0, and top ids -1.
    """
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_or_none(labels, N, dev)
    K = int(top_k)
    if K < 0 or K > min(V, FOAK_LOGPROBS_MAX_K):
        raise ValueError(f"top_k must be between 0 and min(V, {FOAK_LOGPROBS_MAX_K})")
    f32 = torch.float32
    logp = torch.empty(N, dtype=f32, device=dev) if labels is not None else None
    entropy = torch.empty(N, dtype=f32, device=dev) if want_entropy else None
    lse = torch.empty(N, dtype=f32, device=dev) if want_lse else None
    stats = torch.empty(N, 2, dtype=f32, device=dev) if want_stats else None
    top_lp = torch.empty(N, K, dtype=f32, device=dev) if K else None
    top_ids = torch.empty(N, K, dtype=torch.int32, device=dev) if K else None
    err = torch.empty(1, dtype=torch.int32, device=dev)
    handle = _stream_handle(dev, stream)
    ws = _workspace_or_cached(workspace_tensor, _HEADER_BYTES, dev, handle)
    st = lib.foak_logprobs_forward(_addr(logits), dt, ld, _addr(labels), N, V, int(ignore_index), float(temperature), K,
                                   _addr(logp), _addr(entropy), _addr(lse), _addr(stats), _addr(top_lp),
                                   _addr(top_ids), _addr(err), _addr(ws), ws.numel(), handle)
    _check(st, "foak_logprobs_forward")
    return dict(logp=logp, entropy=entropy, lse=lse, stats=stats, top_logprobs=top_lp, top_ids=top_ids, err=err)


@_on_stream
def foak_logprobs_backward(logits, labels, stats, grad_logp=None, entropy=None, grad_entropy=None, *,
                           temperature: float = 1.0, ignore_index: int = -100, dlogits=None, stream=None):
    """Gradient of sum(grad_logp * logp + grad_entropy * entropy); returns (dlogits, err).

    ``stats`` and ``entropy`` come from :func:`foak_logprobs_forward` at the same temperature;
    a gradient that is None is zero.  Pass ``dlogits=logits`` to overwrite in place.
    """
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_arg(labels, N, dev)
    _row_vector(stats, 2 * N, dev, "stats")
    for t, name in ((grad_logp, "grad_logp"), (entropy, "entropy"), (grad_entropy, "grad_entropy")):
        if t is not None:
            _row_vector(t, N, dev, name)
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs the forward's entropy")
    dlogits = _dlogits_arg(dlogits, logits, N, V, ld)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    st = lib.foak_logprobs_backward(_addr(dlogits), _addr(logits), dt, ld, _addr(labels), N, V, int(ignore_index),
                                    float(temperature), _addr(stats), _addr(grad_logp), _addr(entropy),
                                    _addr(grad_entropy), _addr(err), _stream_handle(dev, stream))
    _check(st, "foak_logprobs_backward")
    return dlogits, err


# --------------------------------------------------------------------- distillation
FOAK_DISTILL_MAX_K = 256


def _teacher_args(ids, logprobs, N, device):
    if ids.dim() != 2 or ids.dtype != torch.int32 or logprobs.dim() != 2 or logprobs.dtype != torch.float32:
        raise ValueError("teacher_ids must be int32 and teacher_logprobs float32, both N x K")
    if ids.shape != logprobs.shape or ids.shape[0] != N:
        raise ValueError("teacher_ids, teacher_logprobs and the logits disagree on the rows or K")
    if ids.device != device or logprobs.device != device:
        raise ValueError("the teacher's tensors must live on the logits' device")
    K = ids.shape[1]
    if K < 1 or K > FOAK_DISTILL_MAX_K:
        raise ValueError(f"K must be between 1 and {FOAK_DISTILL_MAX_K}")
    if K > 1 and (ids.stride(1) != 1 or logprobs.stride(1) != 1):
        raise ValueError("the teacher's rows must have unit column stride")
    if N > 1 and ids.stride(0) != logprobs.stride(0):
        raise ValueError("teacher_ids and teacher_logprobs must have the same row stride")
    return K, (ids.stride(0) if N > 1 else K)


@_on_stream
def foak_distill_forward(logits, labels, teacher_ids, teacher_logprobs, *, ce_weight: float = 0.0,
                         kd_weight: float = 1.0, temperature: float = 1.0, normalize: bool = True,
                         ignore_index: int = -100, denom: float = 0.0, want_rows: bool = False,
                         want_stats: bool = True, workspace_tensor=None, stream=None):
    """Mean over valid rows of ce_weight CE + kd_weight KD against the teacher's top tokens.

    ``teacher_ids`` (int32 [N, K], negative: padding) and ``teacher_logprobs`` (float32 [N, K])
    are the top_ids and top_logprobs of :func:`foak_logprobs_forward` at ``temperature``, or
    rows of the same row stride; ``normalize`` rescales each row's K probabilities to sum 1.
    ``labels`` may be None (every row counts) when ``ce_weight`` is 0.  Returns dict(loss,
    row_ce, row_kd, stats, n_valid, err); stats is for :func:`foak_distill_backward`.
    """
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_or_none(labels, N, dev)
    K, ldt = _teacher_args(teacher_ids, teacher_logprobs, N, dev)
    f32 = torch.float32
    loss = torch.empty(1, dtype=f32, device=dev)
    row_ce = torch.empty(N, dtype=f32, device=dev) if want_rows else None
    row_kd = torch.empty(N, dtype=f32, device=dev) if want_rows else None
    stats = torch.empty(N, 4, dtype=f32, device=dev) if want_stats else None
    n_valid = torch.empty(1, dtype=torch.int32, device=dev)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    handle = _stream_handle(dev, stream)
    ws = _workspace_or_cached(workspace_tensor, foak_ce_workspace_size(N), dev, handle)
    st = lib.foak_distill_forward(_addr(logits), dt, ld, _addr(labels), N, V, int(ignore_index), _addr(teacher_ids),
                                  _addr(teacher_logprobs), ldt, K, int(bool(normalize)), float(ce_weight),
                                  float(kd_weight), float(temperature), float(denom), _addr(loss), _addr(row_ce),
                                  _addr(row_kd), _addr(stats), _addr(n_valid), _addr(err), _addr(ws), ws.numel(), handle)
    _check(st, "foak_distill_forward")
    return dict(loss=loss, row_ce=row_ce, row_kd=row_kd, stats=stats, n_valid=n_valid, err=err)


@_on_stream
def foak_distill_fwd_bwd(logits, labels, teacher_ids, teacher_logprobs, *, ce_weight: float = 0.0,
                         kd_weight: float = 1.0, temperature: float = 1.0, normalize: bool = True, g: float = 1.0,
                         ignore_index: int = -100, denom: float = 0.0, dlogits=None, want_rows: bool = False,
                         workspace_tensor=None, stream=None):
    """:func:`foak_distill_forward` and its gradient times ``g`` in one call.

    The gradient overwrites ``logits``, or goes to ``dlogits`` (same strides) if given.
    Returns dict(loss, dlogits, row_ce, row_kd, n_valid, err).
    """
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_or_none(labels, N, dev)
    K, ldt = _teacher_args(teacher_ids, teacher_logprobs, N, dev)
    dlogits = logits if dlogits is None else _dlogits_arg(dlogits, logits, N, V, ld)
    f32 = torch.float32
    loss = torch.empty(1, dtype=f32, device=dev)
    row_ce = torch.empty(N, dtype=f32, device=dev) if want_rows else None
    row_kd = torch.empty(N, dtype=f32, device=dev) if want_rows else None
    n_valid = torch.empty(1, dtype=torch.int32, device=dev)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    handle = _stream_handle(dev, stream)
    ws = _workspace_or_cached(workspace_tensor, foak_ce_workspace_size(N), dev, handle)
    st = lib.foak_distill_fwd_bwd(_addr(logits), _addr(dlogits), dt, ld, _addr(labels), N, V, int(ignore_index),
                                  _addr(teacher_ids), _addr(teacher_logprobs), ldt, K, int(bool(normalize)),
                                  float(ce_weight), float(kd_weight), float(temperature), float(g), float(denom),
                                  _addr(loss), _addr(row_ce), _addr(row_kd), _addr(n_valid), _addr(err), _addr(ws),
                                  ws.numel(), handle)
    _check(st, "foak_distill_fwd_bwd")
    return dict(loss=loss, dlogits=dlogits, row_ce=row_ce, row_kd=row_kd, n_valid=n_valid, err=err)


@_on_stream
def foak_distill_backward(logits, labels, teacher_ids, teacher_logprobs, stats, grad_out=None, *,
                          ce_weight: float = 0.0, kd_weight: float = 1.0, temperature: float = 1.0,
                          normalize: bool = True, ignore_index: int = -100, denom: float = 0.0, dlogits=None,
                          stream=None):
    """The gradient of :func:`foak_distill_forward` from its ``stats``, times ``grad_out`` (a
    float32 scalar tensor, or None for 1); the other arguments as given there.  Returns
    (dlogits, err).  Pass ``dlogits=logits`` to overwrite in place."""
    N, V, ld, dt = _logits_args(logits)
    dev = logits.device
    labels = _labels_or_none(labels, N, dev)
    K, ldt = _teacher_args(teacher_ids, teacher_logprobs, N, dev)
    _row_vector(stats, 4 * N, dev, "stats")
    if grad_out is not None and (grad_out.dtype != torch.float32 or grad_out.numel() != 1 or grad_out.device != dev):
        raise ValueError("grad_out must be a float32 scalar tensor on the logits' device")
    dlogits = _dlogits_arg(dlogits, logits, N, V, ld)
    err = torch.empty(1, dtype=torch.int32, device=dev)
    st = lib.foak_distill_backward(_addr(dlogits), _addr(logits), dt, ld, _addr(labels), N, V, int(ignore_index),
                                   _addr(teacher_ids), _addr(teacher_logprobs), ldt, K, int(bool(normalize)),
                                   float(ce_weight), float(kd_weight), float(temperature), _addr(stats),
                                   _addr(grad_out), float(denom), _addr(err), _stream_handle(dev, stream))
    _check(st, "foak_distill_backward")
    return dlogits, err


# --------------------------------------------------------------------- residual norms
# The calls from here on are often a few microseconds' work on the GPU, so what they check of a
# tensor they ask once, devices are compared by number (a CPU tensor's is -1), and the step that a
# ``stream`` of the caller's takes (:func:`_on_stream`) stands in the call itself.
FOAK_GATE_NONE, FOAK_GATE_CHANNEL, FOAK_GATE_ROW, FOAK_GATE_FULL = 0, 1, 2, 3
FOAK_RESIDUAL_NORM_MAX_D = 32768
_resnorm_ws: dict = {}
_resnorm_lock = threading.Lock()  # a backward's two launches, which hand partial sums on in a workspace
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(di, call, *args):
    """``call(*args, stream)`` on device ``di``'s current stream, with that device as the current one, as a
    launch wants."""
    if di == _current_device():
        return call(*args, _handle_of(di))
    with torch.cuda.device(di):
        return call(*args, _handle_of(di))


def _handle_of(di):
    return torch.cuda.current_stream(di).cuda_stream if _raw_stream is None else _raw_stream(di)


@functools.lru_cache(maxsize=1024)
def foak_residual_norm_workspace_size(N: int, D: int) -> int:
    return int(lib.foak_residual_norm_workspace_size(int(N), int(D)))


def _row_stride(t, shape, dtype, di, name):
    """The row stride of a tensor of this shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != di:
        raise ValueError(f"{name} must be like the other rows: shape, dtype and device")
    ld, unit = t.stride()
    if unit != 1:
        raise ValueError(f"{name} must have unit column stride")
    return ld if shape[0] > 1 else shape[1]


def _channels(t, D, dtype, di, name):
    """The address of a vector of D channels."""
    if t.dim() != 1 or t.numel() != D or t.dtype != dtype or t.get_device() != di or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of D elements in the rows' dtype, on their device")
    return t.data_ptr()


def _gate_arg(gate, shape, dtype, di):
    """(address, kind, stride): [D] is a gate a channel, [N, 1] one a row, [N, D] one an element."""
    if gate is None:
        return None, FOAK_GATE_NONE, 0
    N, D = shape
    if gate.dim() == 1:
        return _channels(gate, D, dtype, di, "gate"), FOAK_GATE_CHANNEL, 0
    if gate.shape == (N, 1):
        if gate.dtype != dtype or gate.get_device() != di:
            raise ValueError("gate must have the rows' dtype and device")
        return gate.data_ptr(), FOAK_GATE_ROW, (gate.stride(0) if N > 1 else 1)
    return gate.data_ptr(), FOAK_GATE_FULL, _row_stride(gate, shape, dtype, di, "gate")


def _rstd_arg(t, N, di, name):
    if t.dtype != torch.float32 or t.numel() != N or t.get_device() != di or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 vector of the N rows, on their device")
    return t.data_ptr()


def foak_residual_norm_forward(X, R, gamma=None, *, gate=None, post_gamma=None, scale: float = 1.0, eps: float = 1e-5,
                               post_eps: float | None = None, H=None, Y=None, want_rstd: bool = True, stream=None):
    """H = R + scale * gate * u with u = X, or the RMSNorm of X by ``post_gamma``; Y = RMSNorm of H by ``gamma``.

    X is a block's output, R the residual stream (bf16 or fp32, N x D), Y the next block's input,
    computed from H before it is rounded.  ``gate`` is [D], [N, 1], [N, D] or None; without
    ``gamma`` there is no Y.  ``H=R`` (or X) updates the stream in place.  ``post_eps`` defaults to
    ``eps``.  Returns dict(H, Y, rstd, post_rstd); the last two (float32 [N]) are for
    :func:`foak_residual_norm_backward`, None unless ``want_rstd`` and their norm is there.
    """
    if stream is not None:
        return _run_on(stream, foak_residual_norm_forward, (X, R, gamma),
                       dict(gate=gate, post_gamma=post_gamma, scale=scale, eps=eps, post_eps=post_eps, H=H, Y=Y,
                            want_rstd=want_rstd))
    N, D, ldx = _rows_arg(X, "X")
    shape, dtype, di = X.shape, X.dtype, X.get_device()
    ldr = _row_stride(R, shape, dtype, di, "R")
    g, kind, ldg = _gate_arg(gate, shape, dtype, di)
    pg = None if post_gamma is None else _channels(post_gamma, D, dtype, di, "post_gamma")
    H = X.new_empty(shape) if H is None else H
    ldh = _row_stride(H, shape, dtype, di, "H")
    gm = y = rstd = post = r = r1 = None
    ldy = 0
    if gamma is not None:
        gm = _channels(gamma, D, dtype, di, "gamma")
        Y = X.new_empty(shape) if Y is None else Y
        ldy = _row_stride(Y, shape, dtype, di, "Y")
        y = Y.data_ptr()
        if want_rstd:
            rstd = torch.empty(N, dtype=torch.float32, device=X.device)
            r = rstd.data_ptr()
    elif Y is not None:
        raise ValueError("Y needs gamma")
    if want_rstd and pg is not None:
        post = torch.empty(N, dtype=torch.float32, device=X.device)
        r1 = post.data_ptr()
    st = _launch(di, lib.foak_residual_norm_forward, X.data_ptr(), ldx, R.data_ptr(), ldr, _DT[dtype], N, D, g, kind, ldg,
                 pg, gm, scale, eps if post_eps is None else post_eps, eps, H.data_ptr(), ldh, y, ldy, r1, r)
    if st:
        _check(st, "foak_residual_norm_forward")
    return dict(H=H, Y=Y, rstd=rstd, post_rstd=post)


def foak_residual_norm_backward(dY, dH, H=None, rstd=None, gamma=None, *, X=None, gate=None, post_gamma=None,
                                post_rstd=None, scale: float = 1.0, dR=None, dX=None, want_dX: bool = True,
                                want_dgate: bool = True, want_dgamma: bool = True, workspace_tensor=None, stream=None):
    """Gradients of :func:`foak_residual_norm_forward` from ``dY`` and from ``dH``, what arrives along
    the residual stream (either may be None: zero; without ``dY``, H, rstd and gamma are not needed).

    H, rstd and post_rstd are the forward's; X is needed with ``post_gamma`` or for the gate's
    gradient; the other arguments as given there.  Returns dict(dR, dX, dgamma, dgate,
    dpost_gamma): dR and dX like the rows; dgamma, dpost_gamma float32 [D]; dgate float32 [D] or
    [N, 1], or like a full gate.  Without gate and ``post_gamma`` and with ``scale`` 1, dX is dR,
    the same tensor, unless ``dX`` is given.
    """
    if stream is not None:
        return _run_on(stream, foak_residual_norm_backward, (dY, dH, H, rstd, gamma),
                       dict(X=X, gate=gate, post_gamma=post_gamma, post_rstd=post_rstd, scale=scale, dR=dR, dX=dX,
                            want_dX=want_dX, want_dgate=want_dgate, want_dgamma=want_dgamma,
                            workspace_tensor=workspace_tensor))
    like = dH if dY is None else dY
    if like is None:
        raise ValueError("dY or dH must be given")
    N, D, ld = _rows_arg(like, "dY or dH")
    shape, dtype, di, dev, f32 = like.shape, like.dtype, like.get_device(), like.device, torch.float32
    lddy = lddh = ldh = ldx = lddx = lddg = 0
    dy = dh = h = x = pg = gm = r = r1 = dx = a = b = c = None
    g, kind, ldg = _gate_arg(gate, shape, dtype, di)
    dgamma = dpost = dgate = None
    if dY is not None:
        if H is None or rstd is None or gamma is None:
            raise ValueError("dY needs the forward's H, rstd and gamma")
        dy, lddy, h, ldh = dY.data_ptr(), ld, H.data_ptr(), _row_stride(H, shape, dtype, di, "H")
        r, gm = _rstd_arg(rstd, N, di, "rstd"), _channels(gamma, D, dtype, di, "gamma")
        if want_dgamma:
            dgamma = torch.empty(D, dtype=f32, device=dev)
            a = dgamma.data_ptr()
    if dH is not None:
        dh, lddh = dH.data_ptr(), (_row_stride(dH, shape, dtype, di, "dH") if dH is not like else ld)
    want_dgate = want_dgate and gate is not None
    if post_gamma is not None or want_dgate:
        if X is None:
            raise ValueError("post_gamma and the gate's gradient need X")
        x, ldx = X.data_ptr(), _row_stride(X, shape, dtype, di, "X")
    if post_gamma is not None:
        if post_rstd is None:
            raise ValueError("post_gamma needs the forward's post_rstd")
        pg, r1 = _channels(post_gamma, D, dtype, di, "post_gamma"), _rstd_arg(post_rstd, N, di, "post_rstd")
        if want_dgamma:
            dpost = torch.empty(D, dtype=f32, device=dev)
            c = dpost.data_ptr()
    if want_dgate:
        if kind == FOAK_GATE_FULL:
            dgate, lddg = like.new_empty(shape), D
        else:
            dgate = torch.empty((D,) if kind == FOAK_GATE_CHANNEL else (N, 1), dtype=f32, device=dev)
        b = dgate.data_ptr()
    dR = like.new_empty(shape) if dR is None else dR
    lddr = _row_stride(dR, shape, dtype, di, "dR")
    same = dX is None and gate is None and post_gamma is None and scale == 1.0
    if dX is None and want_dX and not same:
        dX = like.new_empty(shape)
    if dX is not None:
        dx, lddx = dX.data_ptr(), _row_stride(dX, shape, dtype, di, "dX")
    need = foak_residual_norm_workspace_size(N, D)
    if workspace_tensor is None:  # partial sums only: each is written before it is read
        ws = _cached_workspace(_resnorm_ws, need, dev, _handle_of(di), fill=torch.empty)
    else:
        ws = _workspace_arg(workspace_tensor, dev)
    with _resnorm_lock:
        st = _launch(di, lib.foak_residual_norm_backward, dy, lddy, dh, lddh, h, ldh, x, ldx, _DT[dtype], N, D, g, kind,
                     ldg, pg, gm, r1, r, scale, dR.data_ptr(), lddr, dx, lddx, a, b, lddg, c, ws.data_ptr(), ws.numel())
    if st:
        _check(st, "foak_residual_norm_backward")
    return dict(dR=dR, dX=dR if same and want_dX else dX, dgamma=dgamma, dgate=dgate, dpost_gamma=dpost)


# --------------------------------------------------------------------- rotary positions
FOAK_ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "ramp": 4}


class RotaryPlan:
    """What :func:`foak_rotary_apply` and :func:`foak_kv_append` need of a model's rotary embedding: made once
    by :func:`foak_rotary_plan` and kept as long as a graph that was captured with it is replayed."""

    __slots__ = ("turns", "rotary_dim", "interleaved", "factor", "inv_freq", "device_index")

    def __init__(self, turns, rotary_dim, interleaved, factor, inv_freq):
        self.turns, self.rotary_dim, self.interleaved = turns, rotary_dim, interleaved
        self.factor, self.inv_freq, self.device_index = factor, inv_freq, turns.get_device()


def foak_rotary_inv_freq(rotary_dim: int, *, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                         low: float = 1.0, high: float | None = None, original: float = 0.0):
    """The rotary_dim / 2 angles a position (a list of floats): base^(-2i / rotary_dim), scaled for contexts
    ``factor`` times ``original`` positions.  ``scaling``: "none"; "linear" (positions divided by the factor);
    "ntk" (a larger base); "bands" (by the turns a frequency makes over ``original`` positions: stretched below
    ``low``, kept above ``high``, 4 unless given); "ramp" (the same along the frequencies' index, ``high`` 32).
    """
    if scaling not in FOAK_ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(FOAK_ROTARY_SCALINGS)}")
    if rotary_dim < 2 or rotary_dim % 2 or rotary_dim > 65536:
        raise ValueError("rotary_dim must be even, between 2 and 65536")
    out = (ctypes.c_double * (rotary_dim // 2))()
    high = (32.0 if scaling == "ramp" else 4.0) if high is None else high
    _check(lib.foak_rotary_inv_freq(base, rotary_dim, FOAK_ROTARY_SCALINGS[scaling], factor, low, high, original, out),
           "foak_rotary_inv_freq")
    return list(out)


def foak_rotary_turns(inv_freq):
    """Angles a position as the device calls take them: int64 (fractions of a turn, times 2^64), on the CPU."""
    n = len(inv_freq)
    turns = (ctypes.c_int64 * n)()
    _check(lib.foak_rotary_turns((ctypes.c_double * n)(*inv_freq), n, turns), "foak_rotary_turns")
    return torch.tensor(list(turns), dtype=torch.int64)


def foak_rotary_plan(rotary_dim: int, *, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                     factor: float = 1.0, low: float = 1.0, high: float | None = None, original: float = 0.0,
                     inv_freq=None, attention_factor: float | None = None, device="cuda") -> RotaryPlan:
    """A rotary embedding of a head's first ``rotary_dim`` elements, in pairs (i, i + rotary_dim / 2), or
    (2i, 2i + 1) where ``interleaved``.

    The frequencies are :func:`foak_rotary_inv_freq`'s, or ``inv_freq`` itself (rotary_dim / 2 numbers).
    ``attention_factor`` multiplies what is rotated; by default 1, and 0.1 ln(factor) + 1 for "ramp".
    """
    if inv_freq is None:
        inv_freq = foak_rotary_inv_freq(rotary_dim, base=base, scaling=scaling, factor=factor, low=low, high=high,
                                        original=original)
    else:
        inv_freq = [float(f) for f in inv_freq]
        if rotary_dim < 2 or rotary_dim % 2 or rotary_dim > 65536 or len(inv_freq) != rotary_dim // 2:
            raise ValueError("inv_freq must have rotary_dim / 2 numbers")
    if attention_factor is None:
        attention_factor = 0.1 * math.log(factor) + 1.0 if scaling == "ramp" else 1.0
    if not math.isfinite(attention_factor):
        raise ValueError("attention_factor must be finite")
    dev = _device_of(device)
    turns = foak_rotary_turns(inv_freq).to(dev)
    if dev.type == "cuda":
        torch.cuda.current_stream(dev).synchronize()  # any stream may use the plan from here on
    return RotaryPlan(turns, int(rotary_dim), bool(interleaved), float(attention_factor), inv_freq)


def _heads_arg(x, dtype, di, T, name):
    """(heads, elements, token stride, head stride) of a T x H x d view of this type, device and T."""
    if x.dim() != 3 or x.dtype != dtype or x.get_device() != di:
        raise ValueError(f"{name} must be T x H x d, of the other heads' dtype and device")
    tokens, H, d = x.shape
    ldt, ldh, unit = x.stride()
    if tokens != T or (unit != 1 and d > 1):
        raise ValueError(f"{name} must have the other heads' tokens, and unit stride along a head")
    if H == 1:
        ldh = d
    return H, d, (ldt if T > 1 else max(1, H * d)), ldh


def _first_heads(x, name):
    """(type, device, tokens) that the other tensors have to share."""
    if x.dim() != 3 or x.dtype not in _DT or not x.is_cuda:
        raise ValueError(f"{name} must be a T x H x d bfloat16/float32 CUDA view whose heads have unit stride")
    return x.dtype, x.get_device(), x.shape[0]


def _plan_arg(plan, d, di):
    if plan.device_index != di:
        raise ValueError("the plan must live on the heads' device")
    if plan.rotary_dim > d:
        raise ValueError("the plan rotates more elements than a head has")
    return plan.turns.data_ptr()


def _tokens_arg(t, T, di, name):
    if t.dtype != torch.int64 or t.dim() != 1 or t.numel() != T or t.get_device() != di or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int64 vector of the T tokens, on the heads' device")
    return t.data_ptr()


def _heads_out(x, out, dtype, di, T, name):
    """(output, token stride, head stride): ``out``, x itself among them, or a new contiguous tensor."""
    if out is None:
        out = torch.empty(x.shape, dtype=dtype, device=x.device)
    elif out.shape != x.shape:
        raise ValueError(f"{name} must have its input's shape")
    _, _, ldt, ldh = _heads_arg(out, dtype, di, T, name)
    return out, ldt, ldh


def foak_rotary_apply(plan, positions, q, k=None, *, q_out=None, k_out=None, inverse: bool = False, stream=None):
    """Rotate ``q`` (T x Hq x d) and ``k`` (T x Hk x d) by the angles of ``positions`` (int64 [T]) in one
    launch; with ``inverse`` back by the same angles, which is the gradients' way.

    Views of any token and head strides (a fused QKV product's parts, heads first or tokens first).
    Returns (q_out, k_out): new tensors unless given; ``q_out=q`` rotates in place.  Either of q and k may be None.
    """
    if stream is not None:
        return _run_on(stream, foak_rotary_apply, (plan, positions, q, k),
                       dict(q_out=q_out, k_out=k_out, inverse=inverse))
    if q is None and k is None:
        raise ValueError("q or k must be given")
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("an output without its input")
    dtype, di, T = _first_heads(*((q, "q") if k is None or q is not None else (k, "k")))
    qp = kp = qo = ko = None
    Hq = ldq = ldqh = ldqo = ldqoh = Hk = ldk = ldkh = ldko = ldkoh = 0
    if q is not None:
        Hq, d, ldq, ldqh = _heads_arg(q, dtype, di, T, "q")
        q_out, ldqo, ldqoh = _heads_out(q, q_out, dtype, di, T, "q_out")
        qp, qo = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        Hk, dk, ldk, ldkh = _heads_arg(k, dtype, di, T, "k")
        if q is not None and dk != d:
            raise ValueError("q and k disagree on the head dimension")
        d = dk
        k_out, ldko, ldkoh = _heads_out(k, k_out, dtype, di, T, "k_out")
        kp, ko = k.data_ptr(), k_out.data_ptr()
    st = _launch(di, lib.foak_rotary_apply, qp, ldq, ldqh, qo, ldqo, ldqoh, Hq, kp, ldk, ldkh, ko, ldko, ldkoh, Hk,
                 _DT[dtype], T, d, plan.rotary_dim, plan.interleaved, _tokens_arg(positions, T, di, "positions"),
                 _plan_arg(plan, d, di), plan.factor, inverse)
    if st:
        _check(st, "foak_rotary_apply")
    return q_out, k_out


# --------------------------------------------------------------------- paged cache
def _int32_arg(t, di, name):
    if t.dtype != torch.int32 or t.get_device() != di or t.stride()[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be int32 with unit stride, on the page table's device")
    return t.data_ptr()


def _err_arg(err, di):
    """The address of a caller's error word."""
    if err.dtype != torch.int32 or err.numel() != 1 or err.get_device() != di:
        raise ValueError("err must be a one-element int32 tensor on the tensors' device")
    return err.data_ptr()


def foak_kv_slots(page_table, cache_lens, seq_starts, T: int, *, page_size: int, num_pages: int, err=None, stream=None):
    """Slots and positions of a serving step's T tokens in a paged cache, for the appends of all its layers.

    ``page_table`` (int32 [B, max_pages]) lists each sequence's pages, ``cache_lens`` (int32 [B]) its tokens
    in the cache before the step, ``seq_starts`` (int32 [B + 1], ascending) its first row.  Token t of sequence
    b has position cache_lens[b] + t - seq_starts[b] and slot page * page_size + place; rows of no sequence are
    padding: slot -1.  Returns dict(slots, positions, err): int64 [T] each; a page that is missing or not in
    [0, num_pages) gives slot -1 and sets FOAK_ERRBIT_PAGE_RANGE in ``err``, which is OR-ed into: pass
    a zeroed int32 tensor to keep one for many calls.
    """
    if stream is not None:
        return _run_on(stream, foak_kv_slots, (page_table, cache_lens, seq_starts, T),
                       dict(page_size=page_size, num_pages=num_pages, err=err))
    di = page_table.get_device()
    if di < 0 or page_table.dim() != 2 or cache_lens.dim() != 1 or seq_starts.dim() != 1:
        raise ValueError("page_table (2-D), cache_lens and seq_starts (1-D) must be on a CUDA device")
    B, most = page_table.shape
    if cache_lens.numel() != B or seq_starts.numel() != B + 1:
        raise ValueError("page_table, cache_lens and seq_starts disagree on the sequences")
    T, dev = int(T), page_table.device
    if T < 0:
        raise ValueError("T must not be negative")
    slots = torch.empty(T, dtype=torch.int64, device=dev)
    positions = torch.empty(T, dtype=torch.int64, device=dev)
    if err is None:
        err = torch.zeros(1, dtype=torch.int32, device=dev)
    st = _launch(di, lib.foak_kv_slots, _int32_arg(page_table, di, "page_table"), page_table.stride(0) if B > 1 else most,
                 most, _int32_arg(cache_lens, di, "cache_lens"), _int32_arg(seq_starts, di, "seq_starts"), B, T, page_size,
                 num_pages, slots.data_ptr(), positions.data_ptr(), _err_arg(err, di))
    if st:
        _check(st, "foak_kv_slots")
    return dict(slots=slots, positions=positions, err=err)


def _cache_arg(cache, dtype, di, H, d, heads_first, name):
    """(pages, places, page stride, place stride, head stride) of a cache of H heads of d elements."""
    if cache.dim() != 4 or cache.dtype != dtype or cache.get_device() != di:
        raise ValueError(f"{name} must be 4-D, of the heads' dtype and device")
    pages, places, heads, size = cache.shape
    ld_page, ld_place, ld_head, unit = cache.stride()
    if heads_first:
        places, heads, ld_place, ld_head = heads, places, ld_head, ld_place
    if heads != H or size != d:
        raise ValueError(f"{name} disagrees with its rows on the heads or their size")
    if unit != 1 and d > 1:
        raise ValueError(f"{name} must have unit stride along a head")
    return pages, places, ld_page, ld_place, ld_head


def foak_kv_append(k, v, k_cache, v_cache, slots, *, heads_first: bool = False, plan=None, positions=None, q=None,
                   q_out=None, err=None, stream=None):
    """Append a step's keys and values to one layer's paged cache; with ``plan`` the keys are rotated on
    the way by ``positions``, and ``q`` beside them, in the same launch.

    k (T x Hk x d) and v (T x Hk x dv) are views of any token and head strides; the caches are
    (pages, page_size, Hk, d), or (pages, Hk, page_size, d) with ``heads_first``, views too.  ``slots`` and
    ``positions`` are :func:`foak_kv_slots`'s; of a token with a negative slot nothing is written, q's row
    of ``q_out`` neither (in a new tensor it is undefined).  Returns q_out (a new tensor unless given, None
    without q).  A slot past the cache sets FOAK_ERRBIT_PAGE_RANGE in ``err`` (OR-ed into), if given, and is
    left out.
    """
    if stream is not None:
        return _run_on(stream, foak_kv_append, (k, v, k_cache, v_cache, slots),
                       dict(heads_first=heads_first, plan=plan, positions=positions, q=q, q_out=q_out, err=err))
    dtype, di, T = _first_heads(k, "k")
    Hk, d, ldk, ldkh = _heads_arg(k, dtype, di, T, "k")
    Hv, dv, ldv, ldvh = _heads_arg(v, dtype, di, T, "v")
    if Hv != Hk:
        raise ValueError("k and v disagree on the heads")
    pages, places, ldk_page, ldk_place, ldk_head = _cache_arg(k_cache, dtype, di, Hk, d, heads_first, "k_cache")
    v_pages, v_places, ldv_page, ldv_place, ldv_head = _cache_arg(v_cache, dtype, di, Hk, dv, heads_first, "v_cache")
    if pages != v_pages or places != v_places:
        raise ValueError("k_cache and v_cache disagree on pages or page size")
    Hq = ldq = ldqh = ldqo = ldqoh = r = 0
    qp = qo = at = turns = None
    interleaved, factor = False, 1.0
    if plan is not None:
        if positions is None:
            raise ValueError("a rotation needs positions")
        at, turns = _tokens_arg(positions, T, di, "positions"), _plan_arg(plan, d, di)
        r, interleaved, factor = plan.rotary_dim, plan.interleaved, plan.factor
    if q is not None:
        if plan is None:
            raise ValueError("q is there to be rotated: it needs a plan")
        Hq, dq, ldq, ldqh = _heads_arg(q, dtype, di, T, "q")
        if dq != d:
            raise ValueError("q and k disagree on the head dimension")
        q_out, ldqo, ldqoh = _heads_out(q, q_out, dtype, di, T, "q_out")
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    st = _launch(di, lib.foak_kv_append, k.data_ptr(), ldk, ldkh, v.data_ptr(), ldv, ldvh, Hk, _DT[dtype], T, d, dv,
                 _tokens_arg(slots, T, di, "slots"), k_cache.data_ptr(), ldk_page, ldk_place, ldk_head,
                 v_cache.data_ptr(), ldv_page, ldv_place, ldv_head, pages, places, qp, ldq, ldqh, qo, ldqo, ldqoh, Hq, r,
                 interleaved, at, turns, factor, None if err is None else _err_arg(err, di))
    if st:
        _check(st, "foak_kv_append")
    return q_out
